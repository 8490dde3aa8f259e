// The paged FP8 key/value cache: what the appending and the attention kernels
// share, and their launchers.
#pragma once

#include "common.hpp"

namespace fp8q {

// A scale of the cache counts as the nearest value of this range (NaN as the
// lowest): both ends and their reciprocals are normal fp32 numbers, with room
// for a code's or a softmax term's own exponent.
constexpr float kMinPageScale = 0x1p-100f, kMaxPageScale = 0x1p100f;
constexpr int kMinPageExp = -100, kMaxPageExp = 100;
__device__ __forceinline__ float page_scale(float s)
{
    return s > kMinPageScale ? (s < kMaxPageScale ? s : kMaxPageScale) : kMinPageScale;
}

constexpr int64_t kMaxHeadDim = 256;
constexpr int64_t kMaxPagedLen = (int64_t)1 << 24;      // table_width * page_size
constexpr int64_t kMaxPagedTokens = (int64_t)1 << 26;   // new tokens of a batch
constexpr int64_t kMaxPagedSeqs = (int64_t)1 << 16;
constexpr int64_t kMaxPagedHeads = 1024;
constexpr float kMaxSoftmaxScale = 0x1p127f;            // times log2(e) it is finite
constexpr int64_t kMaxPagedRows = (int64_t)1 << 30;     // tokens * (q_heads / kv_heads)

struct PagedBatch {
    const int* page_table;   // [B, W]
    const int* q_start;      // [B + 1]
    const int* kv_lens;      // [B]
    int T, B, W, max_q;
};

// The new tokens of sequence b as the kernels take them from the batch's
// arrays: n rows from `row` on, the first at position `start` (which may be
// negative: a batch slot without a sequence), `len` tokens in the cache.  Rows
// and lengths outside the batch's bounds are cut off, so that no value in the
// arrays leads to an access out of bounds.
struct PagedSeq {
    int row, n, start, len;
};
__device__ __forceinline__ int clamp_int(int v, int lo, int hi) { return v < lo ? lo : (v > hi ? hi : v); }
__device__ __forceinline__ PagedSeq paged_seq(const PagedBatch& s, int b, int page_size)
{
    const int r0 = clamp_int(s.q_start[b], 0, s.T), r1 = clamp_int(s.q_start[b + 1], r0, s.T);
    const int len = clamp_int(s.kv_lens[b], 0, s.W * page_size);
    return PagedSeq{r0, min(r1 - r0, s.max_q), len - (r1 - r0), len};
}

struct AppendArgs {
    PagedBatch batch;
    uint8_t *k_pages, *v_pages;      // [pages, Hk, P, D], [pages, Hk, D, P]
    float *k_scale, *v_scale;        // [pages, Hk]
    const uint16_t *k, *v, *q;       // [T, Hk, D], [T, Hk, D], [T, Hq, D] with row strides; q may be null
    uint16_t* q_out;
    const float* rope;               // [rows, R]
    int64_t k_stride, v_stride, q_stride, q_out_stride;
    int pages, Hk, P, D, Hq, R, interleaved;
};
hipError_t launch_kv_append(const AppendArgs& a, int dtype, hipStream_t stream);

struct AttendArgs {
    PagedBatch batch;
    const uint8_t *k_pages, *v_pages;
    const float *k_scale, *v_scale;
    const uint16_t* q;               // [T, Hq, D] with a row stride
    uint16_t* y;                     // [T, Hq, D]
    float* lse;                      // [T, Hq] or null
    float* work;
    int64_t q_stride;
    int pages, Hk, P, page_shift, D, Hq, group;
    float scale_log2;                // |softmax scale| * log2(e)
    int q_flip;                      // sign bits of two queries where the scale is negative, else 0
    int causal, window;
};
// With at most this many query rows a sequence, a workgroup can have a key/value head of it whole
// (attend_whole.hip); the tile kernel cuts the keys over workgroups where there are few, with a second
// launch.  Whole, in us, against the tile kernel, 64/8 heads x 128, u = sequences * key/value heads:
//   u = 8    1 x 500 8.5 (13.8)     1 x 1400 12.9 (14.0)   1 x 1700 15.0 (13.0)   1 x 4000 26.6 (14.1)
//   u = 64   8 x 2000 18.3 (21.0)   8 x 2600 21.6 (22.6)   8 x 4000 28.5 (25.6)
//   u = 128  16 x 4000 38 (41)      16 x 8000 67 (64), of up to 8000 57 (45)
//   u = 192  24 x 4000 44 (64)      24 of up to 16000 115 (99)
//   u = 256  32 x 4000 55 (72)      32 of up to 8000 73 (85)
//   u = 512  64 of up to 8000 131 (173), of up to 32000 490 (648)
// Alone, a workgroup's time goes by the codes that it reads, the tile kernel's by its two launches: 2 heads
// x 64, 2 x 2600 11.6 (12.6), 2 x 4000 13.6 (12.7); 4 x 192 1400 15.0 (17.4), 2600 23.0 (16.6); 4 x 256 1000
// 18.4 (19.6), 1400 21.9 (20.1) (four waves, not eight, above 128).
// So whole up to 200 Ki codes of a head's keys, 288 Ki above 128 channels, or 32 u keys, and always from two
// workgroups for each of 256 compute units on.  The host knows the page table's room only, not the lengths.
constexpr int kWholeRows = 16;
inline bool takes_tiles(const AttendArgs& a)
{
    if ((int64_t)a.batch.max_q * a.group > kWholeRows) return true;
    const int64_t u = (int64_t)a.batch.B * a.Hk, keys = (int64_t)a.batch.W * a.P;
    return u < 512 && keys * a.D > (a.D <= 128 ? 200 : 288) * 1024 && keys > 32 * u;
}
hipError_t launch_attend_tiles(const AttendArgs& a, int dtype, hipStream_t stream);
int64_t attend_tiles_work_bytes(const AttendArgs& a);
// Bytes of scratch; looks at the sizes in `a` only.
int64_t attend_work_bytes(const AttendArgs& a);
hipError_t launch_paged_attention(const AttendArgs& a, int dtype, hipStream_t stream);

}  // namespace fp8q
