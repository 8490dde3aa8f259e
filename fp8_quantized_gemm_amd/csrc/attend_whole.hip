// Attention over the paged FP8 cache for few query rows, a key/value head of a
// sequence whole in one workgroup (see paged.hpp for when).
//
//   S^T = K Q^T   MFMA 16x16x32, keys along M, the (token, head) rows along N
//   P   = 2^(S^T * ks + lv - m)   in the lanes of its row
//   Y^T = V^T P   MFMA 16x16x32, channels along M
//
// The waves (8 at most) have equal runs of the key tiles, which they load straight into
// registers, a tile of 64 keys ahead, and join their sums in LDS: no wave waits
// for another before the end, and there is one launch.  Short calls are bound
// by the chain of a launch, the lengths, the page ids, the codes and the
// arithmetic on a tile or two: 1 token of 500 with 64/8 heads takes 8.5 us, of
// 64 5.3 us.  A workgroup by itself reads about 45 GB/s, so from about 128 of
// them on HBM is the bound: 64 of 8192 185 us (5.8 TB/s; reads alone reach 6.45).
// Workgroups of neighbouring heads follow each other, so that a long sequence's
// run side by side: 24 of up to 2048 with 32/32 heads take 50 us, 11% more with
// neighbouring sequences and 7% more with the longest first.
#include "attend.hpp"

namespace fp8q {
namespace {

constexpr int kRows = kWholeRows;         // query rows of a workgroup: (token, head of the group) pairs
// Waves of a workgroup at most: eight where the registers allow.
constexpr int waves_for(int dp) { return dp <= 128 ? 8 : 4; }

// A key tile as a wave holds it: lane (r, g) has 16 channels for each 64 of the keys
// 16 (r / 4) + 4 i + r % 4, i < 4, and the 16 keys from 16 g on of the channels 16 d + r.
template <int DP>
struct KvTile {
    v4i k[4][DP / 64], v[DP / 16];
};

// What a lane needs of the i-th tile of a look-up: the pages of the keys and of the values that it
// loads, the scales of its terms.
struct TilePages {
    int k, v, k_inside, v_inside;
    PageScales sc;
    bool valid;
};
template <bool WIDE>
__device__ __forceinline__ TilePages tile_pages(const AttendArgs& a, const Pages& p, int i, int key0, int r, int g)
{
    if constexpr (WIDE) {
        const auto lane_i = [&](float v) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), i)); };
        const int page = __builtin_amdgcn_readlane(p.page, i), inside = key0 & (a.P - 1);
        return TilePages{page, page, inside, inside,
                         PageScales{lane_i(p.sc.key), lane_i(p.sc.log_value), lane_i(p.sc.inverse_value)},
                         (p.valid >> i & 1) != 0};
    } else {
        const int ik = 4 * i + (r >> 2), iv = 4 * i + g;
        return TilePages{__shfl(p.page, ik), __shfl(p.page, iv), (key0 + 16 * (r >> 2)) & (a.P - 1),
                         (key0 + 16 * g) & (a.P - 1),
                         PageScales{__shfl(p.sc.key, iv), __shfl(p.sc.log_value, iv), __shfl(p.sc.inverse_value, iv)},
                         (p.valid >> iv & 1) != 0};
    }
}

template <int DP, bool WIDE>
__device__ __forceinline__ void load_keys(const AttendArgs& a, KvTile<DP>& t, const TilePages& p, int h,
                                          int r, int g)
{
    constexpr int NC = DP / 64;
    const int64_t page_bytes = (int64_t)a.P * a.D, pool_stride = a.Hk * page_bytes;
    if constexpr (WIDE) {
        // buffer loads: one 32-bit offset a lane, the rest scalar; channels past D are sent out of
        // the buffer's range and read as 0
        const rsrc_t rk = make_rsrc(a.k_pages + p.k * pool_stride + h * page_bytes + p.k_inside * a.D,
                                    (uint32_t)(kKeys * a.D));
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const int d = 64 * c + 16 * g;
                const uint32_t at = (uint32_t)((16 * (r >> 2) + (r & 3)) * a.D + d);
                t.k[i][c] = __builtin_amdgcn_raw_buffer_load_b128(rk, d < a.D ? at : kOOB, uniform(4 * i * a.D),
                                                                  CP_DEFAULT);
            }
    } else {
        const uint8_t* kt = a.k_pages + p.k * pool_stride + h * page_bytes +
                            (int64_t)(p.k_inside + (r & 3)) * a.D;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const int d = 64 * c + 16 * g;
                t.k[i][c] = v4i{0, 0, 0, 0};
                if (d < a.D) t.k[i][c] = *reinterpret_cast<const v4i*>(kt + 4 * i * a.D + d);
            }
    }
}

template <int DP, bool WIDE>
__device__ __forceinline__ void load_values(const AttendArgs& a, KvTile<DP>& t, const TilePages& p, int h,
                                            int r, int g)
{
    constexpr int ND = DP / 16;
    const int64_t page_bytes = (int64_t)a.P * a.D, pool_stride = a.Hk * page_bytes;
    if constexpr (WIDE) {
        const rsrc_t rv = make_rsrc(a.v_pages + p.v * pool_stride + h * page_bytes + p.v_inside,
                                    (uint32_t)(page_bytes - p.v_inside));
#pragma unroll
        for (int d = 0; d < ND; ++d)
            t.v[d] = __builtin_amdgcn_raw_buffer_load_b128(rv, (uint32_t)(r * a.P + 16 * g),
                                                           uniform(16 * d * a.P), CP_DEFAULT);
    } else {
        const uint8_t* vt = a.v_pages + p.v * pool_stride + h * page_bytes + p.v_inside;
#pragma unroll
        for (int d = 0; d < ND; ++d) {
            t.v[d] = v4i{0, 0, 0, 0};
            if (16 * d < a.D) t.v[d] = *reinterpret_cast<const v4i*>(vt + (int64_t)(16 * d + r) * a.P);
        }
    }
}

// What a wave has of 16 query rows: lane (r, g) the sums of row r's channels 16 d + 4 g ..,
// the reference, its own keys' share of the denominator and the reference of that (m, or one of its own
// once a scale of values was `apart`).
template <int DP>
struct Rows {
    v4i q[DP / 64][2];
    v4f acc[DP / 16];
    float m, l, z;
    bool apart;
};

// A tile's terms; keys_read is called when its keys are no longer needed.
template <int DT, int DP, class F>
__device__ __forceinline__ void add_tile(Rows<DP>& x, KvTile<DP>& t, const PageScales& sc, const KeyRange& see,
                                         bool whole, bool valid, int key0, int g, F keys_read)
{
    constexpr int NC = DP / 64, ND = DP / 16;
    v4f s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        s[i] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            s[i] = Half<DT>::mfma(Half<DT>::widen(t.k[i][c][0], t.k[i][c][1]), x.q[c][0], s[i]);
            s[i] = Half<DT>::mfma(Half<DT>::widen(t.k[i][c][2], t.k[i][c][3]), x.q[c][1], s[i]);
        }
    }
    keys_read();
    if (!whole) mask_tile<ND>(s, x.acc, t.v, see, key0, g, valid);

    float top = s[0][0];
#pragma unroll
    for (int i = 1; i < 16; ++i) top = fmaxf(top, s[i >> 2][i & 3]);
    if (x.apart) add_apart(x.z, x.l, top * sc.key, sc.key, [&](int i) { return s[i >> 2][i & 3]; });
    top = __builtin_fmaf(top, sc.key, sc.log_value);
    top = fmaxf(top, __shfl_xor(top, 16));
    top = fmaxf(top, __shfl_xor(top, 32));
    if (__any(top > x.m + kSlack)) {
        const float m1 = fmaxf(x.m, top);
        const float alpha = m1 == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(x.m - m1);
#pragma unroll
        for (int d = 0; d < ND; ++d) x.acc[d] *= alpha;
        x.m = m1;
        x.l *= x.apart ? 1.0f : alpha;
        x.z = x.apart ? x.z : m1;
    }
    const float offset = sc.log_value - ((x.m == -__builtin_inff() ? 0.0f : x.m) - kShift);
    float sum = 0.0f;
    v8h p[2];
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
        const v2f v = {__builtin_amdgcn_exp2f(__builtin_fmaf(s[i >> 2][i & 3], sc.key, offset)),
                       __builtin_amdgcn_exp2f(__builtin_fmaf(s[i >> 2][(i & 3) + 1], sc.key, offset))};
        sum += v[0];
        sum += v[1];
        const v2h w = __builtin_convertvector(v, v2h);
        p[i >> 3][i & 7] = w[0];
        p[i >> 3][(i & 7) + 1] = w[1];
    }
    x.l = __builtin_fmaf(sum, x.apart ? 0.0f : sc.inverse_value, x.l);
#pragma unroll
    for (int d = 0; d < ND; ++d) {
        x.acc[d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(Half<DT_FP16>::widen(t.v[d][0], t.v[d][1]), p[0],
                                                          x.acc[d], 0, 0, 0);
        x.acc[d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(Half<DT_FP16>::widen(t.v[d][2], t.v[d][3]), p[1],
                                                          x.acc[d], 0, 0, 0);
    }
}

// Key/value head h of sequence b; its workgroup has the tiles from tile0 on, this wave `t0` .. of them.
struct Run {
    PagedSeq q;
    int b, h, rows, tile0, t0, t1;
};
template <int DT, int DP, bool WIDE>
__device__ __forceinline__ void attend_run(const AttendArgs& a, const Run& u, Rows<DP>& x)
{
    constexpr int NC = DP / 64, ND = DP / 16;
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4, h = u.h, b = u.b;
    // this lane's query row and the keys it sees
    const int token = r / a.group, head = h * a.group + r % a.group;
    const auto key_of = [&](int t) { return (u.tile0 + t) * kKeys; };
    Pages known = look_up<WIDE>(a, b, u.q.len, key_of(u.t0), h);
    {
        const uint16_t* src = a.q + (int64_t)(u.q.row + token) * a.q_stride + (int64_t)head * a.D;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int d = 64 * c + 16 * g;
            const bool have = r < u.rows && d < a.D;
            const v4i zero = {0, 0, 0, 0};
            x.q[c][0] = have ? *reinterpret_cast<const v4i*>(src + d) ^ a.q_flip : zero;
            x.q[c][1] = have ? *reinterpret_cast<const v4i*>(src + d + 8) ^ a.q_flip : zero;
        }
    }
    KeyRange see = key_range(a, u.q, token);
    if (r >= u.rows) see.lo = see.hi = 0;
    const KeyRange first = key_range(a, u.q, 0),
                   last = key_range(a, u.q, __builtin_amdgcn_readlane(token, u.rows - 1));
#pragma unroll
    for (int d = 0; d < ND; ++d) x.acc[d] = v4f{0.f, 0.f, 0.f, 0.f};
    x.m = x.z = -__builtin_inff();
    x.l = 0.0f;

    // the next tile's keys are asked for when this tile's have been read, its values likewise
    KvTile<DP> tile;
    TilePages pages = tile_pages<WIDE>(a, known, 0, key_of(u.t0), r, g);
    load_keys<DP, WIDE>(a, tile, pages, h, r, g);
    load_values<DP, WIDE>(a, tile, pages, h, r, g);
    x.apart = any_apart(known.sc);
    for (int t = u.t0; t < u.t1; ++t) {
        const int key0 = key_of(t), next = (t + 1 - u.t0) % kLookUp<WIDE>;
        const bool more = t + 1 < u.t1;
        const bool whole = first.lo <= key0 && last.lo <= key0 && first.hi >= key0 + kKeys &&
                           last.hi >= key0 + kKeys && __all(pages.valid);
        const PageScales sc = pages.sc;
        const bool valid = pages.valid;
        add_tile<DT, DP>(x, tile, sc, see, whole, valid, key0, g, [&] {
            if (!more) return;
            if (next == 0) known = look_up<WIDE>(a, b, u.q.len, key0 + kKeys, h);
            pages = tile_pages<WIDE>(a, known, next, key0 + kKeys, r, g);
            load_keys<DP, WIDE>(a, tile, pages, h, r, g);
            if (next == 0) x.apart |= any_apart(known.sc);
        });
        if (more) load_values<DP, WIDE>(a, tile, pages, h, r, g);
    }
    join_lanes(x.z, x.l, 16);                               // the lane groups had keys of their own
    join_lanes(x.z, x.l, 32);
}

// A workgroup has all rows of a key/value head of a sequence, its waves equal runs of the key tiles;
// the waves' sums are joined in LDS.
template <int DT, int DP, bool WIDE, int WAVES>
__global__ void __launch_bounds__(WAVES * 64, DP <= 128 ? 2 : 1) attend_whole_kernel(const AttendArgs a)
{
    constexpr int kWaves = WAVES, kThreads = kWaves * 64, ND = DP / 16;
    constexpr int RS = DP + 4;                              // floats of a row in LDS
    __shared__ __attribute__((aligned(16))) float stat[kWaves][kRows][4];      // m, l, z
    __shared__ __attribute__((aligned(16))) float sums[kWaves][kRows * RS];

    const int lane = threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6), r = lane & 15, g = lane >> 4;
    const uint32_t index = blockIdx.y * gridDim.x + blockIdx.x;         // at most 2^26, and a row of the grid
    if (index >= (uint32_t)(a.batch.B * a.Hk)) return;
    Run u;
    u.b = (int)(index / (uint32_t)a.Hk);
    u.h = (int)(index % (uint32_t)a.Hk);
    u.q = paged_seq(a.batch, u.b, a.P);
    u.rows = u.q.n * a.group;
    if (u.rows == 0) return;
    const int lo = key_range(a, u.q, 0).lo, hi = key_range(a, u.q, u.q.n - 1).hi;
    u.tile0 = lo / kKeys;
    const int tiles = max((hi + kKeys - 1) / kKeys - u.tile0, 1), each = (tiles + kWaves - 1) / kWaves;
    const int used = (tiles + each - 1) / each;             // waves that have tiles
    u.t0 = wave * each;
    u.t1 = min(u.t0 + each, tiles);
    if (wave < used) {
        Rows<DP> x;
        attend_run<DT, DP, WIDE>(a, u, x);
        if (g == 0) *reinterpret_cast<v4f*>(stat[wave][r]) = v4f{x.m, x.l, x.z, 0.0f};
#pragma unroll
        for (int d = 0; d < ND; ++d) *reinterpret_cast<v4f*>(&sums[wave][r * RS + 16 * d + 4 * g]) = x.acc[d];
    }
    __syncthreads();

    const int quads = a.D / 4;
    for (int i = threadIdx.x; i < u.rows * quads; i += kThreads) {
        const int row = i / quads, d = i % quads * 4;
        Joined j{-__builtin_inff(), -__builtin_inff(), 0.0f};
        for (int p = 0; p < used; ++p) {
            const v4f s = *reinterpret_cast<const v4f*>(stat[p][row]);
            j.ref = fmaxf(j.ref, s[0]);
            j.z = fmaxf(j.z, s[2]);
        }
        if (j.ref == -__builtin_inff()) j.ref = 0.0f;
        if (j.z == -__builtin_inff()) j.z = 0.0f;
        v4f o = {0.f, 0.f, 0.f, 0.f};
        for (int p = 0; p < used; ++p) {
            const v4f s = *reinterpret_cast<const v4f*>(stat[p][row]);
            const float f = __builtin_amdgcn_exp2f(s[0] - j.ref);
            j.l += s[1] * __builtin_amdgcn_exp2f(s[2] - j.z);
            o += *reinterpret_cast<const v4f*>(&sums[p][row * RS + d]) * f;
        }
        store_row<DT>(a, u.q.row + row / a.group, u.h * a.group + row % a.group, d, o, j);
    }
}

template <int DT, int DP, bool WIDE, int WAVES>
hipError_t launch_waves(const AttendArgs& a, hipStream_t stream)
{
    constexpr int kThreads = WAVES * 64;
    const int64_t groups = (int64_t)a.batch.B * a.Hk, most = max_groups(kThreads), gx = groups < most ? groups : most;
    hipLaunchKernelGGL((attend_whole_kernel<DT, DP, WIDE, WAVES>),
                       dim3((unsigned)gx, (unsigned)((groups + gx - 1) / gx)), dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}
// Fewer waves where there may be few key tiles: their registers and LDS keep other workgroups away (54
// sequences of up to 200 tokens, 32/32 heads x 128: 24 us with 4 waves, 36 with 8; of up to 4 tokens x 96:
// 10 with 1, 32 with 8).  With few workgroups more waves store the rows sooner (1 of 60, 64/8 heads: 5.8 us
// with 8, 6.8 with 1).
template <int DT, int DP, bool WIDE>
hipError_t launch(const AttendArgs& a, hipStream_t stream)
{
    const int64_t keys = (int64_t)a.batch.W * a.P, groups = (int64_t)a.batch.B * a.Hk;
    if (keys <= kKeys && groups >= 512) return launch_waves<DT, DP, WIDE, 1>(a, stream);
    if (DP <= 128 && keys <= 4 * kKeys) return launch_waves<DT, DP, WIDE, 4>(a, stream);
    return launch_waves<DT, DP, WIDE, waves_for(DP)>(a, stream);
}

template <int DT, int DP>
hipError_t launch(const AttendArgs& a, hipStream_t stream)
{
    return a.P % kKeys == 0 ? launch<DT, DP, true>(a, stream) : launch<DT, DP, false>(a, stream);
}

template <int DT>
hipError_t launch(const AttendArgs& a, hipStream_t stream)
{
    if (a.D <= 64) return launch<DT, 64>(a, stream);
    if (a.D <= 128) return launch<DT, 128>(a, stream);
    if (a.D <= 192) return launch<DT, 192>(a, stream);
    return launch<DT, 256>(a, stream);
}

}  // namespace

hipError_t launch_paged_attention(const AttendArgs& a, int dtype, hipStream_t stream)
{
    if (takes_tiles(a)) return launch_attend_tiles(a, dtype, stream);
    return dtype == DT_BF16 ? launch<DT_BF16>(a, stream) : launch<DT_FP16>(a, stream);
}

int64_t attend_work_bytes(const AttendArgs& a) { return takes_tiles(a) ? attend_tiles_work_bytes(a) : 16; }

}  // namespace fp8q
