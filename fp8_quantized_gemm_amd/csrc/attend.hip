// Attention over the paged FP8 cache for few query rows (see paged.hpp).
#include "attend.hpp"

namespace fp8q {
namespace {

constexpr int kWaves = 4, kThreads = kWaves * 64;
constexpr int kRows = 16;                 // query rows of a unit: (token, head of the group) pairs
constexpr int kMinTiles = 4;              // key tiles that a workgroup takes at least

// The work is a list of units (sequence, key/value head, row tile), each a run
// of 64-token key tiles; workgroup w takes tiles [w * share, (w + 1) * share)
// of the whole list.
struct Share {
    int64_t begin, end;
};

struct SeqWork {
    PagedSeq q;
    int tile0, tiles;                     // key tiles that some row of the sequence sees
    int row_tiles;
    int units;                            // key/value heads x row tiles
};

__device__ __forceinline__ SeqWork seq_work(const AttendArgs& a, int b)
{
    SeqWork w;
    w.q = paged_seq(a.batch, b, a.P);
    const KeyRange first = key_range(a, w.q, 0), last = key_range(a, w.q, w.q.n - 1);
    w.tile0 = first.lo >> 6;
    w.tiles = max(((last.hi + 63) >> 6) - w.tile0, 1);
    w.row_tiles = (w.q.n * a.group + kRows - 1) / kRows;
    w.units = w.row_tiles * a.Hk;
    return w;
}

struct ScanLds {
    int64_t wave[kWaves];
    int64_t before;
    int b;
};

// Tiles of all sequences (the return value) and, for the tile `at`, the sequence that
// holds it and the tiles before that sequence.  Every thread sums a run of sequences.
template <class F>
__device__ __forceinline__ int64_t scan_sequences(const AttendArgs& a, ScanLds& lds, F pick)
{
    const int B = a.batch.B, per = (B + kThreads - 1) / kThreads, lane = threadIdx.x & 63;
    const int b0 = min((int)threadIdx.x * per, B), b1 = min(b0 + per, B);
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) {
        const SeqWork w = seq_work(a, b);
        mine += (int64_t)w.units * w.tiles;
    }
    int64_t sum = mine;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int64_t up = __shfl_up(sum, off);
        if (lane >= off) sum += up;
    }
    if (lane == 63) lds.wave[threadIdx.x >> 6] = sum;
    if (threadIdx.x == 0) lds.b = B;
    __syncthreads();
    int64_t total = 0, before = sum - mine;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        if (w < (int)(threadIdx.x >> 6)) before += lds.wave[w];
        total += lds.wave[w];
    }
    const int64_t at = pick(total);
    if (at >= before && at < before + mine) {
        for (int b = b0; b < b1; ++b) {
            const SeqWork w = seq_work(a, b);
            const int64_t n = (int64_t)w.units * w.tiles;
            if (at < before + n) {
                lds.b = b;
                lds.before = before;
                break;
            }
            before += n;
        }
    }
    __syncthreads();
    return total;
}

__device__ __forceinline__ int64_t share_of(int64_t total, int groups)
{
    const int64_t s = (total + groups - 1) / groups;
    return s > kMinTiles ? s : kMinTiles;
}

// The scratch of G workgroups: for each the unit that it begins and another one
// ends (parts = 0: none), then two partial results for each, of a unit that it
// goes on with and of one that it begins: kRows rows of maximum, denominator and,
// from the fifth float on, DP sums.
struct Unit {
    int parts, token0, head, row0, rows, unused[3];
};
template <int DP>
__device__ __forceinline__ float* part_of(float* work, int groups, int64_t group, bool begins)
{
    return work + groups * (int)(sizeof(Unit) / 4) + (group * 2 + (begins ? 1 : 0)) * (kRows * (DP + 4));
}

template <int DT, int DP>
__global__ void __launch_bounds__(kThreads, DP <= 192 ? 2 : 1) attend_rows_kernel(const AttendArgs a)
{
    constexpr int NC = DP / 64, ND = DP / 16;
    constexpr int RS = DP + 4;                              // floats of a row in LDS
    __shared__ ScanLds scan;
    __shared__ float stat[kWaves][kRows][2];
    __shared__ __attribute__((aligned(16))) float part[kWaves * kRows * RS];

    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
    const int W = gridDim.x;
    const int64_t total = scan_sequences(
        a, scan, [&](int64_t t) { return (int64_t)blockIdx.x * share_of(t, W); });
    const int64_t share = share_of(total, W);
    int64_t at = blockIdx.x * share;
    const int64_t end = at + share < total ? at + share : total;
    bool told = false;                    // in thread 0: a unit is left for the joining kernel
    int b = scan.b;
    int64_t seq_at = scan.before;
    const int64_t page_bytes = (int64_t)a.P * a.D, pool_stride = a.Hk * page_bytes;

    while (at < end) {
        const SeqWork w = seq_work(a, b);
        const int64_t seq_tiles = (int64_t)w.units * w.tiles;
        if (at >= seq_at + seq_tiles) { seq_at += seq_tiles; ++b; continue; }
        const int unit = (int)((at - seq_at) / w.tiles);
        const int64_t unit_at = seq_at + (int64_t)unit * w.tiles;
        const int t0 = (int)(at - unit_at);
        const int t1 = (int)(end - unit_at < w.tiles ? end - unit_at : w.tiles);
        const int h = unit / w.row_tiles, row0 = unit % w.row_tiles * kRows;
        const int rows = min(kRows, w.q.n * a.group - row0);

        // this lane's query row and the keys it sees
        const int my_row = row0 + r, token = my_row / a.group, head = h * a.group + my_row % a.group;
        KeyRange see = key_range(a, w.q, token);
        if (r >= rows) see.lo = see.hi = 0;
        const KeyRange first = key_range(a, w.q, row0 / a.group),
                       last = key_range(a, w.q, (row0 + rows - 1) / a.group);
        v4i qf[NC][2];
        {
            const uint16_t* src = a.q + (int64_t)(w.q.row + token) * a.q_stride + (int64_t)head * a.D;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const int d = 64 * c + 16 * g;
                const bool have = r < rows && d < a.D;
                const v4i zero = {0, 0, 0, 0};
                qf[c][0] = have ? *reinterpret_cast<const v4i*>(src + d) ^ a.q_flip : zero;
                qf[c][1] = have ? *reinterpret_cast<const v4i*>(src + d + 8) ^ a.q_flip : zero;
            }
        }
        v4f acc[ND];
#pragma unroll
        for (int d = 0; d < ND; ++d) acc[d] = v4f{0.f, 0.f, 0.f, 0.f};
        float m = -__builtin_inff(), l = 0.0f;

        for (int t = t0 + wave; t < t1; t += kWaves) {
            const int key0 = (w.tile0 + t) << 6;
            // key rows of the first product are read by row group, values by lane group
            const PageRef kp = page_ref(a, b, w.q.len, key0 + 16 * (r >> 2));
            const PageRef vp = page_ref(a, b, w.q.len, key0 + 16 * g);
            const uint8_t* kt = a.k_pages + kp.page * pool_stride + h * page_bytes +
                                (int64_t)(kp.inside + (r & 3)) * a.D;
            const uint8_t* vt = a.v_pages + vp.page * pool_stride + h * page_bytes + vp.inside;
            v4i kf[4][NC], vf[ND];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    const int d = 64 * c + 16 * g;
                    kf[i][c] = v4i{0, 0, 0, 0};
                    if (d < a.D)
                        kf[i][c] = *reinterpret_cast<const v4i*>(kt + 4 * i * a.D + d);
                }
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                vf[d] = v4i{0, 0, 0, 0};
                if (16 * d < a.D) vf[d] = *reinterpret_cast<const v4i*>(vt + (int64_t)(16 * d + r) * a.P);
            }
            const PageScales sc = page_scales(a, vp.page, h);

            v4f s[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[i] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    s[i] = Half<DT>::mfma(Half<DT>::widen(kf[i][c][0], kf[i][c][1]), qf[c][0], s[i]);
                    s[i] = Half<DT>::mfma(Half<DT>::widen(kf[i][c][2], kf[i][c][3]), qf[c][1], s[i]);
                }
            }
            const bool whole = first.lo <= key0 && last.lo <= key0 && first.hi >= key0 + 64 &&
                               last.hi >= key0 + 64 && __all(vp.valid);
            if (!whole) mask_tile<ND>(s, acc, vf, see, key0, g, vp.valid);

            float top = s[0][0];
#pragma unroll
            for (int i = 1; i < 16; ++i) top = fmaxf(top, s[i >> 2][i & 3]);
            top = __builtin_fmaf(top, sc.key, sc.log_value);
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            if (__any(top > m + kSlack)) {
                const float m1 = fmaxf(m, top);
                const float alpha = m1 == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(m - m1);
                l *= alpha;
#pragma unroll
                for (int d = 0; d < ND; ++d) acc[d] *= alpha;
                m = m1;
            }
            const float offset = sc.log_value - ((m == -__builtin_inff() ? 0.0f : m) - kShift);
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
            l = __builtin_fmaf(sum, sc.inverse_value, l);
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                acc[d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                    Half<DT_FP16>::widen(vf[d][0], vf[d][1]), p[0], acc[d], 0, 0, 0);
                acc[d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                    Half<DT_FP16>::widen(vf[d][2], vf[d][3]), p[1], acc[d], 0, 0, 0);
            }
        }

        // the waves' results together; l is spread over the lane groups
        l += __shfl_xor(l, 16);
        l += __shfl_xor(l, 32);
        if (g == 0) { stat[wave][r][0] = m; stat[wave][r][1] = l; }
        float* mine = part + (wave * kRows + r) * RS + 4 * g;
#pragma unroll
        for (int d = 0; d < ND; ++d) *reinterpret_cast<v4f*>(mine + 16 * d) = acc[d];
        __syncthreads();
        const bool all = t0 == 0 && t1 == w.tiles;
        if (t0 == 0 && t1 < w.tiles && threadIdx.x == 0) {
            const int64_t last_group = (unit_at + w.tiles - 1) / share;
            told = true;
            reinterpret_cast<Unit*>(a.work)[blockIdx.x] =
                Unit{(int)(last_group - blockIdx.x) + 1, w.q.row, h, row0, rows, {0, 0, 0}};
        }
        float* out = part_of<DP>(a.work, W, blockIdx.x, t0 == 0);
        const int quads = a.D / 4;
        for (int i = threadIdx.x; i < rows * quads; i += kThreads) {
            const int row = i / quads, d = i % quads * 4;
            const Joined j = join(stat, row, kWaves);
            v4f o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < kWaves; ++k)
                o += *reinterpret_cast<const v4f*>(part + (k * kRows + row) * RS + d) *
                     __builtin_amdgcn_exp2f(stat[k][row][0] - j.ref);
            if (all) {
                const int gr = row0 + row, at_head = h * a.group + gr % a.group;
                store_row<DT>(a, w.q.row + gr / a.group, at_head, d, o, j);
            } else {
                *reinterpret_cast<v4f*>(out + row * (DP + 4) + 4 + d) = o;
                if (d == 0) { out[row * (DP + 4)] = j.m; out[row * (DP + 4) + 1] = j.l; }
            }
        }
        __syncthreads();
        at = unit_at + t1;
    }
    if (threadIdx.x == 0 && !told) reinterpret_cast<Unit*>(a.work)[blockIdx.x].parts = 0;
}

// Joins the partial results of a unit that several workgroups had, told by the
// first of them: a workgroup for each row, its waves taking turns at the parts.
template <int DT, int DP>
__global__ void __launch_bounds__(kThreads) attend_join_kernel(const AttendArgs a)
{
    __shared__ float stat[kWaves][1][2];
    __shared__ __attribute__((aligned(16))) float part[kWaves][DP];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, row = blockIdx.y;
    const Unit u = reinterpret_cast<const Unit*>(a.work)[blockIdx.x];
    if (u.parts == 0 || row >= u.rows) return;
    float m = -__builtin_inff(), l = 0.0f;
    v4f o = {0.f, 0.f, 0.f, 0.f};
    const int d = 4 * lane;
    for (int k = wave; k < u.parts; k += kWaves) {
        const float* p = part_of<DP>(a.work, gridDim.x, blockIdx.x + k, k == 0) + row * (DP + 4);
        const float pm = p[0], pl = p[1], m1 = fmaxf(m, pm), ref = m1 == -__builtin_inff() ? 0.0f : m1;
        const float f0 = __builtin_amdgcn_exp2f(m - ref), f1 = __builtin_amdgcn_exp2f(pm - ref);
        l = l * f0 + pl * f1;
        if (d < a.D) o = o * f0 + *reinterpret_cast<const v4f*>(p + 4 + d) * f1;
        m = m1;
    }
    if (lane == 0) { stat[wave][0][0] = m; stat[wave][0][1] = l; }
    if (d < a.D) *reinterpret_cast<v4f*>(&part[wave][d]) = o;
    __syncthreads();
    if (wave != 0 || d >= a.D) return;
    const Joined j = join(stat, 0, kWaves);
    o = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < kWaves; ++k)
        o += *reinterpret_cast<const v4f*>(&part[k][d]) * __builtin_amdgcn_exp2f(stat[k][0][0] - j.ref);
    const int gr = u.row0 + row;
    store_row<DT>(a, u.token0 + gr / a.group, u.head * a.group + gr % a.group, d, o, j);
}

constexpr int kGroups = 512;              // two workgroups on each of 256 CUs

template <int DT, int DP>
hipError_t launch(const AttendArgs& a, hipStream_t stream)
{
    hipLaunchKernelGGL((attend_rows_kernel<DT, DP>), dim3(kGroups), dim3(kThreads), 0, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int rows = a.batch.max_q < kRows / a.group ? a.batch.max_q * a.group : kRows;
    hipLaunchKernelGGL((attend_join_kernel<DT, DP>), dim3(kGroups, rows), dim3(kThreads), 0, stream, a);
    return hipGetLastError();
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

int64_t attend_work_bytes(int64_t, int64_t, int64_t D, int64_t)
{
    return (int64_t)kGroups * ((int64_t)sizeof(Unit) + 2 * kRows * ((D + 63) / 64 * 64 + 4) * 4);
}

hipError_t launch_paged_attention(const AttendArgs& a, int dtype, hipStream_t stream)
{
    if ((int64_t)a.batch.max_q * a.group > 32) return launch_attend_prompt(a, dtype, stream);
    return dtype == DT_BF16 ? launch<DT_BF16>(a, stream) : launch<DT_FP16>(a, stream);
}

}  // namespace fp8q
