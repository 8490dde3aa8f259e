// A mixture-of-experts layer for a few tokens on block-scaled FP8 weights, in
// two kernels.
//
//   ids[t, j], weights[t, j]: the top_k experts of token t by logit and their
//     softmax weights;
//   h[t, j, i]  = silu(g) * u,  g = Wg[e] x[t],  u = Wu[e] x[t],  e = ids[t, j];
//   y[t, n]     = sum_j weights[t, j] * (W2[e] h[t, j])[n].
//
// With at most 64 tokens the weights of the chosen experts are nearly all the
// bytes, read once each, and bound the time.  The activations therefore stay
// in their 16-bit type (E4M3 weights convert to bf16 and fp16 exactly) and
// need no quantization pass between the two products.
//
// The first kernel (moe_up) repeats the selection in every workgroup: T * E
// logits are a few KiB, and a launch of its own would cost more.  It then
// deals (expert, 16 columns of h) items out to the workgroups.  The second
// (moe_down) gives each workgroup eight columns of y and all chosen experts,
// so the weighted sum over experts needs no atomics and no third kernel.
//
// Both use the loads and the operand layout of gemv_block_kernel: a wave
// reads the 128-byte lines of eight weight rows, each row's two 64-byte
// halves become two operand rows of the MFMA, the tokens (up to eight) are
// laid out the same way, and the two diagonal 8 x 8 quadrants of the result
// add up to the block's product.
#include <math.h>

#include <algorithm>

#include "block.hpp"
#include "tile.hpp"

namespace fp8q {
namespace {

typedef __bf16 v2b __attribute__((ext_vector_type(2)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));

constexpr int kMaxPairs = kMoeMaxTokens * kMoeMaxTopK;
constexpr int kMoeWaves = 16;
constexpr int kMoeThreads = kMoeWaves * 64;
static_assert(kMoeMaxExperts <= kMoeThreads, "one thread per expert");

// The chosen (token, expert) pairs grouped by expert.  Slot s, the s-th
// expert in ascending order that any token chose, has the pairs
// pairs[start[s]] .. pairs[start[s + 1] - 1], each t * top_k + j, ascending.
struct Routing {
    int count;                                  // slots
    int expert[kMoeMaxExperts];
    int start[kMoeMaxExperts + 1];
    int pairs[kMaxPairs];
};
static_assert(sizeof(Routing) <= kMoeRoutingBytes, "head of the workspace");

// 16 E4M3 codes -> 16 values of the activation's type (exact), in two operands.
template <int DT>
struct Half;
template <>
struct Half<DT_BF16> {
    typedef v8b vec;
    static __device__ __forceinline__ vec widen(int lo, int hi)
    {
        const v2b a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
        const v2b b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
        const v2b c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
        const v2b d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
        return vec{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
    }
    static __device__ __forceinline__ v4f mfma(vec w, v4i x, v4f c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, __builtin_bit_cast(vec, x), c, 0, 0, 0);
    }
};
template <>
struct Half<DT_FP16> {
    typedef v8h vec;
    static __device__ __forceinline__ vec widen(int lo, int hi)
    {
        const v2h a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false);
        const v2h b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true);
        const v2h c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false);
        const v2h d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true);
        return vec{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
    }
    static __device__ __forceinline__ v4f mfma(vec w, v4i x, v4f c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(w, __builtin_bit_cast(vec, x), c, 0, 0, 0);
    }
};

// One block (128 values of K) of eight weight rows times up to eight tokens.
template <int DT>
__device__ __forceinline__ v4f block_product(const v4i& w, const v4i& x0, const v4i& x1)
{
    const v4f p = Half<DT>::mfma(Half<DT>::widen(w[0], w[1]), x0, v4f{0.f, 0.f, 0.f, 0.f});
    return Half<DT>::mfma(Half<DT>::widen(w[2], w[3]), x1, p);
}

// ---------------------------------------------------------------- selection
// One wave, one token: the top_k largest logits, ties to the lower index.
// -inf switches an expert off; a NaN logit counts as -inf.  Lane j returns
// the j-th choice (-1 where fewer than top_k experts are left) and weight.
template <int PER>
__device__ __forceinline__ void route_token(const float* __restrict__ logits, int experts, int top_k,
                                            int renormalize, int lane, int& id, float& weight)
{
    float v[PER];
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = i * 64 + lane;
        v[i] = e < experts ? logits[e] : -INFINITY;
        if (!(v[i] == v[i])) v[i] = -INFINITY;
        m = fmaxf(m, v[i]);
    }
    m = wave_max(m);
    // exp(l - m) with inf - inf = 0
    auto p = [&](float l) { return l == m ? 1.0f : expf(l - m); };
    float total = 0.0f;
    if (!renormalize) {
#pragma unroll
        for (int i = 0; i < PER; ++i) total += v[i] > -INFINITY ? p(v[i]) : 0.0f;
        total = wave_sum(total);
    }
    id = -1;
    weight = 0.0f;
    float chosen = 0.0f;
    for (int j = 0; j < top_k; ++j) {
        float best = v[0];
#pragma unroll
        for (int i = 1; i < PER; ++i) best = fmaxf(best, v[i]);
        best = wave_max(best);
        if (!(best > -INFINITY)) break;
        int e = -1;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (e >= 0) continue;
            const uint64_t at = __ballot(v[i] == best);
            if (at == 0) continue;
            const int l = __ffsll((unsigned long long)at) - 1;
            e = i * 64 + l;
            if (lane == l) v[i] = -INFINITY;
        }
        const float w = p(best);
        chosen += w;
        if (lane == j) {
            id = e;
            weight = w;
        }
    }
    if (id >= 0) weight /= renormalize ? chosen : total;
}

// Groups the pairs by expert; run by the whole workgroup, ids[pairs] in LDS
// and complete.  tmp holds one int per wave.
__device__ __forceinline__ void group_pairs(const int* ids, int npairs, int experts, Routing& rt, int* tmp)
{
    const int e = threadIdx.x;
    const int lane = e & 63, wave = e >> 6;
    int mine = 0;
    if (e < experts)
        for (int p = 0; p < npairs; ++p) mine += ids[p] == e;
    // inclusive scans over experts of (chosen, pairs), packed 16 + 16 bits
    int scan = (mine > 0 ? 1 << 16 : 0) + mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(scan, d);
        if (lane >= d) scan += o;
    }
    if (lane == 63) tmp[wave] = scan;
    __syncthreads();
    for (int w = 0; w < wave; ++w) scan += tmp[w];
    if (mine > 0) {
        const int slot = (scan >> 16) - 1;
        const int end = scan & 0xffff;
        rt.expert[slot] = e;
        rt.start[slot + 1] = end;
        int at = end - mine;
        for (int p = 0; p < npairs; ++p)
            if (ids[p] == e) rt.pairs[at++] = p;
    }
    if (e == kMoeThreads - 1) {
        rt.count = scan >> 16;
        rt.start[0] = 0;
    }
    __syncthreads();
}

// ---------------------------------------------------------------- gate and up projections
constexpr int kUpCols = 16;                 // columns of h per item
constexpr int kUpTokens = 16;               // tokens per pass over an item's weights

template <int DT, int PER>
__global__ __launch_bounds__(kMoeThreads) void moe_up_kernel(
    const uint16_t* __restrict__ x, const float* __restrict__ logits,
    const uint8_t* __restrict__ w13, const float* __restrict__ s13, int* __restrict__ ids_out,
    float* __restrict__ weights_out, Routing* __restrict__ routing, uint16_t* __restrict__ h,
    int T, int H, int I, int E, int top_k, int renormalize)
{
    __shared__ Routing rt;
    __shared__ int ids[kMaxPairs];
    __shared__ int tmp[kMoeWaves];
    __shared__ float red[kMoeWaves][8][64];  // (m-tile, gate / up, row tile) x (token, row)
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, g = lane >> 4, half = r >> 3;
    const int koff = (half * 4 + g) * 16;

    for (int t = wave; t < T; t += kMoeWaves) {
        int id;
        float weight;
        route_token<PER>(logits + (size_t)t * E, E, top_k, renormalize, lane, id, weight);
        if (lane < top_k) {
            ids[t * top_k + lane] = id;
            if (blockIdx.x == 0) {
                ids_out[t * top_k + lane] = id;
                weights_out[t * top_k + lane] = weight;
            }
        }
    }
    __syncthreads();
    group_pairs(ids, T * top_k, E, rt, tmp);
    if (blockIdx.x == 0) {
        for (int i = tid; i < (int)(sizeof(Routing) / 4); i += kMoeThreads)
            reinterpret_cast<int*>(routing)[i] = reinterpret_cast<const int*>(&rt)[i];
    }

    const int nblk = (H + kBlock - 1) / kBlock;
    const int tiles = I / kUpCols;
    const int items = rt.count * tiles;
    const rsrc_t rx = make_rsrc(x, (uint32_t)(T * H * 2));
    for (int it = blockIdx.x; it < items; it += gridDim.x) {
        const int slot = it / tiles;
        const int i0 = (it - slot * tiles) * kUpCols;
        const int e = rt.expert[slot], first = rt.start[slot], last = rt.start[slot + 1];
        const size_t row = (size_t)e * 2 * I + i0;                   // gate row; up: + I
        const rsrc_t rg = make_rsrc(w13 + row * H, (uint32_t)(kUpCols * H));
        const rsrc_t ru = make_rsrc(w13 + (row + I) * H, (uint32_t)(kUpCols * H));
        const int nb = (I + kBlock - 1) / kBlock;
        const float* const sg = s13 + ((size_t)e * 2 * nb + (i0 >> 7)) * nblk;
        const float* const su = sg + (size_t)nb * nblk;
        for (int p0 = first; p0 < last; p0 += kUpTokens) {
            uint32_t xo[2];                                          // of this lane's token
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const int p = p0 + m * 8 + (r & 7);
                xo[m] = p < last ? (uint32_t)(rt.pairs[p] / top_k * H + koff) * 2 : kOOB;
            }
            const bool two = last - p0 > 8;
            v4f acc[2][2][2];
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int t = 0; t < 2; ++t) acc[m][c][t] = v4f{0.f, 0.f, 0.f, 0.f};
            for (int kb = wave; kb < nblk; kb += kMoeWaves) {
                const bool in = kb * kBlock + koff < H;
                const uint32_t off = in ? (uint32_t)((r & 7) * H + kb * kBlock + koff) : kOOB;
                v4i w[2][2], xv[2][2];
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    w[0][t] = buf_load16<CP_NT>(rg, off + t * 8 * H);
                    w[1][t] = buf_load16<CP_NT>(ru, off + t * 8 * H);
                }
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const uint32_t o = in && xo[m] != kOOB ? xo[m] + kb * kBlock * 2 : kOOB;
                    xv[m][0] = buf_load16(rx, o);
                    xv[m][1] = buf_load16(rx, o + 16);
                }
                const float s[2] = {sg[kb], su[kb]};
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    if (m == 1 && !two) break;
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            const v4f p = block_product<DT>(w[c][t], xv[m][0], xv[m][1]);
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                acc[m][c][t][q] = __builtin_fmaf(p[q], s[c], acc[m][c][t][q]);
                        }
                }
            }
            __syncthreads();                                         // red is free
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            // the other half of the block sits 8 columns and 32 lanes away
                            const float v = acc[m][c][t][q] + __shfl_xor(acc[m][c][t][q], 40);
                            if (r < 8 && g < 2) red[wave][m * 4 + c * 2 + t][r * 8 + 4 * g + q] = v;
                        }
            __syncthreads();
            if (tid < kUpTokens * kUpCols) {
                const int col = tid & 15, tok = tid >> 4;
                const int p = p0 + tok;
                if (p < last) {
                    float gv = 0.0f, uv = 0.0f;
                    const int k = (tok & 7) * 8 + (col & 7), b = (tok >> 3) * 4 + (col >> 3);
#pragma unroll
                    for (int w = 0; w < kMoeWaves; ++w) {
                        gv += red[w][b][k];
                        uv += red[w][b + 2][k];
                    }
                    // bf16 has fp32's range (fp16 would overflow); its rounding, 2^-8, is that of y
                    h[(size_t)rt.pairs[p] * I + i0 + col] =
                        (uint16_t)f32_to_bf16_bits(gv / (1.0f + expf(-gv)) * uv);
                }
            }
        }
    }
}

// ---------------------------------------------------------------- down projection
constexpr int kDownRows = 8;                // columns of y (rows of W2) per workgroup
constexpr int kDownBlocks = 4;              // K blocks per item

__global__ __launch_bounds__(kMoeThreads) void moe_down_kernel(
    const uint16_t* __restrict__ h, const uint8_t* __restrict__ w2, const float* __restrict__ s2,
    const Routing* __restrict__ routing, const float* __restrict__ weights,
    uint16_t* __restrict__ y, int T, int H, int I, int top_k)
{
    __shared__ Routing rt;
    __shared__ float wt[kMaxPairs];
    extern __shared__ __attribute__((aligned(16))) float ysum[];   // [waves][T][rows]
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, g = lane >> 4, half = r >> 3;
    const int koff = (half * 4 + g) * 16;
    const int n0 = blockIdx.x * kDownRows;

    for (int i = tid; i < (int)(sizeof(Routing) / 4); i += kMoeThreads)
        reinterpret_cast<int*>(&rt)[i] = reinterpret_cast<const int*>(routing)[i];
    for (int i = tid; i < T * top_k; i += kMoeThreads) wt[i] = weights[i];
    for (int i = tid; i < kMoeWaves * T * kDownRows; i += kMoeThreads) ysum[i] = 0.0f;
    __syncthreads();

    const int nblk = (I + kBlock - 1) / kBlock;
    const int chunks = (nblk + kDownBlocks - 1) / kDownBlocks;
    const int items = rt.count * chunks;
    const rsrc_t rh = make_rsrc(h, (uint32_t)(T * top_k * I * 2));
    float* const mine = ysum + wave * T * kDownRows;
    for (int it = wave; it < items; it += kMoeWaves) {
        const int slot = it / chunks;
        const int kb0 = (it - slot * chunks) * kDownBlocks;
        const int e = rt.expert[slot], first = rt.start[slot], last = rt.start[slot + 1];
        const rsrc_t rw = make_rsrc(w2 + ((size_t)e * H + n0) * I, (uint32_t)(kDownRows * I));
        const float* const sb = s2 + ((size_t)e * ((H + kBlock - 1) / kBlock) + (n0 >> 7)) * nblk;
        v4i w[kDownBlocks];
        float s[kDownBlocks];
#pragma unroll
        for (int c = 0; c < kDownBlocks; ++c) {
            const int kb = kb0 + c;
            w[c] = buf_load16<CP_NT>(rw, kb * kBlock + koff < I
                                             ? (uint32_t)((r & 7) * I + kb * kBlock + koff) : kOOB);
            s[c] = kb < nblk ? sb[kb] : 0.0f;
        }
        for (int p0 = first; p0 < last; p0 += 8) {
            const int p = p0 + (r & 7);
            const int pair = p < last ? rt.pairs[p] : -1;
            v4f acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < kDownBlocks; ++c) {
                const int k = (kb0 + c) * kBlock + koff;
                const uint32_t o = pair >= 0 && k < I ? (uint32_t)(pair * I + k) * 2 : kOOB;
                const v4f q = block_product<DT_BF16>(w[c], buf_load16(rh, o), buf_load16(rh, o + 16));
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(q[i], s[c], acc[i]);
            }
            v4f v;
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = acc[i] + __shfl_xor(acc[i], 40);
            // a token occurs once among an expert's pairs, so no two lanes meet
            if (r < 8 && g < 2 && pair >= 0) {
                v4f* const dst = reinterpret_cast<v4f*>(mine + pair / top_k * kDownRows + 4 * g);
                const float f = wt[pair];
                v4f d = *dst;
#pragma unroll
                for (int i = 0; i < 4; ++i) d[i] = __builtin_fmaf(v[i], f, d[i]);
                *dst = d;
            }
        }
    }
    __syncthreads();
    for (int o = tid; o < T * kDownRows; o += kMoeThreads) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kMoeWaves; ++w) v += ysum[w * T * kDownRows + o];
        y[(size_t)(o / kDownRows) * H + n0 + o % kDownRows] = (uint16_t)f32_to_bf16_bits(v);
    }
}

template <int DT, int PER>
hipError_t launch_up(const MoeArgs& a, hipStream_t stream)
{
    const int64_t slots = std::min<int64_t>(a.E, (int64_t)a.T * a.top_k);
    const int64_t items = slots * (a.I / kUpCols);
    const int grid = (int)std::min<int64_t>(items, 2 * kCUs);
    moe_up_kernel<DT, PER><<<grid, kMoeThreads, 0, stream>>>(
        static_cast<const uint16_t*>(a.x), a.logits, a.w13, a.s13, a.ids, a.weights,
        static_cast<Routing*>(a.work),
        reinterpret_cast<uint16_t*>(static_cast<char*>(a.work) + kMoeRoutingBytes), a.T, a.H, a.I,
        a.E, a.top_k, a.renormalize);
    return hipGetLastError();
}

template <int DT>
hipError_t launch_up_dt(const MoeArgs& a, hipStream_t stream)
{
    if (a.E <= 64) return launch_up<DT, 1>(a, stream);
    if (a.E <= 128) return launch_up<DT, 2>(a, stream);
    if (a.E <= 256) return launch_up<DT, 4>(a, stream);
    return launch_up<DT, 8>(a, stream);
}

}  // namespace

hipError_t launch_moe(const MoeArgs& a, int dtype, hipStream_t stream)
{
    hipError_t e = dtype == DT_BF16 ? launch_up_dt<DT_BF16>(a, stream) : launch_up_dt<DT_FP16>(a, stream);
    if (e != hipSuccess) return e;
    const size_t lds = (size_t)kMoeWaves * a.T * kDownRows * sizeof(float);
    moe_down_kernel<<<a.H / kDownRows, kMoeThreads, lds, stream>>>(
        reinterpret_cast<const uint16_t*>(static_cast<const char*>(a.work) + kMoeRoutingBytes), a.w2,
        a.s2, static_cast<const Routing*>(a.work), a.weights, a.y, a.T, a.H, a.I, a.top_k);
    return hipGetLastError();
}

}  // namespace fp8q
