// A mixture-of-experts layer for a few tokens on block-scaled FP8 weights, in
// two kernels up to 16 tokens and three above.
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
// logits are a few KiB, and up to kRouteInline tokens a launch of its own
// (moe_route_kernel) would cost more.  It then deals items, some columns of
// one expert's h, out to the waves.  The second (moe_down) gives each
// workgroup 8 to 32 columns of y and all chosen experts, so the weighted sum
// over experts needs no atomics and no kernel of its own.
//
// Both stream weight rows through the MFMA operand layout of Layout, a wave
// at a time, without any exchange between lanes or waves.
#include <float.h>
#include <math.h>

#include <algorithm>
#include <atomic>

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
static_assert(kMoeMaxTokens <= 64, "an expert's tokens are a 64-bit mask");

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

// Inclusive sum over the lanes of a wave (DPP).
__device__ __forceinline__ int wave_scan(int v)
{
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, true);    // row_shr 1
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, true);    // row_shr 2
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, true);    // row_shr 4
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, true);    // row_shr 8
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);   // row_bcast15 -> rows 1, 3
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);   // row_bcast31 -> rows 2, 3
    return v;
}

// The experts that any token chose, in ascending order: 64 experts to a word.
// first[i] is the number of pairs of the experts before expert 64 i + lane.
template <int PER>
struct Active {
    uint64_t word[PER];
    int first[PER];
    int count;
    __device__ __forceinline__ void find(const uint64_t* masks, int experts, int lane)
    {
        count = 0;
        int pairs = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = i * 64 + lane;
            const int n = e < experts ? __popcll(masks[e]) : 0;
            word[i] = __ballot(n != 0);
            count += __popcll(word[i]);
            const int scan = wave_scan(n);
            first[i] = pairs + scan - n;
            pairs += __builtin_amdgcn_readlane(scan, 63);
        }
    }
    __device__ __forceinline__ int first_pair(int e) const
    {
        int p = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (e >> 6 == i) p = __builtin_amdgcn_readlane(first[i], e & 63);
        return p;
    }
    // the slot-th of them
    __device__ __forceinline__ int expert(int slot, int lane) const
    {
        int e = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int n = __popcll(word[i]);
            if (slot >= 0 && slot < n) {
                const bool here = (word[i] >> lane & 1) != 0 && lanes_below(word[i]) == slot;
                e = i * 64 + __ffsll((unsigned long long)__ballot(here)) - 1;
            }
            slot -= n;
        }
        return __builtin_amdgcn_readfirstlane(e);
    }
    // set bits of a wave-uniform mask below this lane
    static __device__ __forceinline__ int lanes_below(uint64_t m)
    {
        return __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0));
    }
};

// An expert's tokens, the p-th of them in lane p.
struct Tokens {
    int count, list;
    __device__ __forceinline__ void find(const uint64_t* masks, int e, int lane)
    {
        const uint64_t v = masks[e];
        const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
        const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
        const uint64_t m = (uint64_t)hi << 32 | lo;
        count = __popcll(m);
        // tokens that chose the expert go to the first lanes, the others behind them
        const int below = Active<1>::lanes_below(m);
        const int to = (m >> lane & 1) != 0 ? below : count + lane - below;
        list = __builtin_amdgcn_ds_permute(to << 2, lane);
    }
    // the p-th token, -1 past the last
    __device__ __forceinline__ int at(int p) const
    {
        const int t = __shfl(list, p & 63);
        return p < count ? t : -1;
    }
};

// ---------------------------------------------------------------- operand layout
// R weight rows (8 or 4) per load instruction, 1024 / R bytes of each.  The
// Q = 16 / R lanes r of a row take Q pieces of its K range as operand rows of
// their own, r = Q row + q, so that neighbouring lanes read neighbouring 16
// bytes: lane (r, g) reads unit 2 g + q % 2 of K block q / 2.  (With the lanes
// of a row eight apart every lane is in another line than the lanes beside
// it, and a load instruction occupies the CU's cache for twice as long.)  The
// tokens are laid out the same way, and of the 16 x 16 results those that
// pair equal q add up to the product.
template <int R>
struct Layout {
    static constexpr int Q = 16 / R;
    static constexpr int kBlocks = 8 / R;                  // K blocks per load
    static constexpr int kOut = R / 4;                     // results per lane after fold
    int row, koff, block;                                  // koff, block: within the load's K range
    int out_row;                                           // first of the lane's results
    bool owner;                                            // one lane of Q holds them
    __device__ __forceinline__ explicit Layout(int lane)
    {
        const int r = lane & 15, g = lane >> 4, q = r % Q;
        row = r / Q;
        block = q / 2;
        koff = block * kBlock + (2 * g + q % 2) * 16;
        out_row = kOut * g;
        owner = q == 0;
    }
    // Result 4 g + i of lane (r, g) is row (4 g + i) / Q with piece i % Q, for
    // token r / Q with piece r % Q: picks and adds up the equal ones.
    __device__ __forceinline__ void fold(const v4f& d, int lane, float (&out)[kOut]) const
    {
        if constexpr (R == 8) {
            out[0] = (lane & 1) != 0 ? d[1] : d[0];
            out[1] = (lane & 1) != 0 ? d[3] : d[2];
        } else {
            const float lo = (lane & 1) != 0 ? d[1] : d[0], hi = (lane & 1) != 0 ? d[3] : d[2];
            out[0] = (lane & 2) != 0 ? hi : lo;
        }
#pragma unroll
        for (int i = 0; i < kOut; ++i) {
            out[i] += dpp<0xB1>(out[i]);                   // quad_perm [1,0,3,2]
            if constexpr (R == 4) out[i] += dpp<0x4E>(out[i]);   // quad_perm [2,3,0,1]
        }
    }
    template <int CTRL>
    static __device__ __forceinline__ float dpp(float v)
    {
        return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
    }
};

// Where column i of h stands in its row.  The down projection's lane of unit
// u multiplies columns 16 u .. 16 u + 15 of a block with two MFMAs of eight
// each; the first eights of all units come first, so that each of its two
// loads reads whole 128-byte lines (with the columns in order it read 16 bytes
// of every 32: moe_down at 64 tokens of 128 experts of 768 x 2048, with h in
// bf16, 58.4 us, so 43.8).
// Rows are padded to whole blocks.
__device__ __forceinline__ int h_position(int i)
{
    return (i & ~127) | (i & 8) << 3 | (i >> 4 & 7) << 3 | (i & 7);
}
// h is kept in fp16 with a power of two for every four columns of a pair, the
// exponent of the largest of them: two bytes a value, as in bf16, with 2^-11
// instead of 2^-8 lost, over fp32's whole range.  The stored values bring the
// largest of the four to [2^kHStored, 2^(kHStored + 1)), and moe_down the largest
// of a block to [2^kHTop, 2^(kHTop + 1)), the top of fp16 but one binade for
// the rounding.  Values far below those are subnormal or gone: with half of kHTop
// on either side (the factors are fp16 too) they are off by less than 2^-31 of
// the block's largest.  In bf16 the error of y is 1.4 times that of its own
// rounding, in this form 1.01 times.  64 tokens, 8 of 128 experts, 2048 x 768 take 115 us a call, 110 with
// bf16 alone.  Two bf16 values for each h, the second for what the first
// leaves out, lose less still, but moe_down is bound by its reads of h from
// the L2: 129 us.
constexpr int kHGroup = 4;
constexpr int kHStored = 7, kHTop = 14;

// The exponents of a pair, a byte a group: those of a 16-column unit in the
// `blocks` (1 to 3) K blocks that moe_down takes at a time stand together, so
// that a lane reads them at once and the lanes of a token read neighbouring
// bytes (a load for each block: 64 tokens, 6 of 64 experts, 2048 x 1408 120
// against 116 us).  The room for them is that of three blocks, the most.
__host__ __device__ constexpr int exp_slot(int blocks) { return blocks == 3 ? 16 : 4 * blocks; }
__host__ __device__ constexpr int exp_stride(int I) { return ((I + kBlock - 1) / kBlock + 2) / 3 * 8 * exp_slot(3); }
__device__ __forceinline__ int exp_position(int i, int blocks)
{
    const int kb = i / kBlock, item = kb / blocks;
    return (item * 8 + (i >> 4 & 7)) * exp_slot(blocks) + (kb - item * blocks) * 4 + (i >> 2 & 3);
}

// The larger of the values here and in the lane 16 (32) away.
__device__ __forceinline__ uint32_t max_xor16(uint32_t v)
{
    const auto p = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return max((uint32_t)p[0], (uint32_t)p[1]);
}
__device__ __forceinline__ uint32_t max_xor32(uint32_t v)
{
    const auto p = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return max((uint32_t)p[0], (uint32_t)p[1]);
}

__device__ __forceinline__ int h_stride(int I) { return (I + kBlock - 1) / kBlock * kBlock; }

// ---------------------------------------------------------------- selection, a kernel of its own
// One wave per token.  Used above kRouteInline tokens, where repeating the
// selection in every workgroup of moe_up costs more than a launch.
template <int PER>
__global__ __launch_bounds__(64) void moe_route_kernel(const float* __restrict__ logits,
                                                       int* __restrict__ ids,
                                                       float* __restrict__ weights, int E,
                                                       int top_k, int renormalize)
{
    const int t = blockIdx.x, lane = threadIdx.x;
    int id;
    float weight;
    route_token<PER>(logits + (size_t)t * E, E, top_k, renormalize, lane, id, weight);
    if (lane < top_k) {
        ids[t * top_k + lane] = id;
        weights[t * top_k + lane] = weight;
    }
}

// ---------------------------------------------------------------- gate and up projections
// Every wave works on its own: an item is RT * R columns of h of one expert,
// and the wave streams their gate and up rows (2 RT row tiles, which share the
// loads of x) over all of K, UB loads of each tile at a time, for up to MT * R
// tokens (a longer list takes another pass over the weights).  Items are
// dealt out with consecutive ones on different workgroups, so that few items
// still use every CU.
//
// h and the weights it will be summed with are stored grouped by expert (the
// p-th token of an expert at first_pair + p), so that the second kernel reads
// an expert's rows without looking them up, and each row block by block in
// the order of the second kernel's operands (h_position).
//
// With ROUTED the selection is there already (moe_route_kernel); without it
// every workgroup makes it, and the first one stores it.
template <int DT, int PER, int R, int RT, int MT, int UB, int WAVES, int OCC, bool ROUTED>
__global__ __launch_bounds__(WAVES * 64) __attribute__((amdgpu_waves_per_eu(OCC)))
void moe_up_kernel(
    const uint16_t* __restrict__ x, const float* __restrict__ logits,
    const uint8_t* __restrict__ w13, const float* __restrict__ s13, int* __restrict__ ids_io,
    float* __restrict__ weights_io, uint64_t* __restrict__ masks_out,
    float* __restrict__ pair_weights, uint16_t* __restrict__ h, uint8_t* __restrict__ h_exp, int T,
    int H, int I, int E, int top_k, int renormalize, int down_blocks)
{
    typedef Layout<R> L;
    constexpr int KL = L::kBlocks * kBlock;                // K per load
    constexpr int COLS = R * RT;
    __shared__ uint64_t masks[PER * 64];
    __shared__ int ids[kMaxPairs];
    __shared__ float wt[kMaxPairs];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const L at(lane);

    for (int i = tid; i < PER * 64; i += WAVES * 64) masks[i] = 0;
    __syncthreads();
    auto choose = [&](int pair, int t, int id, float weight) {
        ids[pair] = id;
        wt[pair] = weight;
        // a bit of its own per token: the order of the updates does not matter
        if (id >= 0) atomicOr(reinterpret_cast<uint32_t*>(&masks[id]) + (t >> 5), 1u << (t & 31));
    };
    if constexpr (ROUTED) {
        for (int p = tid; p < T * top_k; p += WAVES * 64) choose(p, p / top_k, ids_io[p], weights_io[p]);
    } else {
        for (int t = wave; t < T; t += WAVES) {
            int id;
            float weight;
            route_token<PER>(logits + (size_t)t * E, E, top_k, renormalize, lane, id, weight);
            if (lane < top_k) {
                const int p = t * top_k + lane;
                choose(p, t, id, weight);
                if (blockIdx.x == 0) {
                    ids_io[p] = id;
                    weights_io[p] = weight;
                }
            }
        }
    }
    __syncthreads();
    if (blockIdx.x == 0)
        for (int i = tid; i < E; i += WAVES * 64) masks_out[i] = masks[i];
    Active<PER> active;
    active.find(masks, E, lane);

    const int nblk = (H + kBlock - 1) / kBlock, nb = (I + kBlock - 1) / kBlock;
    const int tiles = I / COLS;
    const int items = active.count * tiles;
    const rsrc_t rx = make_rsrc(x, (uint32_t)(T * H * 2));
    for (int it = wave * gridDim.x + blockIdx.x; it < items; it += WAVES * gridDim.x) {
        const int slot = it / tiles;
        const int i0 = (it - slot * tiles) * COLS;
        const int e = active.expert(slot, lane);
        const int first = active.first_pair(e);
        Tokens tokens;
        const size_t row = (size_t)e * 2 * I + i0;                   // gate row; up: + I
        const rsrc_t rw[2] = {make_rsrc(w13 + row * H, (uint32_t)(COLS * H)),
                              make_rsrc(w13 + (row + I) * H, (uint32_t)(COLS * H))};
        // an item's columns lie in one block of 128
        const float* const sg = s13 + ((size_t)e * 2 * nb + (i0 >> 7)) * nblk;
        const rsrc_t rs[2] = {make_rsrc(sg, (uint32_t)(nblk * 4)),
                              make_rsrc(sg + (size_t)nb * nblk, (uint32_t)(nblk * 4))};
        int p0 = 0;
        do {                                                         // an active expert has a token
            uint32_t xo[MT];                                         // of this lane's token
            v4f acc[MT][RT][2];
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int n = 0; n < RT; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c) acc[m][n][c] = v4f{0.f, 0.f, 0.f, 0.f};
            for (int k0 = 0; k0 < H; k0 += UB * KL) {
                v4i w[UB][RT][2], xv[UB][MT][2];
                float s[UB][2];
#pragma unroll
                for (int u = 0; u < UB; ++u) {
                    const int k = k0 + u * KL;
                    const uint32_t past = k + at.koff < H ? 0u : kOOB;
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
#pragma unroll
                        for (int n = 0; n < RT; ++n)
                            w[u][n][c] = buf_load16<CP_NT>(
                                rw[c], (uint32_t)((n * R + at.row) * H + k + at.koff) + past);
                        // zero past the last block
                        s[u][c] = __int_as_float(__builtin_amdgcn_raw_buffer_load_b32(
                            rs[c], (uint32_t)((k >> 7) + at.block) * 4, 0, 0));
                    }
                }
                if (k0 == 0) {                                       // beside the first weights' way
                    if (p0 == 0) tokens.find(masks, e, lane);
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        const int t = tokens.at(p0 + m * R + at.row);
                        xo[m] = t >= 0 ? (uint32_t)(t * H + at.koff) * 2 : kOOB;
                    }
                }
#pragma unroll
                for (int u = 0; u < UB; ++u) {
                    const int k = k0 + u * KL;
                    const bool past = k + at.koff >= H;
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        const uint32_t o = past || xo[m] == kOOB ? kOOB : xo[m] + (uint32_t)k * 2;
                        xv[u][m][0] = buf_load16(rx, o);
                        xv[u][m][1] = buf_load16(rx, o + 16);
                    }
                }
                if (i0 == 0 && k0 == 0 && p0 == 0 && lane < tokens.count) {
                    // the weight of expert e among the choices of token tokens.list
                    float v = 0.0f;
                    for (int j = 0; j < top_k; ++j)
                        if (ids[tokens.list * top_k + j] == e) v = wt[tokens.list * top_k + j];
                    pair_weights[first + lane] = v;
                }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int u = 0; u < UB; ++u)
#pragma unroll
                    for (int n = 0; n < RT; ++n)
#pragma unroll
                        for (int c = 0; c < 2; ++c)
#pragma unroll
                            for (int m = 0; m < MT; ++m) {
                                const v4f p = block_product<DT>(w[u][n][c], xv[u][m][0], xv[u][m][1]);
#pragma unroll
                                for (int q = 0; q < 4; ++q)
                                    acc[m][n][c][q] = __builtin_fmaf(p[q], s[u][c], acc[m][n][c][q]);
                            }
            }
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int n = 0; n < RT; ++n) {
                    float gv[L::kOut], uv[L::kOut];
                    at.fold(acc[m][n][0], lane, gv);
                    at.fold(acc[m][n][1], lane, uv);
                    float hv[L::kOut], largest = 0.0f;
#pragma unroll
                    for (int q = 0; q < L::kOut; ++q) {
                        hv[q] = gv[q] / (1.0f + expf(-gv[q])) * uv[q];
                        largest = fmaxf(largest, fabsf(hv[q]));      // passes over a NaN
                    }
                    // a group's columns are 4 / kOut lanes 16 apart
                    uint32_t top = max_xor16(__float_as_uint(largest));
                    if constexpr (L::kOut == 1) top = max_xor32(top);
                    const int exponent = max((int)(top >> 23), 1);
                    const int p = p0 + m * R + at.row, i = i0 + n * R + at.out_row;
                    if (at.owner && p < tokens.count) {
                        uint16_t* const dst = h + (size_t)(first + p) * h_stride(I) + h_position(i);
                        uint32_t bits[L::kOut];
#pragma unroll
                        for (int q = 0; q < L::kOut; ++q)
                            bits[q] = f32_to_f16_bits(__builtin_ldexpf(hv[q], 127 + kHStored - exponent));
                        if constexpr (L::kOut == 2)
                            *reinterpret_cast<uint32_t*>(dst) = bits[0] | bits[1] << 16;
                        else
                            *dst = (uint16_t)bits[0];
                        if (at.out_row % kHGroup == 0)
                            h_exp[(first + p) * exp_stride(I) + exp_position(i, down_blocks)] = (uint8_t)exponent;
                    }
                }
            p0 += MT * R;
        } while (p0 < tokens.count);
    }
}

// ---------------------------------------------------------------- down projection
// A workgroup owns RT row tiles of eight columns of y.  Its waves take items of
// BLOCKS K blocks of one expert; the next item's weights, and the rows of h of
// its first eight tokens, are requested before the current one's products.
// Each wave adds its products, weighted, to sums of its own in LDS; the waves'
// sums are added in a fixed order at the end.
constexpr int kDownRows = 8;                // columns of y (rows of W2) per row tile

template <int PER, int RT, int BLOCKS, int CP>
__global__ __launch_bounds__(kMoeThreads) void moe_down_kernel(
    const uint16_t* __restrict__ h, const uint8_t* __restrict__ h_exp,
    const uint8_t* __restrict__ w2, const float* __restrict__ s2,
    const uint64_t* __restrict__ masks_in, const float* __restrict__ pair_weights,
    uint16_t* __restrict__ y, int T, int H, int I, int E, int top_k)
{
    typedef Layout<kDownRows> L;
    constexpr int COLS = RT * kDownRows;
    // weight scales: one where the columns lie in one block of 128, else one a tile
    constexpr int FS = kBlock % COLS == 0 ? 1 : RT;
    __shared__ uint64_t masks[PER * 64];
    __shared__ float wt[kMaxPairs];
    extern __shared__ __attribute__((aligned(16))) float ysum[];   // [waves][T][COLS]
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const L at(lane);
    const int n0 = blockIdx.x * COLS;

    if (tid < E) masks[tid] = masks_in[tid];
    for (int i = tid; i < T * top_k; i += kMoeThreads) wt[i] = pair_weights[i];
    for (int i = tid; i < kMoeWaves * T * COLS; i += kMoeThreads) ysum[i] = 0.0f;
    __syncthreads();
    Active<PER> active;
    active.find(masks, E, lane);

    const int nblk = (I + kBlock - 1) / kBlock;
    const int chunks = (nblk + BLOCKS - 1) / BLOCKS;
    const int items = active.count * chunks;
    const rsrc_t rh = make_rsrc(h, (uint32_t)(T * top_k * h_stride(I) * 2));
    const rsrc_t re = make_rsrc(h_exp, (uint32_t)(T * top_k * exp_stride(I)));
    float* const mine = ysum + wave * T * COLS;

    struct Rows {
        v4i v[BLOCKS][2];
        uint32_t e[BLOCKS];
    };
    // rows of h of pair p (none: zeros) in the K blocks from kb0, as stored:
    // two operands and the exponents of their four groups.  What is not there
    // is moved out of range by an addition, not by a branch.
    auto load_h = [&](Rows& rows, int p, bool none, int kb0) {
        const uint32_t past = none ? kOOB : 0u;
#pragma unroll
        for (int c = 0; c < BLOCKS; ++c) {
            const int kb = (kb0 + c) * kBlock;
            const uint32_t o = (uint32_t)(p * h_stride(I) + kb + at.koff / 2) * 2 +
                               (kb + at.koff < I ? past : kOOB);
            rows.v[c][0] = buf_load16(rh, o);
            rows.v[c][1] = buf_load16(rh, o + 128);
        }
        const uint32_t o = (uint32_t)(p * exp_stride(I) + (kb0 / BLOCKS * 8 + at.koff / 16) * exp_slot(BLOCKS)) + past;
        if constexpr (BLOCKS == 1) {
            rows.e[0] = __builtin_amdgcn_raw_buffer_load_b32(re, o, 0, 0);
        } else if constexpr (BLOCKS == 2) {
            const auto e = __builtin_amdgcn_raw_buffer_load_b64(re, o, 0, 0);
            rows.e[0] = e[0], rows.e[1] = e[1];
        } else {
            const auto e = __builtin_amdgcn_raw_buffer_load_b96(re, o, 0, 0);
            rows.e[0] = e[0], rows.e[1] = e[1], rows.e[2] = e[2];
        }
    };
    // brings the values of block c to the largest exponent among a token's
    // lanes, and returns the power of two they then lack
    auto align_h = [&](Rows& rows, int c, int kb0) {
        // none are stored past the last column
        const uint32_t e = (kb0 + c) * kBlock + at.koff < I ? rows.e[c] : 0u;
        const int e4[4] = {(int)(e & 255), (int)(e >> 8 & 255), (int)(e >> 16 & 255), (int)(e >> 24)};
        uint32_t top = (uint32_t)max(max(e4[0], e4[1]), max(e4[2], e4[3]));
        top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0xB1, 0xf, 0xf, true));
        top = max_xor32(max_xor16(top));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const _Float16 f = __builtin_amdgcn_ldexph((_Float16)(1 << (kHTop - kHStored)), e4[i] - (int)top);
            v4i& v = rows.v[c][i / 2];
#pragma unroll
            for (int j = i % 2 * 2; j < i % 2 * 2 + 2; ++j) {
                const int two = v[j];          // (a bit cast of v[j] itself reads v[0])
                v[j] = __builtin_bit_cast(int, __builtin_bit_cast(v2h, two) * v2h{f, f});
            }
        }
        return (int)top - 127 - kHTop;
    };
    struct Stage {
        v4i w[BLOCKS][RT];
        Rows h;
        float s[BLOCKS][FS];
        int kb0, first;
        Tokens tokens;
    };
    // past the last item the loads are still issued, out of range, so that
    // the number of loads in flight, and with it the wait, is always the same
    auto request = [&](Stage& st, int it) {
        const uint32_t none = it < items ? 0u : kOOB;
        it = min(it, items - 1);
        const int slot = it / chunks;
        st.kb0 = (it - slot * chunks) * BLOCKS;
        const int e = active.expert(slot, lane);
        const rsrc_t rw = make_rsrc(w2 + ((size_t)e * H + n0) * I, (uint32_t)(min(COLS, H - n0) * I));
        const float* sb[FS];
#pragma unroll
        for (int n = 0; n < FS; ++n)
            sb[n] = s2 + ((size_t)e * ((H + kBlock - 1) / kBlock) + (min(n0 + n * kDownRows, H - 1) >> 7)) *
                             nblk;
#pragma unroll
        for (int c = 0; c < BLOCKS; ++c) {
            const int kb = st.kb0 + c;
#pragma unroll
            for (int n = 0; n < RT; ++n)
                st.w[c][n] = buf_load16<CP>(
                    rw, kb * kBlock + at.koff < I
                            ? (uint32_t)((n * kDownRows + at.row) * I + kb * kBlock + at.koff) | none : kOOB);
#pragma unroll
            for (int n = 0; n < FS; ++n) st.s[c][n] = sb[n][min(kb, nblk - 1)];
        }
        st.first = active.first_pair(e);
        st.tokens.find(masks, e, lane);
        load_h(st.h, st.first + at.row, none != 0 || at.row >= st.tokens.count, st.kb0);
        __builtin_amdgcn_sched_barrier(0);
    };
    auto compute = [&](Stage& st) {
        for (int p0 = 0; p0 < st.tokens.count; p0 += kDownRows) {
            const int p = p0 + at.row;
            if (p0 > 0) load_h(st.h, st.first + p, p >= st.tokens.count, st.kb0);
            const int t = st.tokens.at(p);
            const float f = t >= 0 ? wt[st.first + p] : 0.0f;
            int lack[BLOCKS];
#pragma unroll
            for (int c = 0; c < BLOCKS; ++c) lack[c] = align_h(st.h, c, st.kb0);
#pragma unroll
            for (int n = 0; n < RT; ++n) {
                v4f acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int c = 0; c < BLOCKS; ++c) {
                    const v4f q = block_product<DT_FP16>(st.w[c][n], st.h.v[c][0], st.h.v[c][1]);
                    float f = __builtin_ldexpf(st.s[c][FS == 1 ? 0 : n], lack[c]);
                    f = f > FLT_MAX ? FLT_MAX : f;       // a zero product stays zero
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(q[i], f, acc[i]);
                }
                float v[L::kOut];
                at.fold(acc, lane, v);
                // a token occurs once among an expert's pairs, so no two lanes meet
                if (at.owner && t >= 0) {
                    float2* const dst =
                        reinterpret_cast<float2*>(mine + t * COLS + n * kDownRows + at.out_row);
                    const float2 d = *dst;
                    *dst = make_float2(__builtin_fmaf(v[0], f, d.x), __builtin_fmaf(v[1], f, d.y));
                }
            }
        }
    };
    Stage a, b;
    if (wave < items) {
        request(a, wave);
        for (int it = wave;;) {
            request(b, it += kMoeWaves);
            compute(a);
            if (it >= items) break;
            request(a, it += kMoeWaves);
            compute(b);
            if (it >= items) break;
        }
    }
    __syncthreads();
    for (int o = tid; o < T * COLS; o += kMoeThreads) {
        float v = 0.0f;
#pragma unroll
        for (int i = 0; i < kMoeWaves; ++i) v += ysum[i * T * COLS + o];
        if (n0 + o % COLS < H)
            y[(size_t)(o / COLS) * H + n0 + o % COLS] = (uint16_t)f32_to_bf16_bits(v);
    }
}

// The workspace: the experts' token masks, the weights grouped like h, h and
// its exponents.
struct MoeWork {
    static constexpr int64_t kWeightsAt = kMoeMaxExperts * 8, kHAt = kWeightsAt + kMaxPairs * 4;
    static int64_t h_bytes(int64_t T, int64_t I, int64_t top_k)
    {
        return T * top_k * blocks_of(I) * kBlock * 2;
    }
    static int64_t bytes(int64_t T, int64_t I, int64_t top_k)
    {
        return kHAt + h_bytes(T, I, top_k) + T * top_k * exp_stride((int)I);
    }
    uint64_t* masks;
    float* weights;
    uint16_t* h;
    uint8_t* h_exp;
    explicit MoeWork(const MoeArgs& a)
    {
        char* const p = static_cast<char*>(a.work);
        masks = reinterpret_cast<uint64_t*>(p);
        weights = reinterpret_cast<float*>(p + kWeightsAt);
        h = reinterpret_cast<uint16_t*>(p + kHAt);
        h_exp = reinterpret_cast<uint8_t*>(p + kHAt + h_bytes(a.T, a.I, a.top_k));
    }
};

// moe_down's row tiles of eight columns, which share the loads of h: as many
// as leave at most one workgroup per CU (1024 columns of h, 4 of 16 experts,
// 8 / 40 tokens, microseconds a call: H = 2048 one 26.0 / 37.9, two 27.1 /
// 41.7; 2560 one 37.7 / 57.3, two 30.6 / 47.8; 4096 one 48.3 / 68.5, two 41.2
// / 58.9; 5120 two 54.9 / 80.8, three 49.2 / 68.4; 8192 three 81.6 / 112,
// four 72.9 / 95.1), four at most.
inline int down_tiles(const MoeArgs& a)
{
    return std::min((a.H + kDownRows * kCUs - 1) / (kDownRows * kCUs), 4);
}
// Its K blocks an item.  With one row tile three, what 128 registers hold,
// but two up to four tokens, where the items are few (one token, 8 of 128, 2048
// x 768: two 16.5, three 16.8 us; 64 tokens 120 and 116).  With more row tiles
// one (4096 x 1408, 2 of 8 experts, one token: one 14.6, two 15.2; 64 tokens
// 63.5 and 64.4).
inline int down_blocks(const MoeArgs& a) { return down_tiles(a) > 1 ? 1 : a.T <= 4 ? 2 : 3; }

template <int DT, int PER, int R, int RT, int MT, int UB, int WAVES, int OCC, bool ROUTED>
hipError_t launch_up(const MoeArgs& a, hipStream_t stream)
{
    const MoeWork work(a);
    const int64_t items = std::min<int64_t>(a.E, (int64_t)a.T * a.top_k) * (a.I / (R * RT));
    const int grid = (int)std::min<int64_t>(items, kCUs * OCC * 4 / WAVES);
    moe_up_kernel<DT, PER, R, RT, MT, UB, WAVES, OCC, ROUTED><<<grid, WAVES * 64, 0, stream>>>(
        static_cast<const uint16_t*>(a.x), a.logits, a.w13, a.s13, a.ids, a.weights, work.masks,
        work.weights, work.h, work.h_exp, a.T, a.H, a.I, a.E, a.top_k, a.renormalize, down_blocks(a));
    return hipGetLastError();
}

template <int PER, int RT, int BLOCKS, int CP>
hipError_t launch_down_cp(const MoeArgs& a, hipStream_t stream)
{
    constexpr int COLS = RT * kDownRows;
    auto kern = moe_down_kernel<PER, RT, BLOCKS, CP>;
    const size_t lds = (size_t)kMoeWaves * a.T * COLS * sizeof(float);
    static std::atomic<uint64_t> attr_devices{0};
    if (const hipError_t e = set_lds_limit_once(reinterpret_cast<const void*>(kern),
                                                kMoeWaves * kMoeMaxTokens * COLS * sizeof(float),
                                                attr_devices);
        e != hipSuccess)
        return e;
    const MoeWork work(a);
    kern<<<(a.H + COLS - 1) / COLS, kMoeThreads, lds, stream>>>(work.h, work.h_exp, a.w2, a.s2,
                                                                work.masks, work.weights, a.y, a.T,
                                                                a.H, a.I, a.E, a.top_k);
    return hipGetLastError();
}

// Non-temporal weight loads where rows of W2 are whole 128-byte lines; else a
// line is shared by two rows and has to stay for the second (4 of 32 experts
// of 4096 x 1392, 13 tokens: 96.3 against 91.4 us a call).
template <int PER, int RT, int BLOCKS>
hipError_t launch_down(const MoeArgs& a, hipStream_t stream)
{
    return a.I % kBlock == 0 ? launch_down_cp<PER, RT, BLOCKS, CP_NT>(a, stream)
                             : launch_down_cp<PER, RT, BLOCKS, CP_DEFAULT>(a, stream);
}

// Above this many tokens the selection is a kernel of its own: repeating it in
// every workgroup grows with T, its launch does not (32 tokens, 6 of 64
// experts, 2048 x 1408: 101 us repeated, 94 us with the kernel; 16 tokens, 4
// of 32, 4096 x 1392: 92.5 repeated, 101 with it).
constexpr int kRouteInline = 16;

// moe_up's items.  A wave holds R tokens' columns of R weight rows at once, RT
// such row tiles and MT token tiles (Layout: smaller R means longer runs of K).
//   R = 4 up to four tokens (1 token, 6 of 64, 2048 x 1408: 19.0 us a call,
//     19.7 with 8; 4 of 32, 4096 x 1392: 24.5 against 26.7).
//   Two row tiles share the loads of x wherever that leaves an item for every
//     wave (64 tokens, 6 of 64: 109.7 against 117.9 with one); with fewer
//     items the second tile idles waves (24 tokens, 4 of 32, 4096 x 1392: 114
//     against 102; 32 tokens, 2 of 8, 4096 x 1408: 51.1 against 39.7).
//   Two token tiles, which read an expert's rows once for 16 tokens, where an
//     expert has on average more than 3 tokens (one row tile: 4), so that many
//     have more than 8 (64 tokens, 6 of 64: 122 -> 109.7; 8 of 128, 2048 x
//     768: 115 -> 111; with 2 tokens each, 32 of 8 of 128: 94.2 -> 95.2; one
//     row tile, 48 of 4 of 32: 130 -> 123, 24: 102 -> 108).
// UB, the K steps in flight, is what 128 registers hold.
template <int DT, int PER>
hipError_t launch_both(const MoeArgs& a, hipStream_t stream)
{
    hipError_t e;
    if (a.T <= 4) {
        e = launch_up<DT, PER, 4, 1, 1, 4, 16, 4, false>(a, stream);
    } else if (a.T <= kRouteInline) {
        e = launch_up<DT, PER, 8, 1, 1, 4, 16, 4, false>(a, stream);
    } else {
        moe_route_kernel<PER><<<a.T, 64, 0, stream>>>(a.logits, a.ids, a.weights, a.E, a.top_k,
                                                     a.renormalize);
        const int pairs = a.T * a.top_k;
        if ((int64_t)std::min(a.E, pairs) * (a.I / 16) < kCUs * kMoeWaves) {
            if (pairs <= 4 * a.E)
                e = launch_up<DT, PER, 8, 1, 1, 4, 16, 4, true>(a, stream);
            else
                e = launch_up<DT, PER, 8, 1, 2, 2, 16, 4, true>(a, stream);
        } else {
            if (pairs <= 3 * a.E)
                e = launch_up<DT, PER, 8, 2, 1, 2, 16, 4, true>(a, stream);
            else
                e = launch_up<DT, PER, 8, 2, 2, 1, 16, 4, true>(a, stream);
        }
    }
    if (e != hipSuccess) return e;
    switch (down_tiles(a)) {
    case 1: return down_blocks(a) == 2 ? launch_down<PER, 1, 2>(a, stream) : launch_down<PER, 1, 3>(a, stream);
    case 2: return launch_down<PER, 2, 1>(a, stream);
    case 3: return launch_down<PER, 3, 1>(a, stream);
    default: return launch_down<PER, 4, 1>(a, stream);
    }
}

template <int DT>
hipError_t launch_moe_dt(const MoeArgs& a, hipStream_t stream)
{
    if (a.E <= 64) return launch_both<DT, 1>(a, stream);
    if (a.E <= 128) return launch_both<DT, 2>(a, stream);
    if (a.E <= 256) return launch_both<DT, 4>(a, stream);
    return launch_both<DT, 8>(a, stream);
}

}  // namespace

int64_t moe_work_bytes(int64_t T, int64_t I, int64_t top_k) { return MoeWork::bytes(T, I, top_k); }

hipError_t launch_moe(const MoeArgs& a, int dtype, hipStream_t stream)
{
    return dtype == DT_BF16 ? launch_moe_dt<DT_BF16>(a, stream) : launch_moe_dt<DT_FP16>(a, stream);
}

}  // namespace fp8q
