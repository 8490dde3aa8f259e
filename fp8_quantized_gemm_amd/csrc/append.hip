// Appending to the paged FP8 cache: rotation by position, one power-of-two
// scale per (page, head), E4M3 codes, and the queries' rotation in the same
// launch.
//
//   (a, b) -> (a c - b s, b c + a s);  s = 2^e with amax <= 448 s, never
//   below the page's;  code = E4M3_rne_sat(x / s)
//
// A unit is one page of one sequence that gains tokens; it has one workgroup
// for each key/value head's keys, one for its values and a few for the
// queries of its tokens, so a page's scale has one writer and no atomics are
// needed.  An item is 16 values of one token: with half-split pairs 8 values
// and the 8 they pair with, else 16 neighbours.  A workgroup holds its items
// in registers between the maximum and the quantization, so everything is read
// once.  A power of two as the scale makes the older codes' rescaling, when a
// page's scale grows, a shift of exponents, and divisions multiplications.
//
// Many tokens are bound by HBM: 2048 tokens of 32/32 heads x 128 move 85 MB in
// 22 us (3.9 TB/s; a copy of that size 17 us).  Few are bound by the chain of
// dependent loads (lengths, page, scale) and the launch: 1 token 4.9 us, 48
// tokens 8.5 us, in 64 threads where a page's new tokens have at most 64 items.
// Keys and values asked for before their page is known took as long (9.3 us
// both ways for one token, before the queries had workgroups of 64 items).
#include "paged.hpp"

namespace fp8q {
namespace {

typedef float v8f __attribute__((ext_vector_type(8)));
typedef v8f v8f_aligned16 __attribute__((aligned(16)));
struct Items {
    v8f a, b;
};

template <int DT>
__device__ __forceinline__ v8f load8(const uint16_t* p)
{
    const v4i v = *reinterpret_cast<const v4i*>(p);
    v8f f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = half_bits_to_f32<DT>((uint32_t)v[i] & 0xffffu);
        f[2 * i + 1] = half_bits_to_f32<DT>((uint32_t)v[i] >> 16);
    }
    return f;
}

template <int DT>
__device__ __forceinline__ void store8(uint16_t* p, const v8f& f)
{
    v4i v;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = (int)(f32_to_out_bits<DT>(f[2 * i]) | (f32_to_out_bits<DT>(f[2 * i + 1]) << 16));
    *reinterpret_cast<v4i*>(p) = v;
}
static_assert((int)OUT_BF16 == (int)DT_BF16 && (int)OUT_FP16 == (int)DT_FP16, "one numbering");

// Offsets of an item's two vectors of 8 values in its head.
__device__ __forceinline__ void item_offsets(int item, int R, int interleaved, int& va, int& vb)
{
    const bool split = !interleaved && item < (R >> 4);
    va = split ? 8 * item : 16 * item;
    vb = split ? va + (R >> 1) : va + 8;
}

// Pairs (a, b) -> (a c - b s, b c + a s), each product and sum rounded to fp32.
__device__ __forceinline__ void rotate_item(Items& x, int item, const float* rope, int R,
                                            int interleaved)
{
    if (item >= (R >> 4)) return;
    const v8f c = *reinterpret_cast<const v8f_aligned16*>(rope + 8 * item);
    const v8f s = *reinterpret_cast<const v8f_aligned16*>(rope + (R >> 1) + 8 * item);
    v8f a = x.a, b = x.b;
    if (interleaved) {
        a = __builtin_shufflevector(x.a, x.b, 0, 2, 4, 6, 8, 10, 12, 14);
        b = __builtin_shufflevector(x.a, x.b, 1, 3, 5, 7, 9, 11, 13, 15);
    }
    const v8f ta = a * c - b * s, tb = b * c + a * s;
    x.a = ta;
    x.b = tb;
    if (interleaved) {
        x.a = __builtin_shufflevector(ta, tb, 0, 8, 1, 9, 2, 10, 3, 11);
        x.b = __builtin_shufflevector(ta, tb, 4, 12, 5, 13, 6, 14, 7, 15);
    }
}

__device__ __forceinline__ float finite_abs(float v)
{
    const float a = fabsf(v);
    return a < __builtin_inff() ? a : 0.0f;     // infinities and NaN do not count
}

// The smallest power of two s with amax <= 448 s, 448 = 1.75 * 2^8.
__device__ __forceinline__ float pow2_scale(float amax)
{
    const uint32_t u = __float_as_uint(amax);
    const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return __uint_as_float((uint32_t)(clamp_int(e, kMinPageExp, kMaxPageExp) + 127) << 23);
}

// x / s correctly rounded; a power of two's reciprocal is exact.
struct Divide {
    float s, r;
    bool pow2;
    __device__ __forceinline__ explicit Divide(float s_) : s(s_), r(1.0f / s_)
    {
        pow2 = (__float_as_uint(s_) & 0x7fffffu) == 0;
    }
    __device__ __forceinline__ float operator()(float x) const { return pow2 ? x * r : x / s; }
};

__device__ __forceinline__ v2i codes8(const v8f& f, const Divide& d)
{
    return v2i{(int)e4m3_pack4(d(f[0]), d(f[1]), d(f[2]), d(f[3])),
               (int)e4m3_pack4(d(f[4]), d(f[5]), d(f[6]), d(f[7]))};
}

// Four codes to a smaller share of a larger scale.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float ratio)
{
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
    const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    return e4m3_pack4_in_range(lo[0] * ratio, lo[1] * ratio, hi[0] * ratio, hi[1] * ratio);
}

// The sequence and the number within it of unit u.  A sequence of n new tokens
// touches at most n / P + 2 pages (rounded down), so its units begin at
// q_start[b] / P + 2 b; the workgroup counts the sequences that begin at or
// before u.
template <int NT>
__device__ __forceinline__ int find_sequence(const PagedBatch& s, int u, int P, int* lds, int& first)
{
    int below = 0;
    for (int b = threadIdx.x; b < s.B; b += NT)
        below += clamp_int(s.q_start[b], 0, s.T) / P + 2 * b <= u ? 1 : 0;
    const int b = max(block_sum_int<NT>(below, lds) - 1, 0);
    first = clamp_int(s.q_start[b], 0, s.T) / P + 2 * b;
    return b;
}

// NT threads with at most NI items each.
template <int DT, int NT, int NI>
__global__ void __launch_bounds__(NT) kv_append_kernel(const AppendArgs a, int query_heads)
{
    __shared__ int lds_i[NT / 64];
    __shared__ float lds_f[NT / 64];
    __shared__ __attribute__((aligned(16))) uint8_t tile[NT * NI * 16];

    const PagedBatch& s = a.batch;
    const int P = a.P, D = a.D, tid = threadIdx.x;
    int b = blockIdx.x, first = blockIdx.x;
    if (s.max_q > 1) b = find_sequence<NT>(s, blockIdx.x, P, lds_i, first);
    const PagedSeq q = paged_seq(s, b, P);
    const int begin = max(q.start, 0), slot = begin / P + ((int)blockIdx.x - first);
    const int lo = max(begin, slot * P), hi = min(min(q.len, q.start + q.n), (slot + 1) * P);
    const int count = hi - lo;
    if (count <= 0 || slot < 0 || slot >= s.W) return;
    const int64_t row0 = (int64_t)q.row + (lo - q.start);
    const int per = D >> 4;                        // items of a token and head
    int y = blockIdx.y;

    if (y >= 2 * a.Hk) {                           // the queries of the unit's tokens
        const int h0 = (y - 2 * a.Hk) * query_heads, heads = min(query_heads, a.Hq - h0);
        const int items = count * heads * per;
        for (int i = tid; i < items; i += NT) {
            const int item = i % per, h = h0 + i / per % heads, t = i / (per * heads);
            int va, vb;
            item_offsets(item, a.R, a.interleaved, va, vb);
            const uint16_t* src = a.q + (row0 + t) * a.q_stride + (int64_t)h * D;
            uint16_t* dst = a.q_out + (row0 + t) * a.q_out_stride + (int64_t)h * D;
            Items x;
            x.a = load8<DT>(src + va);
            x.b = load8<DT>(src + vb);
            rotate_item(x, item, a.rope + (int64_t)(lo + t) * a.R, a.R, a.interleaved);
            store8<DT>(dst + va, x.a);
            store8<DT>(dst + vb, x.b);
        }
        return;
    }

    const int page = s.page_table[(int64_t)b * s.W + slot];
    if (page < 0 || page >= a.pages) return;       // no page: the tokens are dropped
    const bool values = y >= a.Hk;
    const int h = values ? y - a.Hk : y;
    const int64_t cell = (int64_t)page * a.Hk + h;
    uint8_t* codes = (values ? a.v_pages : a.k_pages) + cell * P * D;
    float* scale = (values ? a.v_scale : a.k_scale) + cell;
    const int older = lo - slot * P;               // tokens that the page holds already
    const float held = older > 0 ? page_scale(*scale) : 0.0f;

    const uint16_t* src = values ? a.v + row0 * a.v_stride + (int64_t)h * D
                                 : a.k + row0 * a.k_stride + (int64_t)h * D;
    const int64_t stride = values ? a.v_stride : a.k_stride;
    const int items = count * per, R = values ? 0 : a.R;
    Items x[NI];
    float m = 0.0f;
#pragma unroll
    for (int j = 0; j < NI; ++j) {
        const int i = tid + j * NT;
        if (i < items) {
            const int item = i % per, t = i / per;
            int va, vb;
            item_offsets(item, R, a.interleaved, va, vb);
            x[j].a = load8<DT>(src + t * stride + va);
            x[j].b = load8<DT>(src + t * stride + vb);
            rotate_item(x[j], item, a.rope + (int64_t)(lo + t) * R, R, a.interleaved);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                m = fmaxf(m, fmaxf(finite_abs(x[j].a[e]), finite_abs(x[j].b[e])));
        }
    }
    m = block_max<NT>(m, lds_f);
    const float sc = fmaxf(held, pow2_scale(m));
    const Divide div(sc);
    const bool grow = held > 0.0f && sc > held;
    const float ratio = held / sc;
    if (tid == 0) *scale = sc;

#pragma unroll
    for (int j = 0; j < NI; ++j) {
        const int i = tid + j * NT;
        if (i < items) {
            const int item = i % per, t = i / per;
            int va, vb;
            item_offsets(item, R, a.interleaved, va, vb);
            uint8_t* dst = values ? tile + t * D : codes + (older + t) * D;
            *reinterpret_cast<v2i*>(dst + va) = codes8(x[j].a, div);
            *reinterpret_cast<v2i*>(dst + vb) = codes8(x[j].b, div);
        }
    }
    if (!values) {
        if (grow)
            for (int i = tid; i < older * D / 4; i += NT) {
                uint32_t* w = reinterpret_cast<uint32_t*>(codes) + i;
                *w = rescale4(*w, ratio);
            }
        return;
    }
    __syncthreads();
    // channel by channel, 16 tokens at a time: the unit's tokens from the tile, older ones
    // rescaled where the scale grew, the bytes behind left as they are
    const int g0 = grow ? 0 : older >> 4, groups = ((older + count + 15) >> 4) - g0;
    for (int i = tid; i < groups * D; i += NT) {
        const int d = i % D, g = (g0 + i / D) << 4;
        uint8_t* dst = codes + (int64_t)d * P + g;
        const int from = max(older - g, 0), to = min(older + count - g, 16);
        if (from == 0 && to == 16) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint8_t* p = tile + (g + 4 * e - older) * D + d;
                w[e] = (uint32_t)p[0] | (uint32_t)p[D] << 8 | (uint32_t)p[2 * D] << 16 |
                       (uint32_t)p[3 * D] << 24;
            }
            *reinterpret_cast<v4i*>(dst) = v4i{(int)w[0], (int)w[1], (int)w[2], (int)w[3]};
        } else {
            if (grow)
                for (int e = 0; e < min(from, 16); ++e)
                    dst[e] = (uint8_t)(rescale4(dst[e], ratio) & 0xffu);
            for (int e = from; e < to; ++e) dst[e] = tile[(g + e - older) * D + d];
        }
    }
}

template <int DT>
hipError_t launch(const AppendArgs& a, hipStream_t stream)
{
    const PagedBatch& s = a.batch;
    const int most = s.max_q < a.P ? s.max_q : a.P, items = most * a.D / 16;
    const int64_t units = s.max_q == 1 ? s.B : (int64_t)s.T / a.P + 2 * (int64_t)s.B;
    int query_heads = 1, qy = 0;
    if (a.q != nullptr) {
        // a query workgroup's threads have one or two items each: one token with 64 query and 8
        // key/value heads takes 4.9 us (9.3 with all heads in one workgroup of 64 threads), 48 with
        // 32 and 32 heads 8.5 (10.9)
        const int most = items <= 64 ? 64 : 512;
        query_heads = most / (items < most ? items : most);
        if (query_heads > a.Hq) query_heads = a.Hq;
        qy = (a.Hq + query_heads - 1) / query_heads;
    }
    const dim3 grid((unsigned)units, (unsigned)(2 * a.Hk + qy));
    if (items <= 64) {
        hipLaunchKernelGGL((kv_append_kernel<DT, 64, 1>), grid, dim3(64), 0, stream, a, query_heads);
    } else if (items <= 512) {
        hipLaunchKernelGGL((kv_append_kernel<DT, 256, 2>), grid, dim3(256), 0, stream, a, query_heads);
    } else {
        hipLaunchKernelGGL((kv_append_kernel<DT, 256, 8>), grid, dim3(256), 0, stream, a, query_heads);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_append(const AppendArgs& a, int dtype, hipStream_t stream)
{
    return dtype == DT_BF16 ? launch<DT_BF16>(a, stream) : launch<DT_FP16>(a, stream);
}

}  // namespace fp8q
