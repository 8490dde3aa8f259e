// What the attention kernels over the paged FP8 cache share.
#pragma once

#include <float.h>

#include "half.hpp"
#include "paged.hpp"

namespace fp8q {

// A term is kept as fp16(2^kShift * term / reference).  The reference follows
// the largest term only where that outgrows it by more than 2^kSlack, so that
// the sums are seldom rescaled; fp16 then holds terms up to 2^15, and those
// down to 2^-23 of the reference with all its 11 bits.
constexpr float kSlack = 6.0f, kShift = 9.0f, kShiftScale = 0x1p9f;

constexpr int kKeys = 64;                 // keys of a tile

// A value that all lanes of the wave have, told to the compiler.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

struct KeyRange {
    int lo, hi;
};
// The keys that the new token i of a sequence sees.
__device__ __forceinline__ KeyRange key_range(const AttendArgs& a, const PagedSeq& q, int i)
{
    const int pos = q.start + i;
    KeyRange k{0, q.len};
    if (a.causal) {
        k.hi = clamp_int(pos + 1, 0, q.len);
        if (a.window > 0) k.lo = clamp_int(pos - a.window + 1, 0, k.hi);
    }
    return k;
}

struct PageRef {
    int page;                // 0 where there is none, so that an address can be made of it
    bool valid;
};
// The page with a key; none past the sequence's end.
__device__ __forceinline__ PageRef page_ref(const AttendArgs& a, int b, int len, int key)
{
    const int id = key < len ? a.batch.page_table[(int64_t)b * a.batch.W + (key >> a.page_shift)] : -1;
    const bool valid = id >= 0 && id < a.pages;
    return PageRef{valid ? id : 0, valid};
}

// Scales of a page and head: a term is 2^(s * key + log_value) with s = q k^T,
// times the values' scale, and counts inverse_value times that in the sum.
struct PageScales {
    float key, log_value, inverse_value;
};
__device__ __forceinline__ PageScales page_scales(const AttendArgs& a, const PageRef& page, int h)
{
    const int64_t cell = (int64_t)page.page * a.Hk + h;
    const float held = page_scale(a.v_scale[cell]), v = page.valid ? held : 1.0f;
    // never 0, which would make NaN of a masked key's -inf, nor infinite, which would of a logit of 0
    const float k = fminf(fmaxf(page_scale(a.k_scale[cell]) * a.scale_log2, FLT_MIN), FLT_MAX);
    return PageScales{k, __builtin_amdgcn_logf(v), __builtin_amdgcn_rcpf(v) * (1.0f / kShiftScale)};
}

// The denominator is summed from the terms of the numerators, which have the values' scale in them,
// as long as all scales of values lie within 2^-kNear .. 2^kNear.  A key that matters in the denominator
// (2^24 keys of 2^-48 of the largest do not, to fp32) is then a term, and the sum that it is in has a
// factor when the reference moves, of at least 2^(-48 - 2 kNear - kSlack) = 2^-126: nothing is lost.
// From the first scale outside on (`apart`), a wave sums its denominators from exponentials of their
// own, over a reference of their own: on pages of 2^-100 and 2^100 the keys that count most in the
// denominator may be 2^-200 of those in the numerator.  Asking costs prompts 1 to 3% (4096 tokens,
// 64/8 heads x 128: 297 us before, 301 with it) and other calls up to 0.7 us; where a scale is apart
// they take up to 17% more.
constexpr float kNear = 36.0f;
// Whether a lane's scale is apart.  Asked after the first codes of its pages are requested: before, they
// would wait for the scales.
__device__ __forceinline__ bool any_apart(const PageScales& s) { return __ballot(fabsf(s.log_value) > kNear) != 0; }
// 16 logarithms s(i) * key, of which `top` is the largest, to the sum l over the reference z.
template <class S>
__device__ __forceinline__ void add_apart(float& z, float& l, float top, float key, S s)
{
    const float z1 = fmaxf(z, top), ref = z1 == -__builtin_inff() ? 0.0f : z1;
    l *= __builtin_amdgcn_exp2f(z - ref);
#pragma unroll
    for (int i = 0; i < 16; ++i) l += __builtin_amdgcn_exp2f(__builtin_fmaf(s(i), key, -ref));
    z = z1;
}
// A row's denominator from the lanes that are `off` apart.
__device__ __forceinline__ void join_lanes(float& z, float& l, int off)
{
    const float mine = z;
    const float other = __shfl_xor(z, off), more = __shfl_xor(l, off);
    z = fmaxf(z, other);
    const float ref = z == -__builtin_inff() ? 0.0f : z;
    l = l * __builtin_amdgcn_exp2f(mine - ref) + more * __builtin_amdgcn_exp2f(other - ref);
}

// What a wave knows of the pages of the next tiles: lane i of the page with the i-th of 64 tiles where
// a page holds whole tiles (WIDE), else of the i-th of 64 groups of 16 keys.  Looked up together, so
// that no tile waits for its page's id or scales.
struct Pages {
    int page;                             // 0 where there is none
    PageScales sc;
    uint64_t valid;
};
template <bool WIDE>
constexpr int kLookUp = WIDE ? 64 : 16;   // tiles of a look-up
template <bool WIDE>
__device__ __forceinline__ Pages look_up(const AttendArgs& a, int b, int len, int key0, int h)
{
    const int key = key0 + (int)(threadIdx.x & 63) * (WIDE ? kKeys : 16);
    const PageRef p = page_ref(a, b, len, key);
    return Pages{p.page, page_scales(a, p, h), __ballot(p.valid)};
}

// The E4M3 codes of NaN in four codes, as 0x80 in their bytes.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w)
{
    return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}

// Clears the codes of NaN in 16 codes; not 0 if there were any.
__device__ __forceinline__ uint32_t clear_nan(v4i& v)
{
    uint32_t any = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t n = nan_bytes((uint32_t)v[k]);
        v[k] = (int)((uint32_t)v[k] & ~((n >> 7) * 255u));
        any |= n;
    }
    return any;
}
// E4M3 1.0 where NaN is in 16 codes, 0 elsewhere.
__device__ __forceinline__ v4i nan_ones(const v4i& v)
{
    v4i one;
#pragma unroll
    for (int k = 0; k < 4; ++k) one[k] = (int)((nan_bytes((uint32_t)v[k]) >> 7) * 0x38u);
    return one;
}

// Terms of keys that a row does not see become 2^-inf.  Their values must not
// count either, but 0 * NaN would: codes of NaN become 0 and, where a row does
// see one, NaN is added to its sum.
template <int ND>
__device__ __forceinline__ void mask_tile(v4f (&s)[4], v4f (&acc)[ND], v4i (&vf)[ND],
                                          const KeyRange& see, int key0, int g, bool valid)
{
    const float none = -__builtin_inff();
    v8h seen[2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int key = key0 + 16 * g + 4 * i + e;
            const bool in = valid && key >= see.lo && key < see.hi;
            s[i][e] = in ? s[i][e] : none;
            seen[i >> 1][(i & 1) * 4 + e] = in ? (_Float16)1.0f : (_Float16)0.0f;
        }
    uint32_t any = 0;
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int k = 0; k < 4; ++k) any |= nan_bytes((uint32_t)vf[d][k]);
    if (__ballot(any != 0) == 0) return;
#pragma unroll
    for (int d = 0; d < ND; ++d) {
        const v4i one = nan_ones(vf[d]);
        clear_nan(vf[d]);
        v4f hits = {0.f, 0.f, 0.f, 0.f};
        hits = __builtin_amdgcn_mfma_f32_16x16x32_f16(Half<DT_FP16>::widen(one[0], one[1]), seen[0],
                                                      hits, 0, 0, 0);
        hits = __builtin_amdgcn_mfma_f32_16x16x32_f16(Half<DT_FP16>::widen(one[2], one[3]), seen[1],
                                                      hits, 0, 0, 0);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[d][e] += hits[e] > 0.f ? __builtin_nanf("") : 0.f;
    }
}

// References of a row's sums and of its denominator (0 where there was no key), and its denominator.
struct Joined {
    float ref, z, l;
};
// Four channels of a row from its sums, and the row's lse from its first channels.
template <int DT>
__device__ __forceinline__ void store_row(const AttendArgs& a, int64_t token, int head, int d, v4f o,
                                          const Joined& j)
{
    const bool empty = j.l == 0.0f;         // not by the maximum, which skips NaN
    const float f = empty ? 0.0f : 1.0f / (j.l * kShiftScale), e = __builtin_amdgcn_exp2f(j.ref - j.z);
    const int64_t row = token * a.Hq + head;
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const v2f x = {empty ? 0.0f : o[2 * i] * f * e, empty ? 0.0f : o[2 * i + 1] * f * e};
        if constexpr (DT == DT_BF16) w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(x, v2b));
        else w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(x, v2h));
    }
    *reinterpret_cast<v2i*>(a.y + row * a.D + d) = v2i{(int)w[0], (int)w[1]};
    if (d == 0 && a.lse != nullptr)
        a.lse[row] = empty ? -__builtin_inff() : (j.z + __builtin_amdgcn_logf(j.l)) * 0.6931471805599453f;
}

}  // namespace fp8q
