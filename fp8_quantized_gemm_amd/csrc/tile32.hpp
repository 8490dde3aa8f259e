// Attention's arithmetic for 32 query rows and 64 keys a wave, on tiles in LDS:
//
//   S^T = K Q^T   MFMA 32x32x16, keys along M, query rows along N
//   P   = 2^(S^T * ks + lv - m)   in the lane of its row
//   Y^T = V^T P   MFMA 32x32x16, channels along M
//
// The products run on 16-bit operands: E4M3 codes widen exactly to bf16 and
// fp16.  A lane of S^T holds 16 consecutive keys of one row for each 32 keys
// (the rows of K are put in LDS in the order that makes it so), which are the
// lane's part of the second product's operand, so P needs no exchange between
// lanes, and a row's maximum one.
#pragma once

#include "join.hpp"
#include "tile.hpp"

namespace fp8q {
namespace {

typedef float v16f __attribute__((ext_vector_type(16)));

template <int DT>
__device__ __forceinline__ v16f mfma32(typename Half<DT>::vec a, v4i b, v16f c)
{
    if constexpr (DT == DT_BF16)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, __builtin_bit_cast(v8b, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}

// 16 bytes for each active lane to lds_block + 16 * lane, asynchronously: from a buffer, or from any
// address.  Written as assembly because the compiler, which cannot tell the buffer being filled from
// the one being read, would wait for builtin loads of this kind before the next read of LDS, and no
// tile would be under way during the arithmetic.  They write no register; the kernel waits itself.
// Nor does the compiler look into the blocks for what an instruction needs before it reads a register: one
// wait state after a write of m0, five after a vector instruction wrote a word of the resource, which may be
// the last instruction before the block.
__device__ __forceinline__ uint32_t lds_address(const void* p)
{
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
}
__device__ __forceinline__ void buffer_to_lds(const v4i& rsrc, uint32_t lds_block, uint32_t offset)
{
    int m0;                               // kept for the compiler
    asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 2\n\t"
                 "buffer_load_dwordx4 %2, %3, 0 offen lds\n\ts_mov_b32 m0, %0"
                 : "=&s"(m0)
                 : "s"(uniform((int)lds_block)), "v"(offset), "s"(rsrc)
                 : "memory");
}
__device__ __forceinline__ void global_to_lds(const uint8_t* src, uint32_t lds_block)
{
    int m0;
    asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\t"
                 "global_load_lds_dwordx4 %2, off\n\ts_mov_b32 m0, %0"
                 : "=&s"(m0)
                 : "s"(uniform((int)lds_block)), "v"(src)
                 : "memory");
}
// The words of make_rsrc's resource.
__device__ __forceinline__ v4i rsrc_words(const uint8_t* base, int bytes)
{
    const uint64_t p = reinterpret_cast<uint64_t>(base);
    return v4i{uniform((int)(uint32_t)p), uniform((int)(uint32_t)(p >> 32)) & 0xffff, uniform(bytes), 0x00020000};
}

// Tiles in LDS.  Keys: row r of PITCH bytes is key 32 (r / 32) + key_of_row(r % 32), its 16-byte
// units exchanged by row.  Values: a channel's 64 bytes, units exchanged as by swz64.
__device__ __forceinline__ int key_of_row(int r) { return 16 * ((r >> 2) & 1) + 4 * (r >> 3) + (r & 3); }
template <int DP>
struct Tile {
    static constexpr int kPitch = DP <= 64 ? 64 : (DP <= 128 ? 128 : 256);
    static constexpr int kUnits = kPitch / 16;
    static constexpr int kKeyBytes = kKeys * kPitch, kValueBytes = DP * kKeys;
    static constexpr int kKeyBlocks = kKeyBytes / 1024, kValueBlocks = kValueBytes / 1024;
    static __device__ __forceinline__ int swizzle(int row)
    {
        return kUnits == 4 ? (row >> 1) & 3 : row & (kUnits - 1);
    }
    static __device__ __forceinline__ int key_at(int row, int u) { return row * kPitch + ((u ^ swizzle(row)) << 4); }
};

__device__ __forceinline__ v4i value_at(const uint8_t* vt, int d, int tb, int r, int hf)
{
    return *reinterpret_cast<const v4i*>(vt + swz64(32 * d + r, 2 * tb + hf));
}
__device__ __forceinline__ void times16(v16f& sum, const v4i& v, const v8h (&w)[2])
{
    sum = mfma32<DT_FP16>(Half<DT_FP16>::widen(v[0], v[1]), __builtin_bit_cast(v4i, w[0]), sum);
    sum = mfma32<DT_FP16>(Half<DT_FP16>::widen(v[2], v[3]), __builtin_bit_cast(v4i, w[1]), sum);
}

// Values of keys that a row does not see must not count, but 0 * NaN would.  A tile that is not
// whole is looked through for codes of NaN; if there are any the wave goes on with a copy that has
// 0 for them, and notes the channels where a row does see one.
template <int DP>
__device__ __forceinline__ bool any_nan(const uint8_t* vt, int r, int hf)
{
    uint32_t any = 0;
#pragma unroll
    for (int d = 0; d < DP / 32; ++d)
#pragma unroll
        for (int tb = 0; tb < 2; ++tb) {
            const v4i v = value_at(vt, d, tb, r, hf);
            any |= nan_bytes((uint32_t)v[0]) | nan_bytes((uint32_t)v[1]) | nan_bytes((uint32_t)v[2]) |
                   nan_bytes((uint32_t)v[3]);
        }
    return __ballot(any != 0) != 0;
}
template <int DP>
__device__ __forceinline__ void take_nan(uint32_t (&nan)[DP / 64], const uint8_t* vt, uint8_t* clean,
                                         const v8h (&seen)[2][2], int r, int hf)
{
    uint32_t got[DP / 64] = {};
#pragma unroll 1
    for (int d = DP / 32 - 1; d >= 0; --d) {               // 16 bits a time, the first channels last
        v16f hits;
#pragma unroll
        for (int i = 0; i < 16; ++i) hits[i] = 0.0f;
#pragma unroll
        for (int tb = 0; tb < 2; ++tb) {
            v4i v = value_at(vt, d, tb, r, hf);
            times16(hits, nan_ones(v), seen[tb]);
            clear_nan(v);
            *reinterpret_cast<v4i*>(clean + swz64(32 * d + r, 2 * tb + hf)) = v;
        }
#pragma unroll
        for (int j = DP / 64 - 1; j > 0; --j) got[j] = got[j] << 16 | got[j - 1] >> 16;
        got[0] <<= 16;
#pragma unroll
        for (int i = 0; i < 16; ++i) got[0] |= hits[i] > 0.f ? 1u << i : 0u;
    }
#pragma unroll
    for (int j = 0; j < DP / 64; ++j) nan[j] |= got[j];
}

// The larger of a lane's value and that of the lane 32 away.
__device__ __forceinline__ float max_halves(float v)
{
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
}

// What a wave has of its 32 query rows: lane (r, hf) half of row r's channels (32 d + 8 i + 4 hf ..),
// the row's reference, its own keys' share of the denominator and the reference of that (m, or one of
// its own once a scale of values was `apart`); a bit of `nan` for each channel that has seen NaN.
template <int DP>
struct Rows {
    v4i q[DP / 32][2];
    v16f acc[DP / 32];
    uint32_t nan[DP / 64];
    float m, l, z;
    bool apart;
};

// A tile's terms.  whole: every row sees every key; clean: room for a tile of values.
template <int DT, int DP, bool WIDE>
__device__ __forceinline__ void add_tile(Rows<DP>& x, const uint8_t* kt, const PageScales& sc, const KeyRange& see,
                                         int key0, bool valid, bool whole, uint8_t* clean)
{
    using T = Tile<DP>;
    constexpr int NC = DP / 32, ND = DP / 32;
    const int lane = threadIdx.x & 63, r = lane & 31, hf = lane >> 5;
    const uint8_t* vt = kt + T::kKeyBytes;
    v16f s[2];
#pragma unroll
    for (int tb = 0; tb < 2; ++tb)
#pragma unroll
        for (int i = 0; i < 16; ++i) s[tb][i] = 0.0f;
    // neighbouring matrix instructions add to different sums, so that none waits for the last
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        v4i k[2];
#pragma unroll
        for (int tb = 0; tb < 2; ++tb) k[tb] = *reinterpret_cast<const v4i*>(kt + T::key_at(32 * tb + r, 2 * c + hf));
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int tb = 0; tb < 2; ++tb)
                s[tb] = mfma32<DT>(Half<DT>::widen(k[tb][2 * e], k[tb][2 * e + 1]), x.q[c][e], s[tb]);
    }
    if (!whole) {
        const bool on_page[2] = {WIDE ? valid : __shfl(valid ? 1 : 0, hf) != 0,
                                 WIDE ? valid : __shfl(valid ? 1 : 0, 2 + hf) != 0};
        v8h seen[2][2];
#pragma unroll
        for (int tb = 0; tb < 2; ++tb) {
            const int key = key0 + 32 * tb + 16 * hf, lo = see.lo - key, hi = on_page[tb] ? see.hi - key : 0;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const bool in = i >= lo && i < hi;
                s[tb][i] = in ? s[tb][i] : -__builtin_inff();
                seen[tb][i >> 3][i & 7] = in ? (_Float16)1.0f : (_Float16)0.0f;
            }
        }
        if (any_nan<DP>(vt, r, hf)) {
            take_nan<DP>(x.nan, vt, clean, seen, r, hf);
            vt = clean;
        }
    }
    // logarithms: a term is 2^(s * ks + lv), times the values' scale; one page a lane and block
    float ks[2], lv[2], top[2];
#pragma unroll
    for (int tb = 0; tb < 2; ++tb) {
        ks[tb] = WIDE ? sc.key : __shfl(sc.key, 2 * tb + hf);
        lv[tb] = WIDE ? sc.log_value : __shfl(sc.log_value, 2 * tb + hf);
        top[tb] = s[tb][0];
#pragma unroll
        for (int i = 1; i < 16; ++i) top[tb] = fmaxf(top[tb], s[tb][i]);
    }
    if (x.apart) {
#pragma unroll
        for (int tb = 0; tb < 2; ++tb) add_apart(x.z, x.l, top[tb] * ks[tb], ks[tb], [&](int i) { return s[tb][i]; });
    }
#pragma unroll
    for (int tb = 0; tb < 2; ++tb) top[tb] = __builtin_fmaf(top[tb], ks[tb], lv[tb]);
    const float both = fmaxf(top[0], top[1]), highest = max_halves(both);
    if (__any(highest > x.m + kSlack)) {
        const float m1 = fmaxf(x.m, highest);
        const float alpha = m1 == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(x.m - m1);
#pragma unroll
        for (int d = 0; d < ND; ++d) x.acc[d] *= alpha;
        x.m = m1;
        x.l *= x.apart ? 1.0f : alpha;
        x.z = x.apart ? x.z : m1;
    }
    const float ref = x.m == -__builtin_inff() ? 0.0f : x.m;
    v8h p[2][2];
#pragma unroll
    for (int tb = 0; tb < 2; ++tb) {
        const float offset = lv[tb] - (ref - kShift);
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
            const v2f v = {__builtin_amdgcn_exp2f(__builtin_fmaf(s[tb][i], ks[tb], offset)),
                           __builtin_amdgcn_exp2f(__builtin_fmaf(s[tb][i + 1], ks[tb], offset))};
            sum += v[0];
            sum += v[1];
            const v2h w = __builtin_convertvector(v, v2h);
            p[tb][i >> 3][i & 7] = w[0];
            p[tb][i >> 3][(i & 7) + 1] = w[1];
        }
        const float inverse = WIDE ? sc.inverse_value : __shfl(sc.inverse_value, 2 * tb + hf);
        x.l = __builtin_fmaf(sum, x.apart ? 0.0f : inverse, x.l);
    }
#pragma unroll
    for (int tb = 0; tb < 2; ++tb)
#pragma unroll
        for (int d0 = 0; d0 < ND; d0 += 2) {
            const v4i v[2] = {value_at(vt, d0, tb, r, hf), value_at(vt, d0 + 1, tb, r, hf)};
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    x.acc[d0 + i] = mfma32<DT_FP16>(Half<DT_FP16>::widen(v[i][2 * e], v[i][2 * e + 1]),
                                                    __builtin_bit_cast(v4i, p[tb][e]), x.acc[d0 + i]);
        }
}

// The rows' queries, and nothing seen so far.
template <int DP>
__device__ __forceinline__ void begin_rows(const AttendArgs& a, Rows<DP>& x, bool have_row, int64_t token, int head, int hf)
{
    const uint16_t* src = a.q + token * a.q_stride + (int64_t)head * a.D;
    const v4i zero = {0, 0, 0, 0};
#pragma unroll
    for (int c = 0; c < DP / 32; ++c) {
        const int d = 32 * c + 16 * hf;
        const bool have = have_row && d < a.D;
        x.q[c][0] = have ? *reinterpret_cast<const v4i*>(src + d) ^ a.q_flip : zero;
        x.q[c][1] = have ? *reinterpret_cast<const v4i*>(src + d + 8) ^ a.q_flip : zero;
    }
#pragma unroll
    for (int d = 0; d < DP / 32; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) x.acc[d][i] = 0.0f;
#pragma unroll
    for (int d = 0; d < DP / 64; ++d) x.nan[d] = 0u;
    x.m = x.z = -__builtin_inff();
    x.l = 0.0f;
    x.apart = false;
}

// The rows' results: to the output, or to a partial result (at this lane's row).  l is whole already.
template <int DT, int DP>
__device__ __forceinline__ void end_rows(const AttendArgs& a, const Rows<DP>& x, int64_t token, int head, float* part, int hf)
{
    const Joined j{x.m == -__builtin_inff() ? 0.0f : x.m, x.z == -__builtin_inff() ? 0.0f : x.z, x.l};
    if (part != nullptr && hf == 0) { part[0] = x.m; part[1] = x.l; part[2] = x.z; }
#pragma unroll
    for (int d = 0; d < DP / 32; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int c = 32 * d + 8 * e + 4 * hf;
            v4f o;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                o[i] = (x.nan[d >> 1] >> (16 * (d & 1) + 4 * e + i) & 1u) != 0 ? __builtin_nanf("") : x.acc[d][4 * e + i];
            if (c >= a.D) continue;
            if (part != nullptr) *reinterpret_cast<v4f*>(part + 4 + c) = o;
            else store_row<DT>(a, token, head, c, o, j);
        }
}

// The scales of the i-th tile of a look-up as add_tile takes them, and whether its pages are there.
template <bool WIDE>
__device__ __forceinline__ PageScales tile_scales(const Pages& p, int i, bool& valid)
{
    const int lane = threadIdx.x & 63, at = WIDE ? i : 4 * i + (lane & 3);
    valid = (p.valid >> at & 1) != 0;
    const auto pick = [&](float v) {
        return WIDE ? __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), i)) : __shfl(v, at);
    };
    return PageScales{pick(p.sc.key), pick(p.sc.log_value), pick(p.sc.inverse_value)};
}

// Requests KB blocks of a tile's keys and VB of its values, 1 KiB each, from `block` on (in units of KB
// and VB): the i-th tile of a look-up, whose first key is key0, to LDS at dst.  WIDE: the tile is on
// one page, so a lane's offsets are the same in every tile; channels past D are out of the buffer's
// range (values) or sent there (keys) and become 0.  Else a tile's keys are in four groups of 16, each
// on one page, and channels past D are not written.
template <int DP, bool WIDE, int KB, int VB>
__device__ __forceinline__ void request_tile(const AttendArgs& a, const Pages& p, int i, int key0, int h, int block,
                                             uint32_t dst)
{
    using T = Tile<DP>;
    const int lane = threadIdx.x & 63;
    const uint32_t page_bytes = (uint32_t)(a.P * a.D), pool_stride = (uint32_t)a.Hk * page_bytes;
    const uint8_t* const kbase = a.k_pages + (uint32_t)h * page_bytes;
    const uint8_t* const vbase = a.v_pages + (uint32_t)h * page_bytes;
    const auto key_unit = [&](int j, int& key, int& c) {
        const int unit = (block * KB + j) * 64 + lane, row = unit / T::kUnits;
        c = (unit % T::kUnits) ^ T::swizzle(row);
        key = (row & 32) + key_of_row(row & 31);
    };
    const auto value_unit = [&](int j, int& d, int& g) {
        d = (block * VB + j) * 16 + (lane >> 2);
        g = (lane & 3) ^ ((d >> 1) & 3);
    };
    const uint32_t kdst = dst + block * KB * 1024, vdst = dst + T::kKeyBytes + block * VB * 1024;
    if constexpr (WIDE) {
        const uint64_t at = (uint64_t)(uint32_t)__builtin_amdgcn_readlane(p.page, i) * pool_stride;
        const uint32_t inside = (uint32_t)(key0 & (a.P - 1));
        const v4i rk = rsrc_words(kbase + at + inside * (uint32_t)a.D, kKeys * a.D);
        const v4i rv = rsrc_words(vbase + at + inside, (int)(page_bytes - inside));
#pragma unroll
        for (int j = 0; j < KB; ++j) {
            int key, c;
            key_unit(j, key, c);
            buffer_to_lds(rk, kdst + j * 1024, 16 * c < a.D ? (uint32_t)(key * a.D + 16 * c) : kOOB);
        }
#pragma unroll
        for (int j = 0; j < VB; ++j) {
            int d, g;
            value_unit(j, d, g);
            buffer_to_lds(rv, vdst + j * 1024, (uint32_t)(d * a.P + 16 * g));
        }
    } else {
#pragma unroll
        for (int j = 0; j < KB; ++j) {
            int key, c;
            key_unit(j, key, c);
            const uint64_t at = (uint64_t)(uint32_t)__shfl(p.page, 4 * i + (key >> 4)) * pool_stride;
            if (16 * c < a.D)
                global_to_lds(kbase + at + (uint32_t)(((key0 + key) & (a.P - 1)) * a.D + 16 * c), kdst + j * 1024);
        }
#pragma unroll
        for (int j = 0; j < VB; ++j) {
            int d, g;
            value_unit(j, d, g);
            const uint64_t at = (uint64_t)(uint32_t)__shfl(p.page, 4 * i + g) * pool_stride;
            if (d < a.D) global_to_lds(vbase + at + (uint32_t)(d * a.P + ((key0 + 16 * g) & (a.P - 1))), vdst + j * 1024);
        }
    }
}

// Channels that no request fills, where there are any, cleared once: `bytes` of LDS by `threads`.
__device__ __forceinline__ void clear_lds(uint8_t* p, int bytes, int thread, int threads)
{
    for (int i = thread; i < bytes / 16; i += threads) *reinterpret_cast<v4i*>(p + 16 * i) = v4i{0, 0, 0, 0};
}

}  // namespace
}  // namespace fp8q
