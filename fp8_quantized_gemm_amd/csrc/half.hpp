// E4M3 codes widened to 16-bit floats (exact) as operands of the 16-bit MFMA.
#pragma once

#include "common.hpp"

namespace fp8q {

typedef float v2f __attribute__((ext_vector_type(2)));
typedef __bf16 v2b __attribute__((ext_vector_type(2)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));

// Eight codes (two dwords) -> one operand; mfma: 16x16x32 with the widened
// codes as the first operand and 8 values of the type as the second.
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

}  // namespace fp8q
