// half_ops.h -- bf16 and fp16 in pairs, their 4-bit (e2m1) forms and matrix
// products, chosen by mhc_dtype.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "seam_internal.h"

namespace mhc {
namespace {

typedef uint32_t u32;
typedef uint64_t u64;
typedef u32 u32x2 __attribute__((ext_vector_type(2)));
typedef u32 u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// 2^(byte - 127), byte 255 NaN, as the conversions below take it: they read the
// exponent field alone (0 stands for 2^-127)
__device__ __forceinline__ float scale_of(u32 byte) { return __uint_as_float(byte << 23); }

template <int DT> struct Half;

template <> struct Half<MHC_BF16> {
    typedef __bf16 type;
    static constexpr u32 kInf = 0x7f80;            // magnitudes from here on: infinity, NaN
    static constexpr int kLow = -125, kHigh = 125; // exponents of a group's scale
    // Values of byte SEL of w (low half first) times scale, a pair
    template <int SEL> static __device__ __forceinline__ u32 from_fp4(u32 w, float scale)
    {
        return __builtin_bit_cast(u32, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, SEL));
    }
    // Byte SEL of old replaced by the codes of a pair over scale
    template <int SEL> static __device__ __forceinline__ u32 to_fp4(u32 old, u32 pair, float scale)
    {
        return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(old, __builtin_bit_cast(bf16x2, pair), scale, SEL);
    }
    static __device__ __forceinline__ u32 pack(float a, float b)
    {
        return __builtin_bit_cast(u32, bf16x2{(__bf16)a, (__bf16)b});
    }
    static __device__ __forceinline__ float low(u32 w) { return __uint_as_float(w << 16); }
    static __device__ __forceinline__ f32x4 mfma16(const u32x4 &a, const u32x4 &b, const f32x4 &c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b),
                                                       c, 0, 0, 0);
    }
    static __device__ __forceinline__ f32x16 mfma32(const u32x4 &a, const u32x4 &b, const f32x16 &c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b),
                                                       c, 0, 0, 0);
    }
};

template <> struct Half<MHC_F16> {
    typedef _Float16 type;
    static constexpr u32 kInf = 0x7c00;
    static constexpr int kLow = -23, kHigh = 13;
    template <int SEL> static __device__ __forceinline__ u32 from_fp4(u32 w, float scale)
    {
        return __builtin_bit_cast(u32, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, SEL));
    }
    template <int SEL> static __device__ __forceinline__ u32 to_fp4(u32 old, u32 pair, float scale)
    {
        return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(old, __builtin_bit_cast(f16x2, pair), scale, SEL);
    }
    static __device__ __forceinline__ u32 pack(float a, float b)
    {
        return __builtin_bit_cast(u32, f16x2{(_Float16)a, (_Float16)b});
    }
    static __device__ __forceinline__ float low(u32 w) { return (float)__builtin_bit_cast(f16x2, w)[0]; }
    static __device__ __forceinline__ f32x4 mfma16(const u32x4 &a, const u32x4 &b, const f32x4 &c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c,
                                                      0, 0, 0);
    }
    static __device__ __forceinline__ f32x16 mfma32(const u32x4 &a, const u32x4 &b, const f32x16 &c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c,
                                                      0, 0, 0);
    }
};

}  // namespace
}  // namespace mhc
