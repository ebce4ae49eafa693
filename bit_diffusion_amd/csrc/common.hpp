// common.hpp -- device-side helpers shared by the gfx950 kernels of libsvdq.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

namespace svdq {

constexpr int kWave = 64;

__device__ __forceinline__ float bf16_to_f32(uint32_t h16) {
    return __uint_as_float(h16 << 16);
}

// fp32 -> bf16, round to nearest even (NaN kept quiet).
__device__ __forceinline__ uint32_t f32_to_bf16(float f) {
    uint32_t u = __float_as_uint(f);
    if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0x7FC0u;
    u += 0x7FFFu + ((u >> 16) & 1u);
    return u >> 16;
}

// Two fp32 -> two bf16 in one word (the first in the low half), round to nearest even: one
// v_cvt_pk_bf16_f32.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}

// The 8 bf16 words of a 16-byte register block as an MFMA operand.
__device__ __forceinline__ bf16x8 as_bf16x8(uint4 v) { return __builtin_bit_cast(bf16x8, v); }

__device__ __forceinline__ float wave_max_xor(float v, int mask) {
    return fmaxf(v, __shfl_xor(v, mask, kWave));
}

// 1 / sqrt(x), x >= 0, by the hardware's rsq (about 1 ulp), which takes subnormal numbers for 0.
__device__ __forceinline__ float rsqrt_hw(float x) {
    const bool tiny = x < 0x1p-126f;
    const float r = __builtin_amdgcn_rsqf(tiny ? x * 0x1p64f : x);
    return tiny ? r * 0x1p32f : r;
}

// Lane moves by DPP (a few cycles where a shuffle through LDS takes a hundred): lane i gets
// `src` of lane i - N of its row of 16 (kShr + N), of the row before's last lane (kBcast15, rows 1
// and 3) or of lane 31 (kBcast31, rows 2 and 3), and `old` where there is no such lane.  Joining
// with kShr + 1, 2, 4, 8, then kBcast15 (rows 0xa), then kBcast31 (rows 0xc) is an inclusive scan.
constexpr int kShr = 0x110, kBcast15 = 0x142, kBcast31 = 0x143;
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ int dpp(int old, int src) {
    return __builtin_amdgcn_update_dpp(old, src, CTRL, ROWS, 0xf, false);
}
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ float dpp(float old, float src) {
    return __int_as_float(dpp<CTRL, ROWS>(__float_as_int(old), __float_as_int(src)));
}

// GELU, tanh form: 0.5 y (1 + tanh(u)), u = sqrt(2/pi) (y + 0.044715 y^3).  Evaluated as
// the identical y / (1 + exp(-2u)), which keeps full relative accuracy for negative y where
// 1 + tanh(u) would cancel, with the hardware's exp2 and reciprocal (about 1 ulp each):
// e = 2^(-2 log2(e) u) and y * rcp(1 + e).  A relative error d in e moves the result by
// at most e / (1 + e)^2 * d <= d / 4 of y, so the argument's rounding (|d| up to |x| ulp
// for x = -2 log2(e) u) is damped where |x| is large; the result is within a few ulp of
// |y|.  e overflows to inf for large negative y, whose reciprocal 0 gives the limit -0.
__device__ __forceinline__ float gelu_tanh(float y) {
    const float c = 0.7978845608028654f;   // sqrt(2 / pi)
    const float u = c * (y + 0.044715f * y * y * y);
    const float e = __builtin_amdgcn_exp2f(-2.8853900817779268f * u);   // -2 log2(e) u
    return y * __builtin_amdgcn_rcpf(1.0f + e);
}

// SiLU: y / (1 + exp(-y)), on the hardware's exp2 and reciprocal as above.
__device__ __forceinline__ float silu(float y) {
    return y * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * y));
}

// The activation of a svdq_act value.
__device__ __forceinline__ float activate(float y, int act) {
    if (act == 1) return gelu_tanh(y);
    if (act == 2) return silu(y);
    return y;
}

}  // namespace svdq
