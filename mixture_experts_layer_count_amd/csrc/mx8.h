// MXFP8 of activation checkpoints: E4M3 codes with one E8M0 scale per 32
// consecutive values of a row.
//
// Scale: the smallest power of two 2^e with max|x| <= 448 2^e over the
// group's finite values (448 is E4M3's largest value, so nothing saturates),
// e in [-126, 127], byte e + 127; an all-zero group has e = 0. Code:
// E4M3(x 2^-e), round to nearest, ties to even: x 2^-e is exact in fp32, so
// the code is the one rounding. NaN and infinities become the NaN code and do
// not move the group's scale.
// A power of two, not max|x| / 448 as the W8A8 path has: code * 2^e (four
// significant bits) is then a bf16 value, and the backward pass multiplies
// checkpoints on the bf16 matrix cores with no second rounding.
#pragma once

#include "train.h"

namespace moe {
namespace mx8 {

constexpr int kGroup = 32;

__device__ __forceinline__ bool finite_bits(uint32_t b) { return (b & 0x7f800000u) != 0x7f800000u; }

// exponent of a group whose largest finite magnitude has these fp32 bits
__device__ __forceinline__ int scale_exp(uint32_t amax) {
    if (amax == 0) return 0;
    const int e = (int)(amax >> 23) - 135 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);
    return e < -126 ? -126 : e;
}
// fp32 2^e of a normal exponent
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// x 2^-e for the conversion below (inv = 2^-e); non-finite values become NaN
__device__ __forceinline__ float scaled(float x, float inv) {
    return finite_bits(__float_as_uint(x)) ? x * inv : __uint_as_float(0x7fc00000u);
}
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
    int p = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, p, true);
}
// |x| bits for the group maximum (0 for non-finite values)
__device__ __forceinline__ uint32_t amax_bits(float x) {
    const uint32_t b = __float_as_uint(x) & 0x7fffffffu;
    return b < 0x7f800000u ? b : 0u;
}
// the four values of a code word, times 2^e
__device__ __forceinline__ f32x4 values4(uint32_t w, float s) {
    // the conversion multiplies by the scale's exponent
    const auto lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, s, false);
    const auto hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, s, true);
    return f32x4{lo[0], lo[1], hi[0], hi[1]};
}
__device__ __forceinline__ float scale_of(uint8_t byte) { return __uint_as_float((uint32_t)byte << 23); }

}  // namespace mx8
}  // namespace moe
