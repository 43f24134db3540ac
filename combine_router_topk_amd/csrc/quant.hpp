// 8-bit rows: e4m3 codes with one fp32 scale for each block of 128 columns.
// s = max(amax, 2^-100) / 448, code = v / s rounded to nearest even, so a
// block's largest value takes the largest code. 2^-100 keeps s and v / s
// ordinary numbers in a block of zeros. A block that holds an infinity or a
// NaN takes s = NaN: every value of it is NaN.
#pragma once

#include <type_traits>

#include "device.hpp"

namespace moe {

constexpr int kScaleBlock = 128;
constexpr float kE4m3Max = 448.0f;

__host__ __device__ constexpr int scale_blocks(int cols) { return (cols + kScaleBlock - 1) / kScaleBlock; }

// The scale of a block from the largest magnitude in it, as bits: among bits
// without the sign every NaN is above infinity, and that above every number.
__device__ __forceinline__ float block_scale(uint32_t amax_bits) {
  if (amax_bits >= 0x7f800000u) return __uint_as_float(0x7fc00000u);
  const float amax = fmaxf(__uint_as_float(amax_bits), 0x1p-100f);
  const float s = amax * (1.0f / kE4m3Max);  // and what its rounding leaves
  return fmaf(fmaf(-kE4m3Max, s, amax), 1.0f / kE4m3Max, s);
}

// 1 / s of such a scale: the hardware's reciprocal and one Newton step.
__device__ __forceinline__ float inverse(float s) {
  const float i = __builtin_amdgcn_rcpf(s);
  return fmaf(fmaf(-s, i, 1.0f), i, i);
}

// g / (1 + exp(-g)): exp(-g) as 2^t (1 + d), t the rounded product of -g and
// log2(e) and d what its rounding and the constant's leave out; the hardware's
// 2^t and reciprocal are within one step of fp32, so the whole is within 8 half
// steps. Below g = -69, where 1 / (1 + exp(-g)) nears the end of the ordinary
// numbers, the result is g exp(g); g of -infinity gives NaN, as the formula
// does. (expf and a division take as long, 1049 us against 1052 for the gate and
// up products of 16384 tokens, top-2 of 64 experts, 4096 x 2048, and give 0 from
// -88.8 down; without the last branch it is 1030 us.)
__device__ __forceinline__ float silu(float g) {
  constexpr float kLog2e = 1.44269504f, kRest = 1.92596299e-8f, kLn2 = 0.693147181f;
  const float t = keep_f32(-g * kLog2e);  // rounded wherever it is used
  const float d = (fmaf(-g, kLog2e, -t) - g * kRest) * kLn2;
  const float e = __builtin_amdgcn_exp2f(t);
  // beyond that range 1 + e is 1, or d is of no use: it is NaN at infinities
  const float x = fabsf(t) < 126.0f ? fmaf(e, d, e) : e;
  float y = g * __builtin_amdgcn_rcpf(1.0f + x);
  if (ballot(t > 100.0f) != 0) {  // hardly ever
    const float r = __builtin_amdgcn_exp2f(64.0f - t);  // exp(g) 2^64: below 2^-126 the product is 0
    // d has no use for an r of 0, and is infinite where t is (g below -2.36e38)
    if (t > 100.0f) y = g * 0x1p-64f * (t < 256.0f ? fmaf(r, -d, r) : r);
  }
  return y;
}

// Two values in the activation format, the first in the low half; one
// conversion for both in bf16.
template <int ACT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (ACT == 1) {
    return f32_to_f16(a) | (f32_to_f16(b) << 16);
  } else {
    typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
    const v2bf v = {static_cast<__bf16>(a), static_cast<__bf16>(b)};
    return __builtin_bit_cast(uint32_t, v);
  }
}

template <int ACT>
__device__ __forceinline__ uint4 round8(const float (&f)[8]) {
  return make_uint4(pack2<ACT>(f[0], f[1]), pack2<ACT>(f[2], f[3]), pack2<ACT>(f[4], f[5]), pack2<ACT>(f[6], f[7]));
}

// 4 values as 4 codes, the first in the low byte; inv = 1 / s. v inv is within
// 1.5 steps of fp32 of v / s, which takes one reciprocal a block instead of a
// division a value. It exceeds 448 by no more than that, and rounds to 448 then.
__device__ __forceinline__ uint32_t quant4(float a, float b, float c, float d, float inv) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a * inv, b * inv, 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(c * inv, d * inv, w, true);
  return static_cast<uint32_t>(w);
}

__device__ __forceinline__ uint2 quant8(const float (&f)[8], float inv) {
  return make_uint2(quant4(f[0], f[1], f[2], f[3], inv), quant4(f[4], f[5], f[6], f[7], inv));
}

// 4 e4m3 codes as 4 values of the activation format (1: fp16, 2: bf16); every
// e4m3 number is one of either.
template <int ACT>
__device__ __forceinline__ uint2 widen4(uint32_t codes) {
  const int c = static_cast<int>(codes);
  if constexpr (ACT == 1)
    return make_uint2(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c, 1.0f, false)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c, 1.0f, true)));
  else
    return make_uint2(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.0f, false)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.0f, true)));
}

// c += a b for 16 x 32 by 32 x 16 values in 16 bits: lane (r, g) = (lane % 16,
// lane / 16) holds 8 values of row r of each operand, the same columns of
// both, and gets rows 4 g .. 4 g + 3 of column r.
typedef float v4f __attribute__((ext_vector_type(4)));
template <int ACT>
__device__ __forceinline__ v4f mfma16(const uint4& a, const uint4& b, const v4f& c) {
  typedef _Float16 v8h __attribute__((ext_vector_type(8)));
  typedef __bf16 v8b __attribute__((ext_vector_type(8)));
  if constexpr (ACT == 1)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8b, a), __builtin_bit_cast(v8b, b), c, 0, 0, 0);
}

}  // namespace moe
