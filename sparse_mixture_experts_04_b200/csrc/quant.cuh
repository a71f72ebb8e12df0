// Symmetric 8-bit quantisation of a row, shared by the kernels that quantise
// token rows, hidden rows and (at load time) weights.
//
//   scale = max(fl32(max|v| * fl32(1 / 127)), 2^-126)
//   q     = the integer nearest to v / scale, ties to even, in [-127, 127]
//
// (The product with the rounded 1 / 127, not the quotient: it is what torch
// computes on the GPU for a division by a constant, so rows quantised with
// elementary torch operations have the same scales, bit for bit.)
//
// The floor keeps the scale normal (and 1 / scale finite) for rows of zeros
// and of subnormal numbers.  A row holding an infinity or a NaN gets the scale
// NaN and q = 0, so every product with it is NaN.
//
// The nearest integer is that of the REAL quotient, not of the rounded one, so
// that q does not depend on how v / scale is evaluated: q0 = round(v * (1 /
// scale)) is at most one step off and only next to a tie; r = v - q0 * scale,
// one fused multiply-add, is exact there (r is a multiple of half an ulp of
// scale and at most scale / 2 in magnitude, so it has 24 bits; below scale / 2
// q0 is 0 and r is v), and comparing it with scale / 2, also exact, tells
// whether the neighbour is nearer, or as near and even.
#pragma once

#include "common.cuh"

namespace moe {

constexpr float kQuantScaleFloor = 1.17549435e-38f;  // 2^-126

// amax as raw bits of a non-negative float (NaN above infinity above the rest)
__device__ __forceinline__ float quant_scale(unsigned amax_bits) {
  if (amax_bits >= 0x7F800000u) return __uint_as_float(0x7FC00000u);
  return fmaxf(__uint_as_float(amax_bits) * (1.0f / 127.0f), kQuantScaleFloor);
}

__device__ __forceinline__ unsigned abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// The residual v - q0 * scale is scale / 2 or more away: q0's neighbour is
// nearer, or it is a tie.
static __device__ __noinline__ float quant_border(float q0, float r, float half) {
  const float step = r > 0.f ? 1.0f : -1.0f;
  if (fabsf(r) > half) return q0 + step;
  const bool odd = (static_cast<int>(q0) & 1) != 0;
  return odd ? q0 + step : q0;
}

// Four values to four packed bytes (v[0] lowest).  inv = 1 / scale (any
// rounding); with a NaN scale the bytes are 0.
__device__ __forceinline__ uint32_t quant_pack4(const float (&v)[4], float scale, float inv) {
  constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23: adding it rounds to an integer, ties to even
  const float half = 0.5f * scale;
  float t[4], r[4], worst = 0.f;  // t: the integer plus kMagic, whose low byte is the integer's
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    t[i] = fmaf(v[i], inv, kMagic);
    r[i] = fmaf(-(t[i] - kMagic), scale, v[i]);
    worst = fmaxf(worst, fabsf(r[i]));
  }
  if (worst >= half) {  // next to a tie: rare
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (fabsf(r[i]) >= half) t[i] = quant_border(t[i] - kMagic, r[i], half) + kMagic;
  }
  const uint32_t w = __byte_perm(__byte_perm(__float_as_uint(t[0]), __float_as_uint(t[1]), 0x0040),
                                 __byte_perm(__float_as_uint(t[2]), __float_as_uint(t[3]), 0x0040), 0x5410);
  return scale == scale ? w : 0u;
}

__device__ __forceinline__ unsigned warp_max_u32(unsigned v) { return __reduce_max_sync(0xffffffffu, v); }

// 16 bytes of BF16 or FP32 as floats
__device__ __forceinline__ void unpack16(const uint4& q, float (&v)[8], const __nv_bfloat16*) {
  v[0] = bf16_lo(q.x); v[1] = bf16_hi(q.x); v[2] = bf16_lo(q.y); v[3] = bf16_hi(q.y);
  v[4] = bf16_lo(q.z); v[5] = bf16_hi(q.z); v[6] = bf16_lo(q.w); v[7] = bf16_hi(q.w);
}

}  // namespace moe
