// Symmetric 8-bit quantisation of a row, shared by the kernels that quantise
// token rows, hidden rows and (at load time) weights.
//
//   scale = max(fl32(max|v| * fl32(1 / 127)), 2^-126)
//   q     = the integer nearest to v / scale, ties to even, in [-127, 127]
//
// (The product with the rounded 1 / 127, not the quotient: it is what torch
// computes on the GPU for a division by a constant, so rows quantised with
// elementary torch operations have the same scales, bit for bit.  The correctly
// rounded quotient differs in the last bit for 4.7% of the maxima; either rule
// rounds every element to within half a step.)
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

// Two FP32 operations in one instruction, each rounded as the scalar one is.
__device__ __forceinline__ uint64_t pair2(float a, float b) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ void unpair2(uint64_t p, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Four values to four packed bytes (v[0] lowest).  inv = 1 / scale (any
// rounding); with a NaN scale the bytes are 0.
__device__ __forceinline__ uint32_t quant_pack4(const float (&v)[4], float scale, float inv) {
  constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23: adding it rounds to an integer, ties to even
  const float half = 0.5f * scale;
  float t[4], r[4];  // t: the integer plus kMagic, whose low byte is the integer's
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    const uint64_t x = pair2(v[i], v[i + 1]);
    const uint64_t n = fma2(x, pair2(inv, inv), pair2(kMagic, kMagic));
    unpair2(n, t[i], t[i + 1]);
    unpair2(fma2(add2(n, pair2(-kMagic, -kMagic)), pair2(-scale, -scale), x), r[i], r[i + 1]);
  }
  const float worst = fmaxf(fmaxf(fabsf(r[0]), fabsf(r[1])), fmaxf(fabsf(r[2]), fabsf(r[3])));
  // Next to a tie (one BF16 value in 900: half of the row's maximum is one): q0's
  // neighbour is nearer when |r| > half, and even when |r| = half and q0 is odd;
  // in one comparison of the bits, |r| + odd > half.  (Some lane of a warp is here
  // for every eighth group of four, so no branch by element and no call: those cost
  // 12 of the 73 us of 65536 rows of 2048 BF16 and 5 of the 8 us of 600.)
  if (worst >= half) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t n = __float_as_uint(t[i]);
      const uint32_t rb = __float_as_uint(r[i]);
      if ((rb & 0x7FFFFFFFu) + (n & 1u) > __float_as_uint(half)) n += (static_cast<int>(rb) >> 31) | 1;
      t[i] = __uint_as_float(n);
    }
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
