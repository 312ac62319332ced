// E4M3 codes of values that share a scale per block of 128: what the quantisers and
// the norms that write such codes have in common.
#pragma once

#include "learner_common.h"

namespace itl {

constexpr int kCodeBlock = 128;

// Largest of 16 lanes, the same in all of them.
__device__ __forceinline__ float largest16(float x) {
  x = fmaxf(x, lane_move<0xB1>(x));   // as wave_sum_moves: lanes 1 apart, 2, then 8 and 16 mirrored
  x = fmaxf(x, lane_move<0x4E>(x));
  x = fmaxf(x, lane_move<0x141>(x));
  return fmaxf(x, lane_move<0x140>(x));
}

__device__ __forceinline__ float largest8(const float (&v)[8]) {
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v[j]));
  return m;
}

// Quotients by one scale, correctly rounded as a division is, at five instructions
// each instead of about ten: with r the correctly rounded reciprocal, x r corrected
// once is within an ulp of x / s, and corrected once more it is the nearest
// (Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990). The remainders must not underflow: below 2^-80 (blocks of values
// below 2^-71) the division is used.
struct Quotient {
  float s, r;
  __device__ __forceinline__ explicit Quotient(float scale) : s(scale), r(__fdiv_rn(1.0f, scale)) {}
  __device__ __forceinline__ bool plain() const { return s >= 0x1p-80f; }
  __device__ __forceinline__ float of(float x) const {
    float q = x * r;
    q = __builtin_fmaf(-__builtin_fmaf(s, q, -x), r, q);  // (a remainder of -0: -0 stays -0)
    return __builtin_fmaf(-__builtin_fmaf(s, q, -x), r, q);
  }
};

// Codes of eight values, the first in the low byte.
__device__ __forceinline__ uint2 codes8(const float (&v)[8], const Quotient& by) {
  float q[8];
  if (by.plain()) {
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = by.of(v[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = __fdiv_rn(v[j], by.s);
  }
  return make_uint2(e4m3_code4(q[0], q[1], q[2], q[3]), e4m3_code4(q[4], q[5], q[6], q[7]));
}

}  // namespace itl
