// Element access and roundings shared by the learner's kernels (norms, cross
// entropy, optimizer step).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"
#include "itl_config.h"

namespace itl {

// A grid dimension holds less than 2^32 threads: a launch of more (a wavefront
// for each of 2^26 rows) wraps without an error and leaves the rest undone.
// flat_grid lays any number of workgroups out in rows of at most 2^20, flat_group
// is a workgroup's number; fewer than there are rows lie past the end.
inline dim3 flat_grid(long long groups) {
  const long long y = (groups + (1LL << 20) - 1) >> 20;
  return dim3((unsigned)((groups + y - 1) / y), (unsigned)y);
}
__device__ __forceinline__ long long flat_group() { return (long long)blockIdx.y * gridDim.x + blockIdx.x; }

template <int kDtype>
struct Elem;

template <>
struct Elem<0> {
  using T = uint16_t;  // bf16 bits
  static constexpr int kSize = 2;
  __device__ static __forceinline__ float to_f(T x) { return __uint_as_float((uint32_t)x << 16); }
  // Round to nearest even; a NaN stays a (quiet) NaN, an overflow is infinite.
  __device__ static __forceinline__ T from_f(float f) { return __builtin_bit_cast(T, (__bf16)f); }
};

template <>
struct Elem<1> {
  using T = float;
  static constexpr int kSize = 4;
  __device__ static __forceinline__ float to_f(T x) { return x; }
  __device__ static __forceinline__ T from_f(float f) { return f; }
};

// E4M3 code of |x| <= 448 (up to the rounding of a quotient by amax / 448),
// to nearest even, subnormals included, by the conversion instruction
// (gfx950 converts to the OCP format: the codes of all roundings are tested
// against the format's definition).
__device__ __forceinline__ uint32_t e4m3_code(float x) {
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x, x, 0, false) & 0xffu;
}

// Scale of values of at most amax: amax / 448, but no smaller than the least
// normal number. A subnormal scale has few bits left or is 0, and quotients by
// it pass the format's range or are 0 / 0: codes of NaN.
__device__ __forceinline__ float e4m3_scale(float amax) {
  return amax > 0.0f ? fmaxf(__fdiv_rn(amax, 448.0f), 0x1p-126f) : 1.0f;
}

// Four codes, the first in the low byte.
__device__ __forceinline__ uint32_t e4m3_code4(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
  return (uint32_t)w;
}

__device__ __forceinline__ float e4m3_value(uint32_t code) { return __builtin_amdgcn_cvt_f32_fp8((int)code, 0); }

// wave_sum's butterfly (the same additions, so the same bits) with its steps
// within 16 lanes as register moves between lanes instead of LDS permutes:
// after the steps over lanes 1 and 2 apart a quad's lanes hold one value, so
// mirroring 8 lanes is the step 4 apart; then mirroring 16 the step 8 apart.
template <int kControl>
__device__ __forceinline__ float lane_move(float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), kControl, 0xf, 0xf, true));
}
__device__ __forceinline__ float wave_sum_moves(float x) {
  x += lane_move<0xB1>(x);   // lanes 1, 0, 3, 2 of each quad
  x += lane_move<0x4E>(x);   // lanes 2, 3, 0, 1
  x += lane_move<0x141>(x);  // 8 lanes mirrored
  x += lane_move<0x140>(x);  // 16 lanes mirrored
  x += __shfl_xor(x, 16, 64);
  x += __shfl_xor(x, 32, 64);
  return x;
}

}  // namespace itl
