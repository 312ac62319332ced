// y = x keep / (1 - p) over rows, and the same again for its gradient: the
// generator, its counter and its key are dropout.h's.
//
// Bound by memory: every value is read and written once; 16384 x 2560 bf16 26 to
// 31 us (5.4 to 6.5 TB/s), 777 x 1001 fp32 5, launch and latency.

#include <algorithm>

#include "dropout.h"
#include "itl_launch.h"
#include "learner_common.h"

namespace itl {

namespace {

constexpr int kDropThreads = 256;
constexpr int kDropGroups = 4;  // groups of 8 columns per thread, all read before the first is dealt with

// A quotient by a number that a launch fixes, of dividends below 2^31
// (Granlund and Montgomery: division by invariant integers, 1994).
struct Divisor {
  uint32_t d, m, shift;
  __device__ __forceinline__ uint32_t quotient(uint32_t x) const { return (__umulhi(x, m) + x) >> shift; }
};

Divisor divisor(uint32_t d) {
  uint32_t shift = 0;
  while ((1u << shift) < d) ++shift;
  return Divisor{d, (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << shift) - d)) / d + 1), shift};
}

struct DropoutCall {
  const void* x;
  void* y;
  long long n_rows;
  int d;
  long long part_rows;  // rows of a part of the grid (blockIdx.y)
  Divisor per_row;      // groups of 8 columns, the last one of a row with what is left
  DropoutArgs drop;
};

// Widths of a multiple of 8 (16384 x 2560 bf16 28 us, 38 by the kernel below).
template <int kDtype>
__global__ __launch_bounds__(kDropThreads) void dropout_kernel(DropoutCall a) {
  using E = Elem<kDtype>;
  constexpr int kVecs = E::kSize / 2;
  const long long row0 = blockIdx.y * a.part_rows;
  const uint32_t n = (uint32_t)min(a.part_rows, a.n_rows - row0) * a.per_row.d;
  const uint32_t at = blockIdx.x * (uint32_t)(kDropThreads * kDropGroups) + threadIdx.x;
  const uint4* x = reinterpret_cast<const uint4*>(a.x) + (size_t)row0 * a.per_row.d * kVecs;
  uint4* y = reinterpret_cast<uint4*>(a.y) + (size_t)row0 * a.per_row.d * kVecs;
  const DropoutKey key = dropout_key(a.drop);
  uint4 v[kDropGroups][kVecs];
#pragma unroll
  for (int g = 0; g < kDropGroups; ++g)
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
      if (at + g * kDropThreads < n) v[g][i] = x[(size_t)(at + g * kDropThreads) * kVecs + i];
#pragma unroll
  for (int g = 0; g < kDropGroups; ++g) {
    const uint32_t f = at + g * kDropThreads;
    if (f >= n) break;
    const uint32_t row = a.per_row.quotient(f);
    const uint4 u = dropout_numbers(a.drop, key, f - row * a.per_row.d, a.drop.first_row + row0 + row);
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      uint32_t w[4] = {v[g][i].x, v[g][i].y, v[g][i].z, v[g][i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if constexpr (kDtype == 0) {
          const float lo = dropped(__uint_as_float(w[k] << 16), dropout_keeps(u, 2 * k, a.drop.threshold), a.drop.scale);
          const float hi = dropped(__uint_as_float(w[k] & 0xffff0000u), dropout_keeps(u, 2 * k + 1, a.drop.threshold), a.drop.scale);
          w[k] = (uint32_t)E::from_f(lo) | ((uint32_t)E::from_f(hi) << 16);
        } else {
          w[k] = __float_as_uint(dropped(__uint_as_float(w[k]), dropout_keeps(u, 4 * i + k, a.drop.threshold), a.drop.scale));
        }
      }
      y[(size_t)f * kVecs + i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// Any width: loads and stores are 16 bytes wide, wherever a row starts (10000 x 2999
// bf16 28 us from the caches, 36 element by element; 32 from memory, 3.8 TB/s).
template <int kDtype>
__global__ __launch_bounds__(kDropThreads) void dropout_any_kernel(DropoutCall a) {
  using E = Elem<kDtype>;
  using T = typename E::T;
  const long long row0 = blockIdx.y * a.part_rows;
  const uint32_t n = (uint32_t)min(a.part_rows, a.n_rows - row0) * a.per_row.d;
  const uint32_t at = blockIdx.x * (uint32_t)(kDropThreads * kDropGroups) + threadIdx.x;
  const T* x = static_cast<const T*>(a.x) + (size_t)row0 * a.d;
  T* y = static_cast<T*>(a.y) + (size_t)row0 * a.d;
  const DropoutKey key = dropout_key(a.drop);
  T v[kDropGroups][8];
  uint32_t row[kDropGroups], group[kDropGroups];
#pragma unroll
  for (int g = 0; g < kDropGroups; ++g) {
    const uint32_t f = at + g * kDropThreads;
    row[g] = a.per_row.quotient(f);
    group[g] = f - row[g] * a.per_row.d;
    const T* p = x + (size_t)row[g] * a.d + 8 * group[g];
    const int left = f >= n ? 0 : a.d - 8 * (int)group[g];
    if (left >= 8) {
      __builtin_memcpy(v[g], p, sizeof v[g]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[g][j] = j < left ? p[j] : T(0);
    }
  }
#pragma unroll
  for (int g = 0; g < kDropGroups; ++g) {
    const uint32_t f = at + g * kDropThreads;
    const int left = f >= n ? 0 : a.d - 8 * (int)group[g];
    if (left <= 0) break;
    const Kept8 kept = dropout_kept(a.drop, key, group[g], a.drop.first_row + row0 + row[g]);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[g][j] = E::from_f(dropped(E::to_f(v[g][j]), kept.at[j], a.drop.scale));
    T* p = y + (size_t)row[g] * a.d + 8 * group[g];
    if (left >= 8) {
      __builtin_memcpy(p, v[g], sizeof v[g]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < left) p[j] = v[g][j];
    }
  }
}

}  // namespace

hipError_t launch_dropout(const void* x, int dtype, long long n_rows, int d, const DropoutArgs& drop, void* y,
                          hipStream_t stream) {
  const uint32_t per_row = (uint32_t)ceil_div(d, 8);
  DropoutCall a{x, y, n_rows, d, std::min<long long>(n_rows, ((1LL << 31) - 1) / per_row), divisor(per_row), drop};
  const dim3 block(kDropThreads), grid((unsigned)ceil_div(a.part_rows * per_row, kDropThreads * kDropGroups),
                                       (unsigned)ceil_div(n_rows, a.part_rows));
  if (d % 8 == 0) {
    if (dtype == 0) hipLaunchKernelGGL((dropout_kernel<0>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((dropout_kernel<1>), grid, block, 0, stream, a);
  } else {
    if (dtype == 0) hipLaunchKernelGGL((dropout_any_kernel<0>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((dropout_any_kernel<1>), grid, block, 0, stream, a);
  }
  return hipGetLastError();
}

}  // namespace itl
