// Dropout from a counter-based generator: whether a value is kept is computed
// where it is needed, in the forward and again in the backward, and no mask is
// stored.
//
// The generator is Philox 4 x 32 with ten rounds (Salmon, Moraes, Dror, Shaw:
// "Parallel random numbers: as easy as 1, 2, 3", 2011): a bijection of a
// 128-bit counter under a 64-bit key, each round two 32 x 32 -> 64 products, the
// key stepped by two Weyl constants. Key: the seed. Counter: (column / 8, row's
// low word, row's high word, site). One call gives eight 16-bit numbers (word 0's
// low half first), those of the eight columns of the group; a value is dropped
// where its number is below `threshold` = p 2^16, so that a keep bit depends on
// (seed, site, row, column) alone, not on the width, the rows around it, the
// launch, or which way the values are read.
//
// 16 bits a value and not 32: half the calls (a call is 20 products of quarter
// rate, about 560 cycles of a SIMD for a wavefront: 42 M values take about 19 us
// of all SIMDs, hidden behind their 30 us of memory); p is kept to 2^-17.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace itl {

struct DropoutArgs {
  const int64_t* seed;  // null: no dropout
  long long first_row;  // the row number of a call's first row
  uint32_t site;
  uint32_t threshold;  // 0 .. 65536: dropped below it
  float scale;         // of kept values: 65536 / (65536 - threshold), 0 if nothing is kept
};

struct DropoutKey {
  uint32_t k0, k1;
};

__device__ __forceinline__ DropoutKey dropout_key(const DropoutArgs& a) {
  const uint64_t s = (uint64_t)*a.seed;
  return DropoutKey{(uint32_t)s, (uint32_t)(s >> 32)};
}

// The eight numbers of a group of columns of a row.
__device__ __forceinline__ uint4 dropout_numbers(const DropoutArgs& a, DropoutKey key, uint32_t group, long long row) {
  uint32_t c0 = group, c1 = (uint32_t)row, c2 = (uint32_t)((uint64_t)row >> 32), c3 = a.site;
  uint32_t k0 = key.k0, k1 = key.k1;
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t p0 = (uint64_t)c0 * 0xD2511F53u, p1 = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = __builtin_amdgcn_bitop3_b32((uint32_t)(p1 >> 32), c1, k0, 0x96);  // all three, exclusive or
    c1 = (uint32_t)p1;
    c2 = __builtin_amdgcn_bitop3_b32((uint32_t)(p0 >> 32), c3, k1, 0x96);
    c3 = (uint32_t)p0;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

// Whether column j of a group is kept.
__device__ __forceinline__ bool dropout_keeps(const uint4& u, int j, uint32_t threshold) {
  const uint32_t w = j < 2 ? u.x : j < 4 ? u.y : j < 6 ? u.z : u.w;
  return ((j & 1) ? w >> 16 : w & 0xffffu) >= threshold;
}

// Whether columns 8 group + j are kept.
struct Kept8 {
  bool at[8];
};
__device__ __forceinline__ Kept8 dropout_kept(const DropoutArgs& a, DropoutKey key, uint32_t group, long long row) {
  const uint4 u = dropout_numbers(a, key, group, row);
  Kept8 k;
#pragma unroll
  for (int j = 0; j < 8; ++j) k.at[j] = dropout_keeps(u, j, a.threshold);
  return k;
}

// Whether columns first + j step + lane of this wavefront are kept (first,
// step: multiples of 8, the same in all lanes; every lane takes part). A column's
// group has eight lanes, and the wavefront's eight columns per lane are 64
// groups: lane l makes one call, for the group of lanes 8 (l / 8) .. + 7 at
// j = l mod 8; ballots over the numbers' places then hand each lane its byte.
__device__ __forceinline__ Kept8 dropout_kept_across(const DropoutArgs& a, DropoutKey key, uint32_t first, uint32_t step,
                                                     long long row) {
  const uint32_t l = threadIdx.x & 63;
  const uint4 u = dropout_numbers(a, key, (first + (l & 7) * step) / 8 + (l >> 3), row);
  const bool high = l >= 32;
  uint32_t w[8];
#pragma unroll
  for (int b = 0; b < 8; ++b) {  // ballot b: bit 8 g + j is column b of the group of lanes 8 g .. at j
    const uint64_t v = __builtin_amdgcn_ballot_w64(dropout_keeps(u, b, a.threshold));
    w[b] = high ? (uint32_t)(v >> 32) : (uint32_t)v;
  }
  const uint32_t x0 = (l & 1) ? w[1] : w[0], x1 = (l & 1) ? w[3] : w[2];
  const uint32_t x2 = (l & 1) ? w[5] : w[4], x3 = (l & 1) ? w[7] : w[6];
  const uint32_t y0 = (l & 2) ? x1 : x0, y1 = (l & 2) ? x3 : x2;
  const uint32_t bits = ((l & 4) ? y1 : y0) >> (8 * ((l >> 3) & 3));
  Kept8 k;
#pragma unroll
  for (int j = 0; j < 8; ++j) k.at[j] = (bits >> j) & 1;
  return k;
}

// Whether one value is kept (a call for it alone).
__device__ __forceinline__ bool dropout_keeps_one(const DropoutArgs& a, DropoutKey key, uint32_t column, long long row) {
  const uint4 u = dropout_numbers(a, key, column >> 3, row);
  const uint32_t w = (column & 4) ? ((column & 2) ? u.w : u.z) : ((column & 2) ? u.y : u.x);
  return ((column & 1) ? w >> 16 : w & 0xffffu) >= a.threshold;
}

// A value's product with its keep factor: 0 where it is dropped, whatever it is.
__device__ __forceinline__ float dropped(float v, bool keep, float scale) { return keep ? v * scale : 0.0f; }

}  // namespace itl
