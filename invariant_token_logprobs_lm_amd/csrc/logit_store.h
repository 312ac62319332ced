// Writing a tile's logits from the accumulators of the 16 x 16 engines.
#pragma once

#include <stdint.h>

#include "device_common.h"

namespace itl {

// Kept logits are written with buffer stores against a range that ends at
// the wavefront's last valid token row, so rows past n_tok are dropped by
// the hardware instead of a branch. LogitRows: the range (SGPRs) and this
// lane's row offset in bytes, (c16 * ld + 4 quad) * 4 (ld * 4 * 128 < 2^32).
struct LogitRows {
  __amdgpu_buffer_rsrc_t rsrc;
  uint32_t voff;
  uint32_t bn_stride;  // bytes between the token columns of blocks bn and bn + 1 (16 rows)
};

// Built in each epilogue, not once per kernel: kept live across the K loop,
// these registers would push the loop's operands into scratch. The empty asm
// makes the inputs opaque, so the compiler cannot hoist the build out of
// the tile loop.
__device__ __forceinline__ LogitRows logit_rows(float* logits, long long ld, int tok_first, int n_rows, int n_tok,
                                                int c16, int quad) {
  asm volatile("" : "+s"(tok_first));
  LogitRows r;
  const int valid = max(0, min(n_rows, n_tok - tok_first));
  // Raw buffer (stride 0), 32-bit data format: the same descriptor word 3 as
  // the engine's operand loads. The fields are wave-uniform by construction;
  // readfirstlane tells the compiler so (a descriptor it takes for divergent
  // would turn every store into a loop over the lanes' distinct values).
  const uint64_t base = reinterpret_cast<uint64_t>(logits + (size_t)tok_first * (size_t)ld);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)base);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(base >> 32));
  const int nbytes = __builtin_amdgcn_readfirstlane((int)((uint32_t)valid * (uint32_t)ld * 4u));
  r.rsrc = __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(((uint64_t)hi << 32) | lo), 0, nbytes,
                                             0x00020000);
  r.voff = ((uint32_t)c16 * (uint32_t)ld + 4u * (uint32_t)quad) * 4u;
  r.bn_stride = __builtin_amdgcn_readfirstlane(16u * (uint32_t)ld * 4u);
  return r;
}

// Write this lane's 4 logits of a 16 x 16 block: token column bn of the
// rows, vocabulary rows v0 + 4 quad + r (r < 4) from register r (v0 = the
// block's first row, the same for the whole wavefront): 16 contiguous bytes
// of the token's row. In the vocabulary's last tile, rows at or past the
// vocabulary are not written.
template <class kPartial>
__device__ __forceinline__ void store_logits(const LogitRows& rows, int bn, int v0, int quad, int vocab,
                                             const floatx4& z, kPartial) {
  const uint32_t voff = rows.voff + (uint32_t)bn * rows.bn_stride;
  const uint32_t so = (uint32_t)v0 * 4u;
  if constexpr (!kPartial::value) {
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(int4v, z), rows.rsrc, voff, so, kLogitStorePolicy);
  } else {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (v0 + 4 * quad + r < vocab)
        __builtin_amdgcn_raw_buffer_store_b32((int)__float_as_uint(z[r]), rows.rsrc, voff + 4u * r, so,
                                              kLogitStorePolicy);
  }
}

}  // namespace itl
