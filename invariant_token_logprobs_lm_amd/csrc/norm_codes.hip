// The norms around a block with the result as E4M3 rows with a scale for each
// 128 columns, the operand of the block-scaled product, with or without dropout
// of the block's output (norm_kernels.h).

#include "norm_kernels.h"

namespace itl {

hipError_t launch_residual_norm_blocks(const void* x, const void* y, const void* gate, long long gate_stride,
                                       const void* w_post, const void* w_pre, int dtype, long long n_rows, int d,
                                       float scale, float eps, const DropoutArgs& drop, void* h, uint8_t* codes,
                                       float* u_scale, float* rstd_pre, float* rstd_post, hipStream_t stream) {
  const NormArgs a{x, y, gate, w_post, w_pre, h, nullptr, codes, u_scale, rstd_pre, rstd_post, n_rows, gate_stride, d, scale,
                   eps, false};
  if (drop.seed) {
    const NormDropArgs with{a, drop};
    if (dtype == 0) run_norm<0, kBlockCodes, true, true>(with, stream);
    else run_norm<1, kBlockCodes, true, true>(with, stream);
  } else {
    if (dtype == 0) run_norm<0, kBlockCodes, false, true>(a, stream);
    else run_norm<1, kBlockCodes, false, true>(a, stream);
  }
  return hipGetLastError();
}

}  // namespace itl
