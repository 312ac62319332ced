// The norms around a block with dropout of its output (norm_kernels.h).

#include "norm_kernels.h"

namespace itl {

hipError_t launch_residual_norm_dropout(const void* x, const void* y, const void* gate, long long gate_stride,
                                        const void* w_post, const void* w_pre, int dtype, long long n_rows, int d,
                                        float scale, float eps, const DropoutArgs& drop, void* h, void* u, float* rstd_pre,
                                        float* rstd_post, hipStream_t stream) {
  const NormDropArgs a{{x, y, gate, w_post, w_pre, h, u, nullptr, nullptr, rstd_pre, rstd_post, n_rows, gate_stride, d, scale, eps,
                   2 * n_rows * d * (dtype == 0 ? 2 : 4) > kStreamBytes}, drop};
  if (d % 8 == 0) {
    if (dtype == 0) run_norm<0, kOwn, true, true>(a, stream);
    else run_norm<1, kOwn, true, true>(a, stream);
  } else {
    if (dtype == 0) run_norm<0, kOwn, true, false>(a, stream);
    else run_norm<1, kOwn, true, false>(a, stream);
  }
  return hipGetLastError();
}

hipError_t launch_residual_norm_dropout_backward(const void* du, int grad_dtype, const void* dh, const void* h, const void* y,
                                         const void* gate, long long gate_stride, const void* w_post,
                                         const void* w_pre, const float* rstd_pre, const float* rstd_post, int dtype,
                                         long long n_rows, int d, float scale, const DropoutArgs& drop, void* dx, void* dy, void* dgate,
                                         float* dw_pre, float* dw_post, void* workspace, hipStream_t stream) {
  char* ws = static_cast<char*>(workspace);
  const bool shared_gate = gate && gate_stride == 0;
  NormBwdDropArgs a{{du, dh, h, y, gate, w_post, w_pre, rstd_pre, rstd_post, dx, dy, gate && !shared_gate ? dgate : nullptr,
                reinterpret_cast<float*>(ws), reinterpret_cast<float*>(ws + align256((size_t)n_rows * 4)), n_rows,
                gate_stride, d, norm_runs(n_rows, d), scale}, drop};
  if (n_rows > 0) {
    if (dtype == 0) {
      if (grad_dtype == 0) run_norm_backward<0, 0, true>(a, stream);
      else run_norm_backward<0, 1, true>(a, stream);
    } else {
      run_norm_backward<1, 1, true>(a, stream);
    }
  }
  return launch_norm_backward_finish(a.part, a.runs, d, dw_pre, w_post ? dw_post : nullptr,
                                     shared_gate ? static_cast<float*>(dgate) : nullptr, stream);
}

}  // namespace itl
