// The norms around a block without dropout (norm_kernels.h says how), and what
// their backwards share.

#include "norm_kernels.h"

namespace itl {

namespace {

// The runs' sums: 64 columns of one of the three sums per workgroup, its 16
// wavefronts over runs w, w + 16, ... in order, then the wavefronts in order.
constexpr int kFinishWaves = 16;
__global__ __launch_bounds__(64 * kFinishWaves) void norm_backward_finish_kernel(const float* __restrict__ part, int runs,
                                                                                 int d, float* __restrict__ dw_pre,
                                                                                 float* __restrict__ dw_post,
                                                                                 float* __restrict__ dgate) {
  __shared__ float lds[kFinishWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int k = blockIdx.x * 64 + lane;
  float* out = blockIdx.y == 0 ? dw_pre : blockIdx.y == 1 ? dw_post : dgate;
  if (!out) return;
  float s = 0.0f;
  if (k < d) {
#pragma unroll 8
    for (int r = wave; r < runs; r += kFinishWaves) s += part[((size_t)r * 3 + blockIdx.y) * d + k];
  }
  lds[wave][lane] = s;
  __syncthreads();
  if (wave != 0 || k >= d) return;
  for (int w = 1; w < kFinishWaves; ++w) s += lds[w][lane];
  out[k] = s;
}

}  // namespace

hipError_t launch_norm_backward_finish(const float* part, int runs, int d, float* dw_pre, float* dw_post, float* dgate,
                                       hipStream_t stream) {
  hipLaunchKernelGGL(norm_backward_finish_kernel, dim3((unsigned)ceil_div(d, 64), 3), dim3(64 * kFinishWaves), 0, stream, part,
                     runs, d, dw_pre, dw_post, dgate);
  return hipGetLastError();
}

size_t norm_backward_workspace_bytes(long long n_rows, long long d) {
  return align256((size_t)n_rows * 4) + align256((size_t)norm_runs(n_rows, d) * 3 * (size_t)d * 4);
}

hipError_t launch_residual_norm(const void* x, const void* y, const void* gate, long long gate_stride,
                                const void* w_post, const void* w_pre, int dtype, long long n_rows, int d, float scale,
                                float eps, void* h, void* u, uint8_t* codes, float* u_scale, float* rstd_pre,
                                float* rstd_post, hipStream_t stream) {
  const NormArgs a{x, y, gate, w_post, w_pre, h, u, codes, u_scale, rstd_pre, rstd_post, n_rows, gate_stride, d, scale, eps,
                   2 * n_rows * d * (dtype == 0 ? 2 : 4) > kStreamBytes};
  if (codes) {
    if (dtype == 0) run_norm<0, kRowCodes, false, true>(a, stream);
    else run_norm<1, kRowCodes, false, true>(a, stream);
  } else if (d % 8 == 0) {
    if (dtype == 0) run_norm<0, kOwn, false, true>(a, stream);
    else run_norm<1, kOwn, false, true>(a, stream);
  } else {
    if (dtype == 0) run_norm<0, kOwn, false, false>(a, stream);
    else run_norm<1, kOwn, false, false>(a, stream);
  }
  return hipGetLastError();
}

hipError_t launch_residual_norm_backward(const void* du, int grad_dtype, const void* dh, const void* h, const void* y,
                                         const void* gate, long long gate_stride, const void* w_post,
                                         const void* w_pre, const float* rstd_pre, const float* rstd_post, int dtype,
                                         long long n_rows, int d, float scale, void* dx, void* dy, void* dgate,
                                         float* dw_pre, float* dw_post, void* workspace, hipStream_t stream) {
  char* ws = static_cast<char*>(workspace);
  const bool shared_gate = gate && gate_stride == 0;
  NormBwdArgs a{du, dh, h, y, gate, w_post, w_pre, rstd_pre, rstd_post, dx, dy, gate && !shared_gate ? dgate : nullptr,
                reinterpret_cast<float*>(ws), reinterpret_cast<float*>(ws + align256((size_t)n_rows * 4)), n_rows,
                gate_stride, d, norm_runs(n_rows, d), scale};
  if (n_rows > 0) {
    if (dtype == 0) {
      if (grad_dtype == 0) run_norm_backward<0, 0, false>(a, stream);
      else run_norm_backward<0, 1, false>(a, stream);
    } else {
      run_norm_backward<1, 1, false>(a, stream);
    }
  }
  return launch_norm_backward_finish(a.part, a.runs, d, dw_pre, w_post ? dw_post : nullptr,
                                     shared_gate ? static_cast<float*>(dgate) : nullptr, stream);
}

}  // namespace itl
