// The norms around a block, fused with the block's gate and residual scale,
// forward and backward.
//
//   p = y r_post w_post          r_post = (mean y^2 + eps)^-1/2   (w_post absent: p = y)
//   h = x + scale gate p         rounded to the rows' type
//   u = h r_pre w_pre            r_pre = (mean h^2 + eps)^-1/2
//
// u is taken from the kept (rounded) h, so the fused call gives the bits of
// a call that norms a stored h. All arithmetic between loads and stores is
// fp32; h and u are rounded once each, to nearest even. The FP8 form writes
// u as E4M3 codes with a scale per row, amax / 448, straight from the fp32
// u (one rounding, not two).
//
// Backward, with n = h r_pre, q = y r_post and a row mean <.>:
//   dn = du w_pre,  dx = dh + r_pre (dn - n <dn n>)
//   dw_pre = sum_t du n
//   dp = scale gate dx,  dgate = scale p dx (summed over rows for one shared gate)
//   dw_post = sum_t dp q,  dq = dp w_post,  dy = r_post (dq - q <dq q>)
//
// Rows: one workgroup of 256 threads per row; a thread takes columns
// tid, tid + 256, ...; sums go up a fixed tree (thread, wavefront butterfly,
// wavefronts in order), so a row's results depend on the row and its width
// alone. Column sums (dw_pre, dw_post, a shared dgate) are taken over fixed
// runs of rows, then over the runs in order: run-to-run deterministic, no
// atomics.

#include <algorithm>

#include "itl_launch.h"
#include "learner_common.h"

namespace itl {

namespace {

constexpr int kNormThreads = 256;

// Sum over a workgroup of kWaves wavefronts, the same bits in every thread.
template <int kWaves>
__device__ __forceinline__ float block_sum(float x, float* lds) {
  x = wave_sum(x);
  if constexpr (kWaves == 1) return x;
  __syncthreads();  // the previous sum's readers are done
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
  __syncthreads();
  float s = lds[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) s += lds[w];
  return s;
}

template <int kWaves>
__device__ __forceinline__ float block_max(float x, float* lds) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) x = fmaxf(x, __shfl_xor(x, off, 64));
  if constexpr (kWaves == 1) return x;
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
  __syncthreads();
  float s = lds[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) s = fmaxf(s, lds[w]);
  return s;
}

struct NormArgs {
  const void *x, *y, *gate, *w_post, *w_pre;
  void *h, *u;
  uint8_t* codes;
  float *u_scale, *rstd_pre, *rstd_post;
  long long n_rows, gate_stride;
  int d;
  float scale, eps;
};

// Any width: columns one by one, a row's later passes read it again (from
// the caches; h by the thread that wrote it).
template <int kDtype, bool kFp8>
__global__ __launch_bounds__(kNormThreads) void norm_rows_kernel(NormArgs a) {
  using E = Elem<kDtype>;
  using T = typename E::T;
  __shared__ float lds[kNormThreads / 64];
  constexpr int kW = kNormThreads / 64;
  const long long row = blockIdx.x;
  const int d = a.d;
  const size_t base = (size_t)row * d;
  const T* x = static_cast<const T*>(a.x) + base;
  const T* y = a.y ? static_cast<const T*>(a.y) + base : nullptr;
  const T* gate = a.gate ? static_cast<const T*>(a.gate) + (size_t)row * a.gate_stride : nullptr;
  const T* w_post = static_cast<const T*>(a.w_post);
  const T* w_pre = static_cast<const T*>(a.w_pre);
  T* h = y ? static_cast<T*>(a.h) + base : nullptr;
  float r_post = 1.0f;
  if (w_post) {
    float ss = 0.0f;
    for (int k = threadIdx.x; k < d; k += kNormThreads) {
      const float v = E::to_f(y[k]);
      ss += v * v;
    }
    r_post = 1.0f / sqrtf(block_sum<kW>(ss, lds) / (float)d + a.eps);
    if (threadIdx.x == 0 && a.rstd_post) a.rstd_post[row] = r_post;
  }
  float ss = 0.0f;
  for (int k = threadIdx.x; k < d; k += kNormThreads) {
    float v = E::to_f(x[k]);
    if (y) {
      float p = E::to_f(y[k]);
      if (w_post) p = p * r_post * E::to_f(w_post[k]);
      if (gate) p *= E::to_f(gate[k]);
      const T hv = E::from_f(v + a.scale * p);
      h[k] = hv;
      v = E::to_f(hv);
    }
    ss += v * v;
  }
  const float r_pre = 1.0f / sqrtf(block_sum<kW>(ss, lds) / (float)d + a.eps);
  if (threadIdx.x == 0 && a.rstd_pre) a.rstd_pre[row] = r_pre;
  const T* hr = y ? h : x;
  if constexpr (!kFp8) {
    T* u = static_cast<T*>(a.u) + base;
    for (int k = threadIdx.x; k < d; k += kNormThreads) u[k] = E::from_f(E::to_f(hr[k]) * r_pre * E::to_f(w_pre[k]));
  } else {
    float amax = 0.0f;
    for (int k = threadIdx.x; k < d; k += kNormThreads) amax = fmaxf(amax, fabsf(E::to_f(hr[k]) * r_pre * E::to_f(w_pre[k])));
    amax = block_max<kW>(amax, lds);
    const float s = amax > 0.0f ? __fdiv_rn(amax, 448.0f) : 1.0f;
    if (threadIdx.x == 0) a.u_scale[row] = s;
    for (int k = threadIdx.x; k < d; k += kNormThreads)
      a.codes[base + k] = (uint8_t)e4m3_code(__fdiv_rn(E::to_f(hr[k]) * r_pre * E::to_f(w_pre[k]), s));
  }
}

struct NormBwdArgs {
  const void *du, *dh, *h, *y, *gate, *w_post, *w_pre;
  const float *rstd_pre, *rstd_post;
  void *dx, *dy, *dgate_rows;
  float* row_mean;  // <dn n> of every row, for the column sums
  float* part;      // [runs, 3, d] column sums of the runs
  long long n_rows, gate_stride;
  int d, runs;
  float scale;
};

// The rows' part of the backward, any width. means_only: just the rows'
// means, for column sums that are taken before dx is written over dh.
template <int kDtype, int kGrad>
__global__ __launch_bounds__(kNormThreads) void norm_backward_rows_kernel(NormBwdArgs a, bool means_only) {
  using E = Elem<kDtype>;
  using T = typename E::T;
  using EG = Elem<kGrad>;
  using TG = typename EG::T;
  __shared__ float lds[kNormThreads / 64];
  constexpr int kW = kNormThreads / 64;
  const long long row = blockIdx.x;
  const int d = a.d;
  const size_t base = (size_t)row * d;
  const TG* du = static_cast<const TG*>(a.du) + base;
  const T* dh = a.dh ? static_cast<const T*>(a.dh) + base : nullptr;
  const T* h = static_cast<const T*>(a.h) + base;
  const T* y = a.y ? static_cast<const T*>(a.y) + base : nullptr;
  const T* gate = a.gate ? static_cast<const T*>(a.gate) + (size_t)row * a.gate_stride : nullptr;
  const T* w_post = static_cast<const T*>(a.w_post);
  const T* w_pre = static_cast<const T*>(a.w_pre);
  T* dx = static_cast<T*>(a.dx) + base;
  T* dy = y ? static_cast<T*>(a.dy) + base : nullptr;
  T* dgate = a.dgate_rows ? static_cast<T*>(a.dgate_rows) + base : nullptr;
  const float r_pre = a.rstd_pre[row];
  const float r_post = w_post ? a.rstd_post[row] : 1.0f;
  float s = 0.0f;
  for (int k = threadIdx.x; k < d; k += kNormThreads)
    s += (EG::to_f(du[k]) * E::to_f(w_pre[k])) * (E::to_f(h[k]) * r_pre);
  const float c1 = block_sum<kW>(s, lds) / (float)d;
  if (threadIdx.x == 0) a.row_mean[row] = c1;
  if (means_only) return;
  auto grad_h = [&](int k) {
    const float dn = EG::to_f(du[k]) * E::to_f(w_pre[k]);
    const float g = r_pre * (dn - E::to_f(h[k]) * r_pre * c1);
    return dh ? E::to_f(dh[k]) + g : g;
  };
  auto grad_p = [&](int k, float dxv) { return gate ? a.scale * dxv * E::to_f(gate[k]) : a.scale * dxv; };
  s = 0.0f;
  for (int k = threadIdx.x; k < d; k += kNormThreads) {
    const float v = grad_h(k);
    if (w_post) s += (grad_p(k, v) * E::to_f(w_post[k])) * (E::to_f(y[k]) * r_post);
    if (dgate) {
      const float p = w_post ? E::to_f(y[k]) * r_post * E::to_f(w_post[k]) : E::to_f(y[k]);
      dgate[k] = E::from_f(a.scale * p * v);
    }
    if (!w_post && y) dy[k] = E::from_f(grad_p(k, v));
    if (!w_post) dx[k] = E::from_f(v);
  }
  if (!w_post) return;
  const float c2 = block_sum<kW>(s, lds) / (float)d;
  for (int k = threadIdx.x; k < d; k += kNormThreads) {
    const float v = grad_h(k);
    const float dq = grad_p(k, v) * E::to_f(w_post[k]);
    dy[k] = E::from_f(r_post * (dq - E::to_f(y[k]) * r_post * c2));
    dx[k] = E::from_f(v);
  }
}

// Column sums over run blockIdx.y of the rows, 64 columns per workgroup, four
// rows at a time (lanes of four wavefronts, added in order at the end).
template <int kDtype, int kGrad>
__global__ __launch_bounds__(kNormThreads) void norm_backward_columns_kernel(NormBwdArgs a) {
  using E = Elem<kDtype>;
  using T = typename E::T;
  using EG = Elem<kGrad>;
  using TG = typename EG::T;
  __shared__ float lds[3][4][64];
  const int d = a.d;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int k = blockIdx.x * 64 + lane;
  const long long r0 = a.n_rows * blockIdx.y / a.runs, r1 = a.n_rows * (blockIdx.y + 1) / a.runs;
  float s_pre = 0.0f, s_post = 0.0f, s_gate = 0.0f;
  if (k < d) {
    const float w_pre = E::to_f(static_cast<const T*>(a.w_pre)[k]);
    const float w_post = a.w_post ? E::to_f(static_cast<const T*>(a.w_post)[k]) : 1.0f;
    const T* gate = static_cast<const T*>(a.gate);
    for (long long row = r0 + wave; row < r1; row += 4) {
      const size_t at = (size_t)row * d + k;
      const float r_pre = a.rstd_pre[row];
      const float g = EG::to_f(static_cast<const TG*>(a.du)[at]);
      const float hn = E::to_f(static_cast<const T*>(a.h)[at]) * r_pre;
      s_pre += g * hn;
      if (!a.y) continue;
      float v = r_pre * (g * w_pre - hn * a.row_mean[row]);
      if (a.dh) v = E::to_f(static_cast<const T*>(a.dh)[at]) + v;
      float q = E::to_f(static_cast<const T*>(a.y)[at]);
      if (a.w_post) q *= a.rstd_post[row];
      float dp = a.scale * v;
      if (gate) {
        s_gate += a.scale * (a.w_post ? q * w_post : q) * v;
        dp *= E::to_f(gate[(size_t)row * a.gate_stride + k]);
      }
      if (a.w_post) s_post += dp * q;
    }
  }
  lds[0][wave][lane] = s_pre;
  lds[1][wave][lane] = s_post;
  lds[2][wave][lane] = s_gate;
  __syncthreads();
  if (wave < 3 && k < d) {
    const float* c = &lds[wave][0][lane];
    a.part[((size_t)blockIdx.y * 3 + wave) * d + k] = ((c[0] + c[64]) + c[128]) + c[192];
  }
}

// The runs' sums in order: thread (column, which of the three).
__global__ __launch_bounds__(256) void norm_backward_finish_kernel(const float* __restrict__ part, int runs, int d,
                                                                   float* __restrict__ dw_pre,
                                                                   float* __restrict__ dw_post,
                                                                   float* __restrict__ dgate) {
  const int k = blockIdx.x * 256 + threadIdx.x;
  float* out = blockIdx.y == 0 ? dw_pre : blockIdx.y == 1 ? dw_post : dgate;
  if (k >= d || !out) return;
  float s = 0.0f;
  for (int r = 0; r < runs; ++r) s += part[((size_t)r * 3 + blockIdx.y) * d + k];
  out[k] = s;
}

// Runs of rows of the column sums: about 64 rows each, at most 256.
int norm_runs(long long n_rows) { return (int)std::min<long long>(256, ceil_div(n_rows, 64)); }

}  // namespace

size_t norm_backward_workspace_bytes(long long n_rows, long long d) {
  return align256((size_t)n_rows * 4) + align256((size_t)norm_runs(n_rows) * 3 * (size_t)d * 4);
}

hipError_t launch_residual_norm(const void* x, const void* y, const void* gate, long long gate_stride,
                                const void* w_post, const void* w_pre, int dtype, long long n_rows, int d, float scale,
                                float eps, void* h, void* u, uint8_t* codes, float* u_scale, float* rstd_pre,
                                float* rstd_post, hipStream_t stream) {
  const NormArgs a{x, y, gate, w_post, w_pre, h, u, codes, u_scale, rstd_pre, rstd_post, n_rows, gate_stride, d, scale, eps};
  const dim3 grid((unsigned)n_rows), block(kNormThreads);
  if (codes) {
    if (dtype == 0) hipLaunchKernelGGL((norm_rows_kernel<0, true>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((norm_rows_kernel<1, true>), grid, block, 0, stream, a);
  } else {
    if (dtype == 0) hipLaunchKernelGGL((norm_rows_kernel<0, false>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((norm_rows_kernel<1, false>), grid, block, 0, stream, a);
  }
  return hipGetLastError();
}

namespace {

template <int kDtype, int kGrad>
void run_norm_backward(const NormBwdArgs& a, hipStream_t stream) {
  const dim3 rows((unsigned)a.n_rows), columns((unsigned)ceil_div(a.d, 64), (unsigned)a.runs), block(kNormThreads);
  const bool over = a.dx == a.dh;
  hipLaunchKernelGGL((norm_backward_rows_kernel<kDtype, kGrad>), rows, block, 0, stream, a, over);
  hipLaunchKernelGGL((norm_backward_columns_kernel<kDtype, kGrad>), columns, block, 0, stream, a);
  if (over) hipLaunchKernelGGL((norm_backward_rows_kernel<kDtype, kGrad>), rows, block, 0, stream, a, false);
}

}  // namespace

hipError_t launch_residual_norm_backward(const void* du, int grad_dtype, const void* dh, const void* h, const void* y,
                                         const void* gate, long long gate_stride, const void* w_post,
                                         const void* w_pre, const float* rstd_pre, const float* rstd_post, int dtype,
                                         long long n_rows, int d, float scale, void* dx, void* dy, void* dgate,
                                         float* dw_pre, float* dw_post, void* workspace, hipStream_t stream) {
  char* ws = static_cast<char*>(workspace);
  const bool shared_gate = gate && gate_stride == 0;
  NormBwdArgs a{du, dh, h, y, gate, w_post, w_pre, rstd_pre, rstd_post, dx, dy, gate && !shared_gate ? dgate : nullptr,
                reinterpret_cast<float*>(ws), reinterpret_cast<float*>(ws + align256((size_t)n_rows * 4)), n_rows,
                gate_stride, d, norm_runs(n_rows), scale};
  if (n_rows > 0) {
    if (dtype == 0) {
      if (grad_dtype == 0) run_norm_backward<0, 0>(a, stream);
      else run_norm_backward<0, 1>(a, stream);
    } else {
      run_norm_backward<1, 1>(a, stream);
    }
  }
  hipLaunchKernelGGL(norm_backward_finish_kernel, dim3((unsigned)ceil_div(d, 256), 3), dim3(256), 0, stream, a.part,
                     a.runs, d, dw_pre, w_post ? dw_post : nullptr, shared_gate ? static_cast<float*>(dgate) : nullptr);
  return hipGetLastError();
}

}  // namespace itl
