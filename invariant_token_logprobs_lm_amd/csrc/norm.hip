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
// u as E4M3 codes with a scale per row, amax / 448 (no less than 2^-126),
// straight from the fp32 u (one rounding, not two).
//
// Backward, with n = h r_pre, q = y r_post and a row mean <.>:
//   dn = du w_pre,  dx = dh + r_pre (dn - n <dn n>)
//   dw_pre = sum_t du n
//   dp = scale gate dx,  dgate = scale p dx (summed over rows for one shared gate)
//   dw_post = sum_t dp q,  dq = dp w_post,  dy = r_post (dq - q <dq q>)
//
// Rows of up to kNormMaxWidth values are held in registers: read once,
// written once. A row belongs to one wavefront (up to kWaveWidth values) or
// to a workgroup of four; a thread holds groups of 8 values, consecutive ones
// (16-byte loads) where the width is a multiple of 8, else ones a row of
// threads apart (whole lines per wavefront still). Wider rows are walked by
// norm_rows_kernel, which reads them again for each pass. Sums go up a fixed
// tree (thread, wavefront butterfly, wavefronts in order) chosen by the width
// alone, so a row's results depend on the row and its width alone.
//
// The backward needs two means per row, the second of values that hold the
// first; written out, <dq q> = <s (dh + r_pre dn)> - <dn n> <s r_pre n> with
// s = scale gate w_post q, so three sums in one go give both. A thread keeps
// the column sums (dw_pre, dw_post, a shared dgate) of its columns over all
// rows of its workgroup in registers; the workgroups' sums are then added in
// order: run-to-run deterministic, no atomics.
//
// Bound by memory: 16384 x 2560 bf16 with a post norm and a gate 64 to 71 us
// forward (336 MB, 4.7 to 5.2 TB/s), 137 to 150 us backward (fp32 du; 590 MB,
// 3.9 to 4.3 TB/s); 4096 x 7168 to E4M3 rows 39 to 44 us. One decode token
// takes 4.2 us, launch and latency.

#include <algorithm>

#include "itl_launch.h"
#include "learner_common.h"

namespace itl {

namespace {

constexpr int kNormThreads = 256;

// Sum over a workgroup of kWaves wavefronts, the same bits in every thread.
template <int kWaves>
__device__ __forceinline__ float block_sum(float x, float* lds) {
  x = wave_sum_moves(x);
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
  bool stream;
};

// ---- rows in registers

// Eight columns of a thread: group c of a row of T threads. Whole vectors:
// columns 8 (c T + lane) .. + 7; else c 8 T + j T + lane.
template <bool kVec>
struct Columns {
  int d, T, lane;
  __device__ __forceinline__ int at(int c, int j) const { return kVec ? 8 * (c * T + lane) + j : (8 * c + j) * T + lane; }
};

// Group c as it lies in memory (zeros past the row), and its values.
template <int kDtype, bool kVec>
struct Group {
  using E = Elem<kDtype>;
  using T = typename E::T;
  uint32_t w[kVec ? 2 * E::kSize : 8];

  __device__ __forceinline__ void load(const void* row, const Columns<kVec>& k, int c) {
    if constexpr (kVec) {
      const int at = k.at(c, 0);
#pragma unroll
      for (int i = 0; i < E::kSize / 2; ++i) {
        const uint4 v = at < k.d ? reinterpret_cast<const uint4*>(static_cast<const T*>(row) + at)[i]
                                 : make_uint4(0u, 0u, 0u, 0u);
        w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int at = k.at(c, j);
        const T v = at < k.d ? static_cast<const T*>(row)[at] : T(0);
        if constexpr (kDtype == 0) w[j] = v;
        else w[j] = __float_as_uint(v);
      }
    }
  }
  __device__ __forceinline__ float operator[](int j) const {
    if constexpr (kDtype == 1) return __uint_as_float(w[j]);
    else if constexpr (kVec) return __uint_as_float((j & 1) ? (w[j >> 1] & 0xffff0000u) : (w[j >> 1] << 16));
    else return __uint_as_float(w[j] << 16);
  }
};

template <int kDtype, bool kVec>
__device__ __forceinline__ void load_group(const void* row, const Columns<kVec>& k, int c, float (&v)[8]) {
  Group<kDtype, kVec> g;
  g.load(row, k, c);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = g[j];
}

// Stores group c rounded to the type; v becomes the stored values. kStream:
// past the caches (see kStreamBytes).
template <int kDtype, bool kStream = false, bool kVec>
__device__ __forceinline__ void store_group(void* row, const Columns<kVec>& k, int c, float (&v)[8]) {
  using E = Elem<kDtype>;
  using T = typename E::T;
  if constexpr (kDtype == 0 && kVec) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      w[j] = (uint32_t)E::from_f(v[2 * j]) | ((uint32_t)E::from_f(v[2 * j + 1]) << 16);
      v[2 * j] = __uint_as_float(w[j] << 16);
      v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
    const int at = k.at(c, 0);
    if constexpr (kStream) {
      const int4v o = {(int)w[0], (int)w[1], (int)w[2], (int)w[3]};
      if (at < k.d) __builtin_nontemporal_store(o, reinterpret_cast<int4v*>(static_cast<T*>(row) + at));
    } else {
      if (at < k.d) *reinterpret_cast<uint4*>(static_cast<T*>(row) + at) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  } else if constexpr (kVec) {
    const int at = k.at(c, 0);
    if (at < k.d) {
      if constexpr (kStream) {
        floatx4* o = reinterpret_cast<floatx4*>(static_cast<float*>(row) + at);
        __builtin_nontemporal_store(floatx4{v[0], v[1], v[2], v[3]}, o);
        __builtin_nontemporal_store(floatx4{v[4], v[5], v[6], v[7]}, o + 1);
      } else {
        float4* o = reinterpret_cast<float4*>(static_cast<float*>(row) + at);
        o[0] = make_float4(v[0], v[1], v[2], v[3]);
        o[1] = make_float4(v[4], v[5], v[6], v[7]);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const T s = E::from_f(v[j]);
      v[j] = E::to_f(s);
      const int at = k.at(c, j);
      if (at < k.d) static_cast<T*>(row)[at] = s;
    }
  }
}

// One row per kWaves wavefronts, kGroups groups of 8 values per thread.
template <int kDtype, bool kFp8, bool kVec, bool kStream, int kWaves, int kGroups>
__global__ __launch_bounds__(kNormThreads) void norm_held_kernel(NormArgs a) {
  using T = typename Elem<kDtype>::T;
  __shared__ float lds[kWaves];
  const long long row = kWaves == 1 ? flat_group() * (kNormThreads / 64) + (threadIdx.x >> 6) : flat_group();
  if (row >= a.n_rows) return;  // (whole wavefronts where one is alone, else whole workgroups)
  const Columns<kVec> k{a.d, 64 * kWaves, kWaves == 1 ? (int)(threadIdx.x & 63) : (int)threadIdx.x};
  const size_t base = (size_t)row * a.d;
  const float inv_d = (float)a.d;
  float x[kGroups][8], y[kGroups][8];
#pragma unroll
  for (int c = 0; c < kGroups; ++c) {
    load_group<kDtype>(static_cast<const T*>(a.x) + base, k, c, x[c]);
    if (a.y) load_group<kDtype>(static_cast<const T*>(a.y) + base, k, c, y[c]);
  }
  if (a.y) {
    if (a.w_post) {
      float ss = 0.0f;
#pragma unroll
      for (int c = 0; c < kGroups; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) ss += y[c][j] * y[c][j];
      const float r_post = 1.0f / sqrtf(block_sum<kWaves>(ss, lds) / inv_d + a.eps);
      if (k.lane == 0 && a.rstd_post) a.rstd_post[row] = r_post;
#pragma unroll
      for (int c = 0; c < kGroups; ++c) {
        float w[8];
        load_group<kDtype>(a.w_post, k, c, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[c][j] = y[c][j] * r_post * w[j];
      }
    }
    if (a.gate) {
#pragma unroll
      for (int c = 0; c < kGroups; ++c) {
        float w[8];
        load_group<kDtype>(static_cast<const T*>(a.gate) + (size_t)row * a.gate_stride, k, c, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[c][j] *= w[j];
      }
    }
#pragma unroll
    for (int c = 0; c < kGroups; ++c) {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[c][j] += a.scale * y[c][j];
      store_group<kDtype, kStream>(static_cast<T*>(a.h) + base, k, c, x[c]);
    }
  }
  float ss = 0.0f;
#pragma unroll
  for (int c = 0; c < kGroups; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) ss += x[c][j] * x[c][j];
  const float r_pre = 1.0f / sqrtf(block_sum<kWaves>(ss, lds) / inv_d + a.eps);
  if (k.lane == 0 && a.rstd_pre) a.rstd_pre[row] = r_pre;
#pragma unroll
  for (int c = 0; c < kGroups; ++c) {
    float w[8];
    load_group<kDtype>(a.w_pre, k, c, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[c][j] = x[c][j] * r_pre * w[j];
    if constexpr (!kFp8) store_group<kDtype, kStream>(static_cast<T*>(a.u) + base, k, c, x[c]);
  }
  if constexpr (kFp8) {
    float amax = 0.0f;
#pragma unroll
    for (int c = 0; c < kGroups; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(x[c][j]));
    amax = block_max<kWaves>(amax, lds);
    const float s = e4m3_scale(amax);
    if (k.lane == 0) a.u_scale[row] = s;
#pragma unroll
    for (int c = 0; c < kGroups; ++c) {
      const int at = k.at(c, 0);
      float q[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) q[j] = __fdiv_rn(x[c][j], s);
      if (at < k.d)
        *reinterpret_cast<uint2*>(a.codes + base + at) =
            make_uint2(e4m3_code4(q[0], q[1], q[2], q[3]), e4m3_code4(q[4], q[5], q[6], q[7]));
    }
  }
}

// ---- rows of any width

// Any width: columns one by one, a row's later passes read it again (from
// the caches; h by the thread that wrote it).
template <int kDtype, bool kFp8>
__global__ __launch_bounds__(kNormThreads) void norm_rows_kernel(NormArgs a) {
  using E = Elem<kDtype>;
  using T = typename E::T;
  __shared__ float lds[kNormThreads / 64];
  constexpr int kW = kNormThreads / 64;
  const long long row = flat_group();
  if (row >= a.n_rows) return;
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
    const float s = e4m3_scale(amax);
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

// The whole backward of rows blockIdx.x, + gridDim.x, ... (kGroups groups of 8
// columns per thread, blockDim.x threads per row), its column sums to
// part[blockIdx.x].
constexpr int kBwdMaxWaves = 8;

template <int kDtype, int kGrad, bool kVec, int kGroups>
__global__ __launch_bounds__(64 * kBwdMaxWaves, kGroups == 1 ? 3 : 2) void norm_backward_held_kernel(NormBwdArgs a) {
  using T = typename Elem<kDtype>::T;
  using TG = typename Elem<kGrad>::T;
  __shared__ float lds[2][kBwdMaxWaves][3];
  const Columns<kVec> k{a.d, (int)blockDim.x, (int)threadIdx.x};
  const int wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const float inv_d = (float)a.d;
  const bool shared_gate = a.gate && a.gate_stride == 0;
  float s_pre[kGroups][8], s_post[kGroups][8], s_gate[kGroups][8];
#pragma unroll
  for (int c = 0; c < kGroups; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) s_pre[c][j] = s_post[c][j] = s_gate[c][j] = 0.0f;
  using G = Group<kDtype, kVec>;
  G w_pre[kGroups], w_post[kGroups], gate[kGroups];
#pragma unroll
  for (int c = 0; c < kGroups; ++c) {
    w_pre[c].load(a.w_pre, k, c);
    if (a.w_post) w_post[c].load(a.w_post, k, c);
    if (shared_gate) gate[c].load(a.gate, k, c);
  }
  // A row's values as loaded: the next row's are on their way while a row is
  // summed and written.
  Group<kGrad, kVec> r_du[kGroups];
  G r_h[kGroups], r_dh[kGroups], r_y[kGroups], r_gate[kGroups];
  float n_pre, n_post;
  auto fetch = [&](long long row) {
    const size_t base = (size_t)row * a.d;
    n_pre = a.rstd_pre[row];
    n_post = a.w_post ? a.rstd_post[row] : 1.0f;
#pragma unroll
    for (int c = 0; c < kGroups; ++c) {
      r_du[c].load(static_cast<const TG*>(a.du) + base, k, c);
      r_h[c].load(static_cast<const T*>(a.h) + base, k, c);
      if (a.dh) r_dh[c].load(static_cast<const T*>(a.dh) + base, k, c);
      if (a.y) r_y[c].load(static_cast<const T*>(a.y) + base, k, c);
      if (a.gate && !shared_gate) r_gate[c].load(static_cast<const T*>(a.gate) + base, k, c);
    }
  };
  constexpr bool kAhead = kGroups == 1;  // (two groups have no registers left for it)
  if (kAhead && blockIdx.x < a.n_rows) fetch(blockIdx.x);
  int flip = 0;
  for (long long row = blockIdx.x; row < a.n_rows; row += gridDim.x, flip ^= 1) {
    const size_t base = (size_t)row * a.d;
    if constexpr (!kAhead) fetch(row);
    const float r_pre = n_pre, r_post = n_post;
    // g = dx without the mean's part, n, q
    float g[kGroups][8], n[kGroups][8], q[kGroups][8];
    float A = 0.0f, B = 0.0f, C = 0.0f;
#pragma unroll
    for (int c = 0; c < kGroups; ++c) {
      if (!shared_gate) gate[c] = r_gate[c];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float u = r_du[c][j];
        n[c][j] = r_h[c][j] * r_pre;
        s_pre[c][j] += u * n[c][j];
        const float dn = u * w_pre[c][j];
        A += dn * n[c][j];
        const float v = r_pre * dn;
        g[c][j] = a.dh ? r_dh[c][j] + v : v;
        q[c][j] = a.y ? r_y[c][j] * r_post : 0.0f;
      }
      if (a.w_post) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float s = a.scale * (a.gate ? gate[c][j] : 1.0f) * w_post[c][j] * q[c][j];
          B += s * g[c][j];
          C += s * (r_pre * n[c][j]);
        }
      }
    }
    if (kAhead && row + gridDim.x < a.n_rows) fetch(row + gridDim.x);
    A = wave_sum_moves(A);
    if (a.w_post) B = wave_sum_moves(B), C = wave_sum_moves(C);
    // (two buffers: a row's sums are read while the next row's are written)
    if ((threadIdx.x & 63) == 0) {
      lds[flip][wave][0] = A;
      lds[flip][wave][1] = B;
      lds[flip][wave][2] = C;
    }
    __syncthreads();
    A = lds[flip][0][0], B = lds[flip][0][1], C = lds[flip][0][2];
    for (int w = 1; w < waves; ++w) A += lds[flip][w][0], B += lds[flip][w][1], C += lds[flip][w][2];
    const float c1 = A / inv_d;
    const float c2 = (B - c1 * C) / inv_d;
#pragma unroll
    for (int c = 0; c < kGroups; ++c) {
#pragma unroll
      for (int j = 0; j < 8; ++j) g[c][j] -= r_pre * (n[c][j] * c1);
      if (a.y) {
        float dy[8], dg[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float sdx = a.scale * g[c][j];
          const float dp = a.gate ? sdx * gate[c][j] : sdx;
          if (a.gate) {
            dg[j] = sdx * (a.w_post ? q[c][j] * w_post[c][j] : q[c][j]);
            s_gate[c][j] += dg[j];
          }
          if (a.w_post) {
            s_post[c][j] += dp * q[c][j];
            dy[j] = r_post * (dp * w_post[c][j] - q[c][j] * c2);
          } else {
            dy[j] = dp;
          }
        }
        store_group<kDtype>(static_cast<T*>(a.dy) + base, k, c, dy);
        if (a.dgate_rows) store_group<kDtype>(static_cast<T*>(a.dgate_rows) + base, k, c, dg);
      }
      store_group<kDtype>(static_cast<T*>(a.dx) + base, k, c, g[c]);
    }
  }
  float* part = a.part + (size_t)blockIdx.x * 3 * a.d;
#pragma unroll
  for (int c = 0; c < kGroups; ++c) {
    store_group<1>(part, k, c, s_pre[c]);
    if (a.w_post) store_group<1>(part + a.d, k, c, s_post[c]);
    if (shared_gate) store_group<1>(part + 2 * (size_t)a.d, k, c, s_gate[c]);
  }
}

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

// Two results of more bytes than this together are stored past the caches: the
// next reader would not find them there (the Infinity Cache holds 256 MiB),
// and the operands still to come keep their place (16384 x 2560 bf16: 71 -> 64
// us; 4096 x 7168 the same either way, and a decode step's rows stay cached).
// The backward's gradients are not: 137 us with plain stores, 141 past them.
constexpr long long kStreamBytes = 128LL << 20;

constexpr int kWaveWidth = 4096;      // widest row of one wavefront
constexpr int kNormMaxWidth = 16384;  // widest row held in registers
constexpr int kBwdMaxWidth = 8192;    // the same of the backward

// Whether the backward holds the rows (two groups of scattered columns would
// not fit the registers), and its wavefronts per row then.
bool held_backward(long long d) { return d <= (d % 8 == 0 ? kBwdMaxWidth : kBwdMaxWidth / 2); }
int held_waves(long long d) {
  const long long groups = ceil_div(d, 8);
  return (int)(groups <= 64 * kBwdMaxWaves ? ceil_div(groups, 64) : ceil_div(groups, 128));
}

// Runs of rows of the column sums. Held rows: a workgroup's, as many
// workgroups as run at once (12 wavefronts per CU with one group, 8 with two:
// their registers), so that few sums are left to add, and 4 rows each where
// there are fewer. Other rows: about 64 rows each, at most 256.
int norm_runs(long long n_rows, long long d) {
  if (!held_backward(d)) return (int)std::min<long long>(256, ceil_div(n_rows, 64));
  const int per_cu = std::max(1, (ceil_div(d, 8) <= 64 * kBwdMaxWaves ? 12 : 8) / held_waves(d));
  return (int)std::min<long long>(256 * std::min(per_cu, 8), ceil_div(n_rows, 4));
}

template <int kDtype, bool kFp8, bool kVec>
void run_norm(const NormArgs& a, hipStream_t stream) {
  const dim3 block(kNormThreads), one = flat_grid(ceil_div(a.n_rows, kNormThreads / 64)), four = flat_grid(a.n_rows);
  // As many groups per thread as the width takes: the sums' order and bits are
  // those of more (empty groups add zeros), and no lane holds or loads any. With
  // 1, 2, 4, 5 and 8 groups (four wavefronts: 3, 4 and 8) alone, us of 16384 rows
  // (from 8960 on 4096), bf16, then to E4M3 rows: width 1536 32.9 -> 32.2, 33.1 ->
  // 32.5; 2944 66 -> 61, 95 -> 76; 3584 76 -> 73, 105 -> 88; 8960 57 -> 46, 71 -> 50;
  // 10240 60 -> 50, 87 -> 60; fp32 within 4 % either way.
  const int groups = (int)ceil_div(ceil_div(a.d, 8), a.d <= kWaveWidth ? 64 : kNormThreads);
#define ITL_NORM(waves, n, grid)                                                                            \
  case n:                                                                                                   \
    if (kVec && !kFp8 && a.stream)                                                                          \
      hipLaunchKernelGGL((norm_held_kernel<kDtype, kFp8, kVec, kVec && !kFp8, waves, n>), grid, block, 0, stream, a); \
    else                                                                                                    \
      hipLaunchKernelGGL((norm_held_kernel<kDtype, kFp8, kVec, false, waves, n>), grid, block, 0, stream, a); \
    break
  if (a.d <= kWaveWidth) {
    switch (groups) {
      ITL_NORM(1, 1, one);
      ITL_NORM(1, 2, one);
      ITL_NORM(1, 3, one);
      ITL_NORM(1, 4, one);
      ITL_NORM(1, 5, one);
      ITL_NORM(1, 6, one);
      ITL_NORM(1, 7, one);
      ITL_NORM(1, 8, one);
    }
  } else if (a.d <= kNormMaxWidth) {
    switch (groups) {
      ITL_NORM(4, 3, four);
      ITL_NORM(4, 4, four);
      ITL_NORM(4, 5, four);
      ITL_NORM(4, 6, four);
      ITL_NORM(4, 7, four);
      ITL_NORM(4, 8, four);
    }
  } else {
    hipLaunchKernelGGL((norm_rows_kernel<kDtype, kFp8>), four, block, 0, stream, a);
  }
#undef ITL_NORM
}

}  // namespace

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
    if (dtype == 0) run_norm<0, true, true>(a, stream);
    else run_norm<1, true, true>(a, stream);
  } else if (d % 8 == 0) {
    if (dtype == 0) run_norm<0, false, true>(a, stream);
    else run_norm<1, false, true>(a, stream);
  } else {
    if (dtype == 0) run_norm<0, false, false>(a, stream);
    else run_norm<1, false, false>(a, stream);
  }
  return hipGetLastError();
}

namespace {

template <int kDtype, int kGrad, bool kVec>
void run_held_backward(const NormBwdArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)a.runs), block((unsigned)held_waves(a.d) * 64);
  if (ceil_div(a.d, 8) <= 64 * kBwdMaxWaves)
    hipLaunchKernelGGL((norm_backward_held_kernel<kDtype, kGrad, kVec, 1>), grid, block, 0, stream, a);
  else if constexpr (kVec)
    hipLaunchKernelGGL((norm_backward_held_kernel<kDtype, kGrad, kVec, 2>), grid, block, 0, stream, a);
}

template <int kDtype, int kGrad>
void run_norm_backward(const NormBwdArgs& a, hipStream_t stream) {
  if (held_backward(a.d)) {
    if (a.d % 8 == 0) run_held_backward<kDtype, kGrad, true>(a, stream);
    else run_held_backward<kDtype, kGrad, false>(a, stream);
    return;
  }
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
                gate_stride, d, norm_runs(n_rows, d), scale};
  if (n_rows > 0) {
    if (dtype == 0) {
      if (grad_dtype == 0) run_norm_backward<0, 0>(a, stream);
      else run_norm_backward<0, 1>(a, stream);
    } else {
      run_norm_backward<1, 1>(a, stream);
    }
  }
  hipLaunchKernelGGL(norm_backward_finish_kernel, dim3((unsigned)ceil_div(d, 64), 3), dim3(64 * kFinishWaves), 0, stream, a.part,
                     a.runs, d, dw_pre, w_post ? dw_post : nullptr, shared_gate ? static_cast<float*>(dgate) : nullptr);
  return hipGetLastError();
}

}  // namespace itl
