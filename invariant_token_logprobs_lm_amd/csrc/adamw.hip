// One AdamW step over many tensors.
//
//   g = clip * grad              clip = min(1, max_norm / (|grads| + 1e-6)), |.| over all tensors
//   m = beta1 m + (1 - beta1) g
//   v = beta2 v + (1 - beta2) g^2
//   w = w (1 - lr decay) - lr / (1 - beta1^t) * m / (sqrt(v) / sqrt(1 - beta2^t) + eps)
//
// w is the fp32 master of a bf16 weight (the weight then gets its rounding)
// or the weight itself. Every product, sum, quotient and root is rounded to
// fp32 on its own (nothing is fused), t and the powers are fp64.
//
// 8-bit states: m and sqrt(v) as E4M3 codes with an fp32 scale per 256
// elements (the largest at 448, the scale no less than 2^-126; 1 for an
// all-zero block), to nearest even.
// The root is stored rather than v because its dynamic range is half of v's
// in the exponent: the codes then hold v down to 2^-36 of a block's largest.
// A root that is not zero never gets code 0 (the smallest code instead): a
// later m / sqrt(v) of an element whose v was lost would run away. The
// weights are updated from the fp32 m and v before they are stored.
//
// The step count and the learning rate are read from device memory and the
// count is raised by the step itself, so a captured step replays right.
// A norm that is not finite leaves everything, the count too, as it was.
//
// The pieces of work (up to 2048 elements of one tensor) are laid out once
// in the plan: one launch for all tensors, one workgroup per piece. The
// square sum of the gradients takes a fixed set of pieces per workgroup and
// adds the workgroups in order, in fp64: run-to-run deterministic.
//
// Bound by memory: 252 M bf16 weights with fp32 masters and states, 7.1 GB,
// update in 1.20 to 1.31 ms (5.4 to 5.9 TB/s; a large copy moves 4.7), with the
// norm's 0.5 GB 1.33 to 1.46 ms; 389 M with 8-bit states and fp32 gradients 7.0
// GB in 1.18 to 1.32 ms, with the norm 1.53 to 1.64 ms. Pieces of 2048 elements, one pass of 8 per thread, beat
// 4096 (two passes; 9 % slower) and 1024 on 128 threads (3 %): many short
// workgroups keep loads and stores of different pieces in flight together.

#include <math.h>

#include "adamw_plan.h"
#include "itl_launch.h"
#include "learner_common.h"

namespace itl {

namespace {

// Eight consecutive values of a bf16 or fp32 array, those past `left` zero.
template <bool kF32>
__device__ __forceinline__ void load8(const void* p, int i, int left, bool vec, float (&v)[8]) {
  if (vec && left >= 8) {
    if constexpr (kF32) {
      const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
      const float4 a = s[0], b = s[1];
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
      const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
      const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = __uint_as_float((j & 1) ? (w[j >> 1] & 0xffff0000u) : (w[j >> 1] << 16));
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if constexpr (kF32) v[j] = j < left ? static_cast<const float*>(p)[i + j] : 0.0f;
    else v[j] = j < left ? Elem<0>::to_f(static_cast<const uint16_t*>(p)[i + j]) : 0.0f;
  }
}

template <bool kF32>
__device__ __forceinline__ void store8(void* p, int i, int left, bool vec, const float (&v)[8]) {
  if (vec && left >= 8) {
    if constexpr (kF32) {
      float4* s = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
      s[0] = make_float4(v[0], v[1], v[2], v[3]);
      s[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[j] = (uint32_t)Elem<0>::from_f(v[2 * j]) | ((uint32_t)Elem<0>::from_f(v[2 * j + 1]) << 16);
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (j >= left) break;
    if constexpr (kF32) static_cast<float*>(p)[i + j] = v[j];
    else static_cast<uint16_t*>(p)[i + j] = Elem<0>::from_f(v[j]);
  }
}

__device__ __forceinline__ double block_sum_d(double x, double* lds, int waves) {
  x = wave_sum_d(x);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
  __syncthreads();
  double s = lds[0];
  for (int w = 1; w < waves; ++w) s += lds[w];
  return s;
}

// Square sum of the gradients of pieces blockIdx.x, + gridDim.x, ..., in fp64
// (no gradient's square overflows or vanishes).
__global__ __launch_bounds__(kAdamThreads) void adamw_norm_kernel(const AdamPiece* __restrict__ pieces, long long n,
                                                                  double* __restrict__ part) {
  __shared__ double lds[kAdamThreads / 64];
  double sum = 0.0;
  for (long long c = blockIdx.x; c < n; c += gridDim.x) {
    const AdamPiece p = pieces[c];
#pragma unroll
    for (int at = 0; at < kAdamPiece; at += kAdamThreads * kAdamVec) {
      const int i = at + threadIdx.x * kAdamVec;
      if (i >= p.count) break;
      float g[8];
      if (p.flags & kAdamGradF32) load8<true>(p.grad, i, p.count - i, p.flags & kAdamVectors, g);
      else load8<false>(p.grad, i, p.count - i, p.flags & kAdamVectors, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum += (double)g[j] * (double)g[j];
    }
  }
  sum = block_sum_d(sum, lds, kAdamThreads / 64);
  if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

// The norm, the clip factor, the step count and the factors that go by it.
__global__ __launch_bounds__(256) void adamw_scalars_kernel(const double* __restrict__ part, int n_part,
                                                            bool with_norm, float max_norm, double beta1, double beta2,
                                                            const float* __restrict__ lr, int64_t* __restrict__ step,
                                                            float* __restrict__ norm_out,
                                                            AdamScalars* __restrict__ out) {
  __shared__ double lds[4];
  double s = 0.0;
  for (int i = threadIdx.x; i < n_part; i += 256) s += part[i];
  s = block_sum_d(s, lds, 4);
  if (threadIdx.x != 0) return;
  AdamScalars o;
  o.clip = 1.0f;
  o.skip = 0;
  if (with_norm) {
    const float norm = (float)sqrt(s);
    if (norm_out) *norm_out = norm;
    o.clip = fminf(max_norm / (norm + 1e-6f), 1.0f);
    o.skip = !(norm < INFINITY);
  }
  const int64_t t = *step + 1;
  if (!o.skip) *step = t;
  const double l = (double)*lr;
  o.lr = *lr;
  o.rate = (float)(l / (1.0 - pow(beta1, (double)t)));
  o.root = (float)(1.0 / sqrt(1.0 - pow(beta2, (double)t)));
  *out = o;
}

struct AdamArgs {
  const AdamPiece* pieces;
  const AdamScalars* scalars;
  void *m, *v;
  float *m_scale, *v_scale, *master;
  float beta1, one_minus_beta1, beta2, one_minus_beta2, eps;
};

// Largest of a block's 256 values, held by 32 lanes.
__device__ __forceinline__ float block_amax(const float (&x)[8]) {
  float a = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) a = fmaxf(a, fabsf(x[j]));
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) a = fmaxf(a, __shfl_xor(a, off, 64));
  return a;
}

template <bool k8Bit>
__global__ __launch_bounds__(kAdamThreads) void adamw_update_kernel(AdamArgs a) {
  const AdamScalars sc = *a.scalars;
  if (sc.skip) return;
  const AdamPiece p = a.pieces[blockIdx.x];
  const bool pf32 = p.flags & kAdamParamF32, vec = p.flags & kAdamVectors;
  const float decay = 1.0f - sc.lr * p.weight_decay;
  float* master = a.master && !pf32 ? a.master + p.state : nullptr;
#pragma unroll
  for (int at = 0; at < kAdamPiece; at += kAdamThreads * kAdamVec) {
    const int i = at + threadIdx.x * kAdamVec;
    const int left = p.count - i;  // may be <= 0: the lane then only helps its block
    if (at >= p.count) return;     // whole workgroup
    const long long si = p.state + i;
    const bool live = left > 0;
    float g[8], w[8], m[8], v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] = w[j] = m[j] = v[j] = 0.0f;
    if (live) {
      if (p.flags & kAdamGradF32) load8<true>(p.grad, i, left, vec, g);
      else load8<false>(p.grad, i, left, vec, g);
      if (master) load8<true>(master, i, left, true, w);
      else if (pf32) load8<true>(p.param, i, left, vec, w);
      else load8<false>(p.param, i, left, vec, w);
      if constexpr (!k8Bit) {
        load8<true>(static_cast<float*>(a.m) + p.state, i, left, true, m);
        load8<true>(static_cast<float*>(a.v) + p.state, i, left, true, v);
      } else {
        // whole blocks are stored, so a block's last codes may be read past `left`
        const uint2 mc = *reinterpret_cast<const uint2*>(static_cast<uint8_t*>(a.m) + si);
        const uint2 vc = *reinterpret_cast<const uint2*>(static_cast<uint8_t*>(a.v) + si);
        const float ms = a.m_scale[si / kAdamBlock], vs = a.v_scale[si / kAdamBlock];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t mw = j < 4 ? mc.x : mc.y, vw = j < 4 ? vc.x : vc.y;
          m[j] = e4m3_value((mw >> (8 * (j & 3))) & 0xffu) * ms;
          const float r = e4m3_value((vw >> (8 * (j & 3))) & 0xffu) * vs;
          v[j] = r * r;
        }
      }
    }
    float r[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float gc = g[j] * sc.clip;
      m[j] = m[j] * a.beta1 + gc * a.one_minus_beta1;
      v[j] = v[j] * a.beta2 + gc * gc * a.one_minus_beta2;
      r[j] = sqrtf(v[j]);
      w[j] = w[j] * decay - m[j] / (r[j] * sc.root + a.eps) * sc.rate;
      if (k8Bit && j >= left) m[j] = r[j] = 0.0f;  // nothing of the elements past the tensor in the block's scale
    }
    if (live) {
      if (master) store8<true>(master, i, left, true, w);
      if (pf32) store8<true>(p.param, i, left, vec, w);
      else store8<false>(p.param, i, left, vec, w);
    }
    if constexpr (!k8Bit) {
      if (live) {
        store8<true>(static_cast<float*>(a.m) + p.state, i, left, true, m);
        store8<true>(static_cast<float*>(a.v) + p.state, i, left, true, v);
      }
    } else {
      const float ma = block_amax(m), ra = block_amax(r);
      const float ms = e4m3_scale(ma), vs = e4m3_scale(ra);
      float q[8], o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        q[j] = m[j] / ms;
        o[j] = r[j] / vs;
        o[j] = r[j] > 0.0f ? fmaxf(o[j], 0x1p-9f) : o[j];
      }
      if (live) {
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.m) + si) =
            make_uint2(e4m3_code4(q[0], q[1], q[2], q[3]), e4m3_code4(q[4], q[5], q[6], q[7]));
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.v) + si) =
            make_uint2(e4m3_code4(o[0], o[1], o[2], o[3]), e4m3_code4(o[4], o[5], o[6], o[7]));
        if ((threadIdx.x & 31) == 0) {
          a.m_scale[si / kAdamBlock] = ms;
          a.v_scale[si / kAdamBlock] = vs;
        }
      }
    }
  }
}

}  // namespace

size_t adamw_workspace_bytes() { return align256(kAdamNormGroups * sizeof(double)) + align256(sizeof(AdamScalars)); }

hipError_t launch_adamw_step(const void* plan, long long n_pieces, int state_bits, void* m, void* v, float* m_scale,
                             float* v_scale, float* master, const float* lr, int64_t* step, double beta1, double beta2,
                             double eps, bool with_norm, float max_norm, float* norm, void* workspace,
                             hipStream_t stream) {
  const AdamPiece* pieces = static_cast<const AdamPiece*>(plan);
  double* part = static_cast<double*>(workspace);
  AdamScalars* scalars = reinterpret_cast<AdamScalars*>(static_cast<char*>(workspace) + align256(kAdamNormGroups * sizeof(double)));
  const int groups = with_norm ? (int)(n_pieces < kAdamNormGroups ? n_pieces : kAdamNormGroups) : 0;
  if (groups > 0)
    hipLaunchKernelGGL(adamw_norm_kernel, dim3((unsigned)groups), dim3(kAdamThreads), 0, stream, pieces, n_pieces, part);
  hipLaunchKernelGGL(adamw_scalars_kernel, dim3(1), dim3(256), 0, stream, part, groups, with_norm, max_norm, beta1,
                     beta2, lr, step, norm, scalars);
  const AdamArgs a{pieces, scalars, m, v, m_scale, v_scale, master,
                   (float)beta1, (float)(1.0 - beta1), (float)beta2, (float)(1.0 - beta2), (float)eps};
  if (n_pieces == 0) return hipGetLastError();
  const dim3 grid((unsigned)n_pieces), block(kAdamThreads);
  if (state_bits == 8) hipLaunchKernelGGL(adamw_update_kernel<true>, grid, block, 0, stream, a);
  else hipLaunchKernelGGL(adamw_update_kernel<false>, grid, block, 0, stream, a);
  return hipGetLastError();
}

}  // namespace itl
