// E4M3 codes with a scale for each block of 128 values, the operands of the
// block-scaled product (matmul_fp8.hip):
//   blocks: scale[b, r] = amax over columns 128 b .. of row r / 448
//   tiles:  scale[i, j] = amax over the 128 x 128 tile (i, j) / 448
//   code = E4M3(x / scale), to nearest even (1 for zeros, no less than 2^-126)
// and, for the products whose contraction runs over the rows, the same of the
// transpose (blocks: of 128 rows; tiles: the same codes). Rows of codes are
// padded with zeros to whole blocks, so that a product needs no end of its own.
//
// Scales of blocks lie block by block ([blocks, rows]): a product's workgroup
// takes one block of 256 rows at a time, 1 KB in a line instead of 256 lines.
//
// Bound by memory: each value is read once, also where both directions are
// written: a workgroup holds a 128 x 128 tile in registers (thread: 8 rows by 8
// columns), takes the rows' maxima over 16 lanes and the columns' through LDS,
// and turns the codes through 16 KB of LDS so that both are written in whole
// lines. 16384 x 2560 bf16 rows alone 31 to 33 us (3.8 to 4.0 TB/s), the
// transpose alone 28 (4.6), both ways 39 to 42 (4.0 to 4.3; 68 % of the cycles issue vector
// instructions); by tiles 23, 24 and 33 (5.0 to 5.4); 8960 x 1536 fp32 by tiles, both ways,
// 16 to 19 (4.3 to 5.2). Odd widths: 10000 x 2999 bf16 26, 35 and 45 (2.6 to 3.4), by tiles
// 30, 30 and 36. One decode token 3, launch and latency.

#include <algorithm>

#include "block_codes.h"
#include "itl_launch.h"

namespace itl {

namespace {

constexpr int kQuantThreads = 256;

struct QuantArgs {
  const void* X;
  long long n_rows, d;
  uint8_t *Xq, *Xtq;
  float *scale, *t_scale;
};

// Eight consecutive values of a row from column k on, zeros past its end, by 16-byte
// loads. kWhole: rows are whole groups of 8 and start at 16 bytes; others start at
// any element (10000 x 2999 bf16 took 41 us element by element, 24 this way), and
// whole rows without the branch on their end 40 us where 58 with it.
template <int kDtype, bool kWhole>
__device__ __forceinline__ void load8(const void* X, long long row, long long d, long long k, bool in, float (&v)[8]) {
  using E = Elem<kDtype>;
  using T = typename E::T;
  const T* p = static_cast<const T*>(X) + (size_t)row * d + k;
  if constexpr (kWhole) {
    uint4 w[E::kSize / 2];
#pragma unroll
    for (int i = 0; i < E::kSize / 2; ++i) w[i] = in && k < d ? reinterpret_cast<const uint4*>(p)[i] : make_uint4(0u, 0u, 0u, 0u);
    T t[8];
    __builtin_memcpy(t, w, sizeof t);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = E::to_f(t[j]);
  } else {
    T t[8];
    if (in && k + 8 <= d) {
      __builtin_memcpy(t, p, sizeof t);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) t[j] = in && k + j < d ? p[j] : T(0);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = E::to_f(t[j]);
  }
}

// Blocks of rows alone: 16 lanes have a block, a thread kQuantGroups of them,
// all read before the first is dealt with.
constexpr int kQuantGroups = 4;

template <int kDtype, bool kWhole>
__global__ __launch_bounds__(kQuantThreads) void quantize_block_rows_kernel(QuantArgs a) {
  const int blocks = (int)((a.d + kCodeBlock - 1) / kCodeBlock);
  const long long all = a.n_rows * blocks;
  const long long first = flat_group() * (kQuantGroups * kQuantThreads / 16) + (threadIdx.x >> 4);
  const int lane16 = threadIdx.x & 15;
  float v[kQuantGroups][8];
  long long row[kQuantGroups];
  int block[kQuantGroups];
#pragma unroll
  for (int g = 0; g < kQuantGroups; ++g) {
    const long long f = first + g * (kQuantThreads / 16);
    row[g] = f < (1LL << 32) ? (uint32_t)f / (uint32_t)blocks : f / blocks;
    block[g] = (int)(f - row[g] * blocks);
    load8<kDtype, kWhole>(a.X, row[g], a.d, (long long)block[g] * kCodeBlock + lane16 * 8, f < all, v[g]);
  }
#pragma unroll
  for (int g = 0; g < kQuantGroups; ++g) {
    const long long f = first + g * (kQuantThreads / 16);
    const float s = e4m3_scale(largest16(largest8(v[g])));
    if (f < all) {
      *reinterpret_cast<uint2*>(a.Xq + (size_t)f * kCodeBlock + lane16 * 8) = codes8(v[g], Quotient(s));
      if (lane16 == 0) a.scale[(size_t)block[g] * a.n_rows + row[g]] = s;
    }
  }
}

// A 128 x 128 tile per workgroup: rows' codes (Xq), the transpose's (Xtq), or both.
template <int kDtype, bool kWhole, bool kTiles>
__global__ __launch_bounds__(kQuantThreads) void quantize_tile_kernel(QuantArgs a) {
  __shared__ float tops[4][kCodeBlock];
  __shared__ uint2 turned[kCodeBlock * 16];  // [column][8 rows], chunk c of column k at c ^ (k / 8)
  const int across = (int)((a.d + kCodeBlock - 1) / kCodeBlock);
  const long long down = (a.n_rows + kCodeBlock - 1) / kCodeBlock;
  const long long tile = flat_group();
  if (tile >= across * down) return;
  const long long ti = tile / across;
  const int tj = (int)(tile - ti * across);
  const int cg = threadIdx.x & 15, rg = threadIdx.x >> 4;  // columns 8 cg .., rows 8 rg ..
  const long long r0 = ti * kCodeBlock + 8 * rg, k0 = (long long)tj * kCodeBlock + 8 * cg;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float x[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) load8<kDtype, kWhole>(a.X, r0 + i, a.d, k0, r0 + i < a.n_rows, x[i]);
  float s = 1.0f, s_column[8];
  if constexpr (kTiles) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, largest8(x[i]));
    m = largest16(m);
    m = fmaxf(m, __shfl_xor(m, 16, 64));
    m = fmaxf(m, __shfl_xor(m, 32, 64));
    if (lane == 0) tops[wave][0] = m;
    __syncthreads();
    s = e4m3_scale(fmaxf(fmaxf(tops[0][0], tops[1][0]), fmaxf(tops[2][0], tops[3][0])));
    if (threadIdx.x == 0) {
      if (a.Xq) a.scale[(size_t)ti * across + tj] = s;
      if (a.Xtq) a.t_scale[(size_t)tj * down + ti] = s;
    }
  } else if (a.Xtq) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float m = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i][j]));
      m = fmaxf(m, __shfl_xor(m, 16, 64));
      m = fmaxf(m, __shfl_xor(m, 32, 64));
      if (lane < 16) tops[wave][8 * cg + j] = m;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int k = 8 * cg + j;
      s_column[j] = e4m3_scale(fmaxf(fmaxf(tops[0][k], tops[1][k]), fmaxf(tops[2][k], tops[3][k])));
      if (rg == 0 && k0 + j < a.d) a.t_scale[(size_t)ti * a.d + k0 + j] = s_column[j];
    }
  }
  const size_t width = (size_t)across * kCodeBlock;
  const Quotient one(s);
  if (a.Xq) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (!kTiles) s = e4m3_scale(largest16(largest8(x[i])));
      if (r0 + i >= a.n_rows) continue;
      *reinterpret_cast<uint2*>(a.Xq + (size_t)(r0 + i) * width + k0) = codes8(x[i], kTiles ? one : Quotient(s));
      if (!kTiles && cg == 0) a.scale[(size_t)tj * a.n_rows + r0 + i] = s;
    }
  }
  if (!a.Xtq) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = x[i][j];
    turned[(8 * cg + j) * 16 + (rg ^ cg)] = codes8(v, kTiles ? one : Quotient(s_column[j]));
  }
  __syncthreads();
  const size_t height = (size_t)down * kCodeBlock;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int k = (threadIdx.x >> 3) + 32 * i, c = 2 * (threadIdx.x & 7), x8 = k >> 3;
    const long long column = (long long)tj * kCodeBlock + k;
    const uint2 lo = turned[k * 16 + (c ^ x8)], hi = turned[k * 16 + ((c + 1) ^ x8)];
    if (column < a.d)
      *reinterpret_cast<uint4*>(a.Xtq + (size_t)column * height + (size_t)ti * kCodeBlock + 8 * c) = make_uint4(lo.x, lo.y, hi.x, hi.y);
  }
}

template <int kDtype, bool kWhole>
void run_quantize(const QuantArgs& a, bool tiles, hipStream_t stream) {
  const long long across = ceil_div(a.d, kCodeBlock), down = ceil_div(a.n_rows, kCodeBlock);
  const dim3 block(kQuantThreads);
  if (tiles)
    hipLaunchKernelGGL((quantize_tile_kernel<kDtype, kWhole, true>), flat_grid(across * down), block, 0, stream, a);
  else if (a.Xtq)
    hipLaunchKernelGGL((quantize_tile_kernel<kDtype, kWhole, false>), flat_grid(across * down), block, 0, stream, a);
  else
    hipLaunchKernelGGL((quantize_block_rows_kernel<kDtype, kWhole>),
                       flat_grid(ceil_div(a.n_rows * across, kQuantGroups * kQuantThreads / 16)), block, 0, stream, a);
}

}  // namespace

hipError_t launch_quantize_blocks(const void* X, int dtype, long long n_rows, long long d, bool tiles, uint8_t* Xq,
                                  float* scale, uint8_t* Xtq, float* t_scale, hipStream_t stream) {
  const QuantArgs a{X, n_rows, d, Xq, Xtq, scale, t_scale};
  const bool whole = d % 8 == 0 && (reinterpret_cast<uintptr_t>(X) & 15) == 0;
  if (dtype == 0) {
    if (whole) run_quantize<0, true>(a, tiles, stream);
    else run_quantize<0, false>(a, tiles, stream);
  } else {
    if (whole) run_quantize<1, true>(a, tiles, stream);
    else run_quantize<1, false>(a, tiles, stream);
  }
  return hipGetLastError();
}

}  // namespace itl
