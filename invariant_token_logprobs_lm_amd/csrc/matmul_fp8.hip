// The product of two E4M3 matrices with a scale for each block of 128 along the
// contraction: a linear layer's forward, and its two gradients, in 8 bits.
//   C[i, j] = sum_b a_scale[b, i] b_scale[j / 128, b] p_b[i, j],
//   p_b[i, j] = sum over k in block b of A[i, k] B[j, k]
// A [m, k] has a scale for each 128 values of a row, B [n, k] one for each
// 128 x 128 tile.
//
// The scales are fp32 and enter after the matrix cores: acc = fma(p_b, a_scale
// b_scale, acc), blocks in ascending order. So an element's bits depend on its
// row of A, its row of B and their scales alone: every kernel here has the same
// instructions on the same fragments and the same chain, whatever its tile and
// however a workgroup's wavefronts share the blocks.
//
// bf16 results: v_mfma_scale_f32_16x16x128_f8f6f4 (its own scales 1) takes a whole
// block of 16 rows of each operand. It adds the eight products of a lane's eight
// consecutive bytes with 13 bits below the largest (measured: a product 2^-14 of
// it is lost; the sixteen sums of eight are added in fp32), so p_b is off by 1e-6 to
// 4e-5 of itself, far inside a bf16 result's 2^-9.
// fp32 results: the codes become bf16, which holds every one of them, and
// v_mfma_f32_16x16x32_bf16 sums their products in fp32 (off by 1e-8 of p_b; twice
// the instructions' time). A lane's 32 bytes are four instructions' fragments.
//
// B's rows are the instruction's first operand: a lane then holds four
// consecutive columns of a row of C (register i: column 4 (l / 16) + i of 16,
// row l mod 16), and A's scale is one per lane and 16 rows, B's one per
// wavefront: 4 fused multiply-adds and a fraction of a product per instruction.

#include <algorithm>

#include "itl_launch.h"
#include "learner_common.h"
#include "tile_engine.h"

namespace itl {

namespace {

constexpr int kBlock = 128;
static_assert(kBlock == kStepBytes, "a block is one K step");

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

// Eight codes as bf16 values (exact).
__device__ __forceinline__ bf16x8_t widen8(uint32_t lo, uint32_t hi) {
  bf16x2_t v[4];
  v[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
  v[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
  v[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
  v[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  return __builtin_bit_cast(bf16x8_t, v);
}

// A lane's 32 codes of a row and block as the result's type wants them, and the
// block's products of 16 x 16.
template <int kOut>
struct Operand;
template <>
struct Operand<0> {
  Frag8 v;
  __device__ __forceinline__ void set(const uint4& lo, const uint4& hi) { v = Frag8{lo, hi}; }
  // p[i] = b a[i]
  template <int kN>
  __device__ static __forceinline__ void products(const Operand& b, const Operand (&a)[kN], floatx4 (&p)[kN]) {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      p[i] = floatx4{};
      mma_f8_16(p[i], b.v, a[i].v);
    }
  }
};
template <>
struct Operand<1> {
  bf16x8_t v[4];
  __device__ __forceinline__ void set(const uint4& lo, const uint4& hi) {
    v[0] = widen8(lo.x, lo.y);
    v[1] = widen8(lo.z, lo.w);
    v[2] = widen8(hi.x, hi.y);
    v[3] = widen8(hi.z, hi.w);
  }
  template <int kN>
  __device__ static __forceinline__ void products(const Operand& b, const Operand (&a)[kN], floatx4 (&p)[kN]) {
#pragma unroll
    for (int i = 0; i < kN; ++i) p[i] = floatx4{};
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < kN; ++i) p[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b.v[j], a[i].v[j], p[i], 0, 0, 0);
  }
};

struct ProductArgs {
  const uint8_t *A, *B;
  const float *a_scale, *b_scale;
  void* C;
  long long m, n;
  int k, tiles_n;
  long long tiles;
  bool quads;  // C's rows are whole fours of columns, aligned as such
};

// Four consecutive columns of a row of C.
template <int kOut>
__device__ __forceinline__ void store4(const ProductArgs& a, long long row, long long col, const floatx4& v) {
  using E = Elem<kOut>;
  using T = typename E::T;
  if (row >= a.m || col >= a.n) return;
  T* out = static_cast<T*>(a.C) + row * a.n + col;
  if (a.quads) {
    if constexpr (kOut == 0) {
      *reinterpret_cast<uint2*>(out) = make_uint2((uint32_t)E::from_f(v[0]) | ((uint32_t)E::from_f(v[1]) << 16),
                                                  (uint32_t)E::from_f(v[2]) | ((uint32_t)E::from_f(v[3]) << 16));
    } else {
      *reinterpret_cast<float4*>(out) = make_float4(v[0], v[1], v[2], v[3]);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (col + i < a.n) out[i] = E::from_f(v[i]);
}

// kBR columns of C (rows of B) by kAR rows, a grid of kWB x kWA wavefronts, both
// operands through kSlots LDS slots loaded kSlots - 1 steps ahead.
template <int kOut, int kBR, int kAR, int kWB, int kWA, int kSlots>
__global__ __launch_bounds__(64 * kWB * kWA) void product_tile_kernel(ProductArgs a) {
  constexpr int kWaves = kWB * kWA;
  constexpr int kBM = kBR / kWB / 16, kAN = kAR / kWA / 16;  // 16-row blocks per wavefront
  constexpr int kBDma = kBR / 8 / kWaves, kADma = kAR / 8 / kWaves;
  constexpr int kBChunks = kBR * kRowChunks, kAChunks = kAR * kRowChunks;
  constexpr int kChunks = kBChunks + kAChunks + kAR / 4;  // of a slot: the rows, then A's scales
  static_assert(kBDma * 8 * kWaves == kBR && kADma * 8 * kWaves == kAR, "whole loads per wavefront");
  static_assert(kBlock % (kBR / kWB) == 0 && kAR % 64 == 0 && kAR / 64 <= kWaves, "a wavefront has one scale of B");
  __shared__ uint4 smem[kSlots * kChunks];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wb = wave % kWB, wa = wave / kWB;
  const int quad = lane >> 4, c16 = lane & 15;
  const long long tile = flat_group();
  if (tile >= a.tiles) return;
  const long long i0 = tile / a.tiles_n * kAR;
  const long long j0 = tile % a.tiles_n * kBR;
  const int steps = a.k / kBlock;
  const int4v b_rsrc = rsrc_words(a.B + (size_t)j0 * a.k, (uint32_t)min((long long)kBR, a.n - j0) * (uint32_t)a.k);
  const int4v a_rsrc = rsrc_words(a.A + (size_t)i0 * a.k, (uint32_t)min((long long)kAR, a.m - i0) * (uint32_t)a.k);
  const uint32_t rows = (uint32_t)min((long long)kAR, a.m - i0);
  // Lane i of a load fetches row i / 8 of eight at logical chunk (i % 8) ^ swz(row).
  const int lr = lane >> 3;
  uint32_t b_off[kBDma], a_off[kADma];
#pragma unroll
  for (int j = 0; j < kBDma; ++j) {
    const int r = (wave * kBDma + j) * 8 + lr;
    b_off[j] = (uint32_t)r * (uint32_t)a.k + (uint32_t)(((lane & 7) ^ swz(r)) * 16);
  }
#pragma unroll
  for (int j = 0; j < kADma; ++j) {
    const int r = (wave * kADma + j) * 8 + lr;
    a_off[j] = (uint32_t)r * (uint32_t)a.k + (uint32_t)(((lane & 7) ^ swz(r)) * 16);
  }
  const uint32_t lds0 = (uint32_t)(size_t)((__attribute__((address_space(3))) uint4*)smem);
  // Step s into its slot: rows of B, rows of A, and 64 of A's scales per
  // wavefront (wavefronts past the last 64 fetch some of them again, the same).
  const int sc = wave % (kAR / 64);
  auto load = [&](int s) {
    const uint32_t slot = lds0 + (uint32_t)(s % kSlots) * kChunks * 16;
    const uint32_t at = (uint32_t)s * kBlock;
#pragma unroll
    for (int j = 0; j < kBDma; ++j) dma16(b_rsrc, b_off[j], at, slot + (uint32_t)(wave * kBDma + j) * 1024);
#pragma unroll
    for (int j = 0; j < kADma; ++j) dma16(a_rsrc, a_off[j], at, slot + kBChunks * 16 + (uint32_t)(wave * kADma + j) * 1024);
    dma4(rsrc_words(a.a_scale + (size_t)s * a.m + i0, rows * 4), (uint32_t)(sc * 64 + lane) * 4, 0,
         slot + (kBChunks + kAChunks) * 16 + (uint32_t)sc * 256);
  };
  constexpr int kLoads = kBDma + kADma + 1;
  // B's scales of 64 steps, lane l that of step l; the wavefront's rows are within one tile.
  const long long bt = min((j0 + wb * (kBR / kWB)) / kBlock, (a.n - 1) / kBlock);
  const float* b_scale = a.b_scale + bt * steps;
  float sb64 = lane < steps ? b_scale[lane] : 0.0f;
  asm volatile("" ::"v"(sb64));  // (landed before the loads that are counted)

  int fo[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) fo[h] = c16 * kRowChunks + ((4 * h + lane_chunk(quad)) ^ swz(c16));
  const int b_row = wb * (kBR / kWB) * kRowChunks, a_row = kBChunks + wa * (kAR / kWA) * kRowChunks;
  floatx4 acc[kBM][kAN];
#pragma unroll
  for (int bm = 0; bm < kBM; ++bm)
#pragma unroll
    for (int an = 0; an < kAN; ++an) acc[bm][an] = floatx4{};

#pragma unroll
  for (int p = 0; p < kSlots - 1; ++p)
    if (p < steps) load(p);
  for (int s = 0; s < steps; ++s) {
    // (past the end nothing is loaded, and fewer loads are in flight)
    if (s + kSlots - 2 < steps) wait_and_barrier<(kSlots - 2) * kLoads>();
    else wait_and_barrier<0>();
    if (s + kSlots - 1 < steps) load(s + kSlots - 1);
    if (s > 0 && (s & 63) == 0) {
      sb64 = s + lane < steps ? b_scale[s + lane] : 0.0f;
      asm volatile("" ::"v"(sb64));
    }
    const float sb = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(sb64), s & 63));
    const uint4* slot = smem + (s % kSlots) * kChunks;
    const float* scales = reinterpret_cast<const float*>(slot + kBChunks + kAChunks) + wa * (kAR / kWA) + c16;
    Operand<kOut> fa[kAN];
    float sc_ab[kAN];
#pragma unroll
    for (int an = 0; an < kAN; ++an) {
      fa[an].set(slot[a_row + an * 16 * kRowChunks + fo[0]], slot[a_row + an * 16 * kRowChunks + fo[1]]);
      sc_ab[an] = scales[an * 16] * sb;
    }
#pragma unroll
    for (int bm = 0; bm < kBM; ++bm) {
      Operand<kOut> fb;
      fb.set(slot[b_row + bm * 16 * kRowChunks + fo[0]], slot[b_row + bm * 16 * kRowChunks + fo[1]]);
      floatx4 p[kAN];
      Operand<kOut>::products(fb, fa, p);
#pragma unroll
      for (int an = 0; an < kAN; ++an)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[bm][an][i] = __builtin_fmaf(p[an][i], sc_ab[an], acc[bm][an][i]);
    }
  }
#pragma unroll
  for (int an = 0; an < kAN; ++an)
#pragma unroll
    for (int bm = 0; bm < kBM; ++bm)
      store4<kOut>(a, i0 + wa * (kAR / kWA) + an * 16 + c16, j0 + wb * (kBR / kWB) + bm * 16 + 4 * quad, acc[bm][an]);
}

template <int kOut, int kBR, int kAR, int kWB, int kWA, int kSlots>
void run_tiles(ProductArgs a, hipStream_t stream) {
  a.tiles_n = (int)ceil_div(a.n, kBR);
  a.tiles = ceil_div(a.m, kAR) * a.tiles_n;
  hipLaunchKernelGGL((product_tile_kernel<kOut, kBR, kAR, kWB, kWA, kSlots>), flat_grid(a.tiles), dim3(64 * kWB * kWA), 0, stream, a);
}

template <int kOut>
void run_product(const ProductArgs& a, hipStream_t stream) {
  run_tiles<kOut, 128, 128, 2, 2, 2>(a, stream);
}

}  // namespace

hipError_t launch_matmul_fp8_blocks(const MatmulFp8& c, hipStream_t stream) {
  const uintptr_t four = c.out_dtype == 0 ? 7 : 15;
  const ProductArgs a{c.A, c.B, c.a_scale, c.b_scale, c.C, c.m, c.n, (int)c.k, 0, 0,
                      c.n % 4 == 0 && (reinterpret_cast<uintptr_t>(c.C) & four) == 0};
  if (c.out_dtype == 0) run_product<0>(a, stream);
  else run_product<1>(a, stream);
  return hipGetLastError();
}

}  // namespace itl
