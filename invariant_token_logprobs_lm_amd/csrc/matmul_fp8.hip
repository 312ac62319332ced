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
// (The scales' product is an fp32 number, one per lane and 16 rows instead of a second
// product per sum: where it is subnormal a block's sum, below 2^25, meets up to
// 2^-150 of rounding: at most 2^-125 of C.)
//
// bf16 results: v_mfma_scale_f32_16x16x128_f8f6f4 (its own scales 1) takes a whole
// block of 16 rows of each operand. It adds the eight products of a lane's eight
// consecutive bytes with 13 bits below the largest (measured: a product 2^-14 of
// it is lost; the sixteen sums of eight are added in fp32), so p_b is off by 7 2^-13 of
// its products' absolute sum at worst, by 1e-6 to 4e-5 of itself on random operands, beside
// a bf16 result's 2^-9. Where the products cancel it is the products that count: with
// results 1 / 1800 of their products' sum, 300 x 500 x 2560 is off by 1.73e-3 of its norm,
// bf16's rounding alone by 1.66e-3.
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
#include "tile_engine8.h"

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
  long long scale_rows, c_cols;  // of a_scale and C: m and n, or more where these are some of them
  int k, tiles_n;
  long long tiles;
  bool quads;  // C's rows are whole fours of columns, aligned as such
  bool lines;  // C's rows are whole 16-byte pieces, aligned as such
  bool runs;   // a die's workgroups take consecutive tiles (see tiles_in_runs)
};

// Four consecutive columns of a row of C, aligned as such or not (1321 x 72281 x 128, fp32
// 99 to 104 us by 16-byte stores at any element; element by element twice the time).
template <int kOut, bool kAligned = true>
__device__ __forceinline__ void put4(typename Elem<kOut>::T* out, const floatx4& v) {
  using E = Elem<kOut>;
  std::conditional_t<kOut == 0, uint2, floatx4> w;
  if constexpr (kOut == 0)
    w = make_uint2((uint32_t)E::from_f(v[0]) | ((uint32_t)E::from_f(v[1]) << 16),
                   (uint32_t)E::from_f(v[2]) | ((uint32_t)E::from_f(v[3]) << 16));
  else
    w = v;
  if constexpr (kAligned) *reinterpret_cast<decltype(w)*>(out) = w;
  else __builtin_memcpy(out, &w, sizeof w);
}

// The same within C, of any alignment.
template <int kOut>
__device__ __forceinline__ void store4(const ProductArgs& a, long long row, long long col, const floatx4& v) {
  using E = Elem<kOut>;
  using T = typename E::T;
  if (row >= a.m || col >= a.n) return;
  T* out = static_cast<T*>(a.C) + row * a.c_cols + col;
  if (a.quads) return put4<kOut>(out, v);
  if (col + 4 <= a.n) return put4<kOut, false>(out, v);
#pragma unroll
  for (int i = 0; i < 3; ++i)
    if (col + i < a.n) out[i] = E::from_f(v[i]);
}

// Eight bf16 columns of a row within C, of any alignment.
__device__ __forceinline__ void store8(const ProductArgs& a, uint16_t* to, uint4 v, long long row, long long col) {
  if (row >= a.m || col >= a.n) return;
  if (a.lines) {
    *reinterpret_cast<uint4*>(to) = v;
    return;
  }
  if (col + 8 <= a.n) {
    __builtin_memcpy(to, &v, sizeof v);
    return;
  }
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 7; ++e)
    if (col + e < a.n) to[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
}

// Medium products, and all larger ones with fp32 results: kBR columns of C (rows of B) by
// kAR rows, a grid of kWB x kWA wavefronts, both operands through kSlots LDS slots loaded
// kSlots - kPer steps ahead, kPer steps per barrier.
//
// Few rows are bound by B's bytes: 16 x 129280 x 7168, fp32, 161 to 190 us (4.9 to 5.8 TB/s).
// Few steps are bound by latency: 777 x 1001 x 1536 7 to 8 us, 12 steps of 0.3 and the launch.
// Large fp32 results: 2048 x 8192 x 8192 (256 tiles of 256 x 256) 234 to 240 us, 1.15 PFLOP/s
// (the library's bf16 product reaches 1.31 to 1.46 at 8192 x 8192 x 8192); 2560 x 10240 x 16384
// 763 to 835 us (1.03 to 1.13). A step issues 5 cycles of vector instructions per 4 of the matrix
// cores, 3 of them conversions (two codes in 8 cycles). Widening each code once per
// workgroup and passing it on through LDS as bf16 (twice the LDS bytes, a second barrier a
// step) took 1071 us, where this took 857.
template <int kOut, int kBR, int kAR, int kWB, int kWA, int kSlots, int kPer = 1>
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
  const long long group = flat_group();
  if (group >= a.tiles) return;
  const int die = (int)(group & 7);  // consecutive workgroups go to the eight dies in turn
  const long long tile = a.runs ? die * (a.tiles >> 3) + min((long long)die, a.tiles & 7) + (group >> 3) : group;
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
    dma4(rsrc_words(a.a_scale + (size_t)s * a.scale_rows + i0, rows * 4), (uint32_t)(sc * 64 + lane) * 4, 0,
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

  auto multiply = [&](int s) {
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
  };
  // kPer steps per barrier, loaded kSlots - kPer steps ahead.
  constexpr int kAhead = kSlots - kPer;
#pragma unroll
  for (int p = 0; p < kAhead; ++p)
    if (p < steps) load(p);
  int s = 0;
  for (; s + kPer <= steps; s += kPer) {
    // (past the end nothing is loaded, and fewer loads are in flight)
    if (s + kAhead <= steps) wait_and_barrier<(kAhead - kPer) * kLoads>();
    else wait_and_barrier<0>();
#pragma unroll
    for (int p = 0; p < kPer; ++p)
      if (s + kAhead + p < steps) load(s + kAhead + p);
#pragma unroll
    for (int p = 0; p < kPer; ++p) multiply(s + p);
  }
  if constexpr (kPer > 1) {
    wait_and_barrier<0>();
    for (; s < steps; ++s) multiply(s);
  }
  if constexpr (kOut == 1) {
#pragma unroll
    for (int an = 0; an < kAN; ++an)
#pragma unroll
      for (int bm = 0; bm < kBM; ++bm)
        store4<kOut>(a, i0 + wa * (kAR / kWA) + an * 16 + c16, j0 + wb * (kBR / kWB) + bm * 16 + 4 * quad, acc[bm][an]);
  } else {
    // 16 rows of a wavefront at a time through LDS, so that a lane stores eight columns and
    // a row's are one stretch (264 x 94720 x 512 in 128 x 128 tiles 35 us, straight from the
    // registers 40; 389 x 12864 x 256 7.1 and 9). fp32 results, four columns a lane either
    // way, took longer through LDS (8192 x 8192 x 640: 117 us, 104 straight).
    constexpr int kRowBytes = kBM * 32, kPitch = kRowBytes + 16;   // (16 rows take kPitch chunks)
    constexpr int kPieces = kRowBytes / 16, kAtOnce = 64 / kPieces;  // 8 columns each; rows per store
    static_assert(16 % kAtOnce == 0 && kWaves * kPitch <= kSlots * kChunks, "within the slots");
    __syncthreads();  // (the last step's slot has been read)
    int ln = lane;
    asm volatile("" : "+v"(ln));  // (per-lane addresses formed here, not kept across the steps)
    char* turn = reinterpret_cast<char*>(smem + wave * kPitch);
    char* put = turn + (ln & 15) * kPitch + (ln >> 4) * 8;
    const char* get = turn + ln / kPieces * kPitch + ln % kPieces * 16;
    const long long row0 = i0 + wa * (kAR / kWA) + ln / kPieces, col = j0 + wb * (kBR / kWB) + ln % kPieces * 8;
#pragma unroll
    for (int an = 0; an < kAN; ++an) {
#pragma unroll
      for (int bm = 0; bm < kBM; ++bm) put4<0>(reinterpret_cast<uint16_t*>(put + bm * 32), acc[bm][an]);
#pragma unroll
      for (int r = 0; r < 16 / kAtOnce; ++r) {
        const uint4 v = *reinterpret_cast<const uint4*>(get + r * kAtOnce * kPitch);
        const long long row = row0 + an * 16 + r * kAtOnce;
        store8(a, static_cast<uint16_t*>(a.C) + row * a.c_cols + col, v, row, col);
      }
    }
  }
}

// 256 x 256 tiles for large products (bf16 results): eight wavefronts, each 128 columns of C by
// 64 rows, one workgroup per CU that walks its tiles without letting the loads
// run dry between them.
//
// Wavefronts w and w + 4 share a SIMD, so that one's waits lie under the other's
// instructions. A step is 32 of them. The first 16 take B's blocks 0 .. 3 one after
// the other against A's four, the last 16 A's blocks one after the other against
// B's 4 .. 7: each of the eight fragments in registers is refilled right after its
// last use, three instructions or more before its next. The step's last reads are
// under way after the first half, so its one barrier comes a little after that; it
// publishes the next step (loaded one step before) and frees this step's slot,
// whose loads for the step after next are spread over the second half. An
// instruction's sums are scaled into the accumulators three instructions later,
// when they are there.
//
// 16384 x 10240 x 2560 takes 390 to 420 us (2.05 to 2.2 PFLOP/s; the library's product of
// E4M3 matrices with one scale each reaches 2.77 at 8192 x 8192 x 8192). The matrix cores
// are busy 55 % of the cycles, vector instructions issue in 50 %, at 1.9 to 2.1 GHz: the
// busier they are, the lower the clock (8192 x 8192 x 8192: 61 % at 1.85). A tile's stores
// cost 3.6 us, which the next tile's second step waits for.
constexpr int kWide = 256;
constexpr int kWideRows = kWide * kRowChunks;          // chunks of an operand's rows of a step
constexpr int kWideSlot = 2 * kWideRows + 64 + 16;     // and A's 256 scales, B's two (of 64 lanes)
constexpr int kTurnPitch = 128 + 16;                   // bytes of a row of a wavefront's turned results
constexpr int kTurnChunks = 16 * kTurnPitch / 16;      // of 16 rows
constexpr int kCUs = 256;

// Tile t's place, in tiles. Four rows of tiles are walked together, column by
// column: the 32 tiles that a die works on at a time share 12 strips of operands.
__device__ __forceinline__ int2 wide_tile(int tiles_m, int tiles_n, int t) {
  const int band = t / (4 * tiles_n), in = t - band * 4 * tiles_n;
  const int rows = min(4, tiles_m - band * 4);
  const int j = in / rows;
  return make_int2(__builtin_amdgcn_readfirstlane(band * 4 + in - j * rows), __builtin_amdgcn_readfirstlane(j));
}

__global__ __launch_bounds__(kThreads8, 2) void product_wide_kernel(ProductArgs a) {
  __shared__ uint4 smem[2 * kWideSlot + 8 * kTurnChunks];
  const Lanes8 L = lanes8();
  const int lane = L.lane, quad = L.quad, c16 = L.c16;
  const int steps = a.k / kBlock;
  // A die (every eighth workgroup) has a run of consecutive tiles, its workgroups
  // take them in turn.
  const int die = blockIdx.x & 7, seats = gridDim.x >> 3;
  const int tiles = (int)a.tiles, tiles_m = (int)((a.m + kWide - 1) / kWide);
  const int t_end = (int)((long long)tiles * (die + 1) / 8);
  int t = (int)((long long)tiles * die / 8) + (blockIdx.x >> 3);
  if (t >= t_end) return;

  const int lr = lane >> 3;
  uint32_t voff[kDma8PerWave];
#pragma unroll
  for (int j = 0; j < kDma8PerWave; ++j)
    voff[j] = (uint32_t)(L.wave * 32 + j * kDmaRows + lr) * (uint32_t)a.k + (((lane & 7) ^ lr ^ (j & 1)) * 16);
  const uint32_t lds0 = (uint32_t)(size_t)((__attribute__((address_space(3))) uint4*)smem);
  const uint32_t my_rows = (uint32_t)L.wave * 32 * kStepBytes;
  // Wavefronts 0 .. 3 fetch 64 of A's scales each, the others B's two (all four the
  // same ones; lanes past the two lie past the range).
  const bool of_a = L.wave < 4;
  const uint32_t scale_off = of_a ? (uint32_t)(L.wave * 64 + lane) * 4u : lane < 2 ? (uint32_t)(lane * steps) * 4u : 0x80000000u;
  const uint32_t scale_lds = 2 * kWideRows * 16 + (of_a ? (uint32_t)L.wave * 256u : 1024u);
  const uint64_t scale_step = of_a ? (uint64_t)a.scale_rows * 4 : 4;
  // A tile's operands and scales. With no tile the ranges are empty: zeros are
  // written into slots that nothing reads.
  struct Source {
    uint64_t b, a, scale;
    uint32_t b_bytes, a_bytes, scale_bytes;
  };
  auto source = [&](int2 at, bool any) {
    const long long i0 = (long long)at.x * kWide, j0 = (long long)at.y * kWide;
    const uint32_t rows = (uint32_t)min((long long)kWide, a.m - i0), cols = (uint32_t)min((long long)kWide, a.n - j0);
    const uint32_t tiles_b = cols > kBlock ? 2 : 1;
    Source f;
    f.b = (uint64_t)a.B + (uint64_t)j0 * (uint32_t)a.k;
    f.a = (uint64_t)a.A + (uint64_t)i0 * (uint32_t)a.k;
    f.scale = of_a ? (uint64_t)(a.a_scale + i0) : (uint64_t)(a.b_scale + (uint64_t)(2 * at.y) * (uint32_t)steps);
    f.b_bytes = any ? cols * (uint32_t)a.k : 0;
    f.a_bytes = any ? rows * (uint32_t)a.k : 0;
    f.scale_bytes = any ? (of_a ? rows : tiles_b * (uint32_t)steps) * 4u : 0;
    return f;
  };
  // The loads' own walk over the steps, two ahead: with three steps or more, in the
  // next tile at most. (No branch: a step is one block, whose order stands as written.)
  int2 at = wide_tile(tiles_m, a.tiles_n, t);
  Source from = source(at, true), ahead = from;
  int ld_s = 0;
  auto words = [](uint64_t base, uint32_t bytes) {
    return int4v{(int)(uint32_t)base, (int)((uint32_t)(base >> 32) & 0xffffu), (int)bytes, 0x00020000};
  };
  auto load = [&](int slot, int j) {  // the j-th of a step's nine loads
    const uint32_t base = lds0 + (uint32_t)slot * kWideSlot * 16;
    if (j < 4) {
      dma16(words(from.b, from.b_bytes), voff[j & 3], (uint32_t)ld_s * kBlock, base + my_rows + j * 1024);
    } else if (j < 8) {
      dma16(words(from.a, from.a_bytes), voff[j & 3], (uint32_t)ld_s * kBlock, base + kWideRows * 16 + my_rows + (j & 3) * 1024);
    } else {
      dma4(words(from.scale, from.scale_bytes), scale_off, 0, base + scale_lds);
      const bool last = ld_s + 1 == steps;
      ld_s = last ? 0 : ld_s + 1;
      from.b = last ? ahead.b : from.b;
      from.a = last ? ahead.a : from.a;
      from.scale = last ? ahead.scale : from.scale + scale_step;
      from.b_bytes = last ? ahead.b_bytes : from.b_bytes;
      from.a_bytes = last ? ahead.a_bytes : from.a_bytes;
      from.scale_bytes = last ? ahead.scale_bytes : from.scale_bytes;
    }
  };
  auto load_all = [&](int slot) {
#pragma unroll
    for (int j = 0; j < 9; ++j) load(slot, j);
  };

  int b_off[2], a_off[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int pc = (4 * h + lane_chunk(quad)) ^ swz(c16);
    b_off[h] = (L.wv * 128 + c16) * kRowChunks + pc;
    a_off[h] = kWideRows + (L.tq * 64 + c16) * kRowChunks + pc;
  }
  Frag8 FB[4], FA[4];
  float xs[4], sb;
  auto read_b = [&](int slot, int bm) {
    FB[bm & 3].lo = smem[slot * kWideSlot + b_off[0] + bm * 16 * kRowChunks];
    FB[bm & 3].hi = smem[slot * kWideSlot + b_off[1] + bm * 16 * kRowChunks];
  };
  auto read_a = [&](int slot, int an) {
    FA[an].lo = smem[slot * kWideSlot + a_off[0] + an * 16 * kRowChunks];
    FA[an].hi = smem[slot * kWideSlot + a_off[1] + an * 16 * kRowChunks];
  };
  auto read_scales = [&](int slot) {
    const float* f = reinterpret_cast<const float*>(smem + slot * kWideSlot + 2 * kWideRows);
#pragma unroll
    for (int an = 0; an < 4; ++an) xs[an] = f[L.tq * 64 + an * 16 + c16];
    sb = f[256 + L.wv];
  };
  floatx4 acc[8][4];
  constexpr int kLag = 3;  // instructions between one and the use of its result
  // One step. kNext: the next step's first fragments are read in it (not in a
  // tile's last: they are read after its results are stored). kPending: loads and
  // stores issued after the next step's loads that may be in flight at the barrier.
  auto step = [&](auto next, auto pending, int slot) {
    floatx4 R[32];
    float sab[4];
#pragma unroll
    for (int an = 0; an < 4; ++an) sab[an] = xs[an] * sb;
    auto place = [](int i) { return i < 16 ? make_int2(i >> 2, i & 3) : make_int2(4 + (i & 3), (i - 16) >> 2); };
    auto scale = [&](int i) {
      const int2 at = place(i);
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[at.x][at.y][e] = __builtin_fmaf(R[i][e], sab[at.y], acc[at.x][at.y][e]);
    };
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const int2 at = place(i);
      R[i] = floatx4{};
      mma_f8_16(R[i], FB[at.x & 3], FA[at.y]);
      if (i >= kLag) scale(i - kLag);
      if (i < 16 && (i & 3) == 3) read_b(slot, 4 + (i >> 2));
      if (i == 19) wait_and_barrier<decltype(pending)::value>();
      if (i >= 20 && i < 29) load(slot, i - 20);
      if constexpr (decltype(next)::value) {
        if (i >= 19 && (i & 3) == 3) read_a(slot ^ 1, (i - 19) >> 2);
        if (i >= 28) read_b(slot ^ 1, i - 28);
        if (i == 27) read_scales(slot ^ 1);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int i = 32 - kLag; i < 32; ++i) scale(i);
    __builtin_amdgcn_sched_barrier(0);
  };
  auto read_first = [&](int slot) {
    read_scales(slot);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      read_b(slot, i);
      read_a(slot, i);
    }
  };
  using Yes = std::true_type;
  using No = std::false_type;
  constexpr int kStores = 16;  // of a whole tile, per wavefront
  using AfterStores = std::integral_constant<int, kStores>;
  using None = std::integral_constant<int, 0>;

  load_all(0);
  load_all(1);
  wait_and_barrier<0>();
  int slot = 0;
  for (;;) {
    const bool more = t + seats < t_end;
    const int2 to = more ? wide_tile(tiles_m, a.tiles_n, t + seats) : at;
    ahead = source(to, more);
    read_first(slot);
#pragma unroll
    for (int bm = 0; bm < 8; ++bm)
#pragma unroll
      for (int an = 0; an < 4; ++an) acc[bm][an] = floatx4{};
    // (the tile before has left at most its stores behind this one's loads)
    step(Yes{}, AfterStores{}, slot);
    slot ^= 1;
    for (int s = 1; s + 1 < steps; ++s, slot ^= 1) step(Yes{}, None{}, slot);
    step(No{}, None{}, slot);
    slot ^= 1;
    // (the last step stays before the branches below, which its results alone would sink into)
#pragma unroll
    for (int bm = 0; bm < 8; ++bm)
#pragma unroll
      for (int an = 0; an < 4; ++an) asm volatile("" : "+v"(acc[bm][an]));
    int ln = lane;
    asm volatile("" : "+v"(ln));  // (per-lane addresses formed here, not kept across the steps)
    // 16 rows by 64 columns at a time through LDS, so that whole 128-byte lines are
    // written (8 bytes per lane in 32-byte pieces took twice as long)
    char* turn = reinterpret_cast<char*>(smem + 2 * kWideSlot + L.wave * kTurnChunks);
    char* put = turn + (ln & 15) * kTurnPitch + (ln >> 4) * 8;
    const char* get = turn + (ln >> 3) * kTurnPitch + (ln & 7) * 16;
    const long long row0 = (long long)at.x * kWide + L.tq * 64 + (ln >> 3), col0 = (long long)at.y * kWide + L.wv * 128 + (ln & 7) * 8;
    uint16_t* out = static_cast<uint16_t*>(a.C) + row0 * a.c_cols + col0;
    const bool whole = a.lines && (long long)(at.x + 1) * kWide <= a.m && (long long)(at.y + 1) * kWide <= a.n;
#pragma unroll
    for (int an = 0; an < 4; ++an) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
#pragma unroll
        for (int b = 0; b < 4; ++b) put4<0>(reinterpret_cast<uint16_t*>(put + b * 32), acc[4 * half + b][an]);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint4 v = *reinterpret_cast<const uint4*>(get + r * 8 * kTurnPitch);
          uint16_t* to = out + (an * 16 + r * 8) * a.c_cols + half * 64;
          if (whole) *reinterpret_cast<uint4*>(to) = v;
          else store8(a, to, v, row0 + an * 16 + r * 8, col0 + half * 64);
        }
      }
    }
    if (!whole) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // (how many there were is not known)
    if (!more) break;
    t += seats;
    at = to;
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // (no load into LDS outlives the workgroup)
}

void run_wide(ProductArgs a, hipStream_t stream) {
  a.tiles_n = (int)ceil_div(a.n, kWide);
  a.tiles = ceil_div(a.m, kWide) * a.tiles_n;
  hipLaunchKernelGGL((product_wide_kernel), dim3((unsigned)std::min<long long>(ceil_div(a.tiles, 8) * 8, kCUs)), dim3(kThreads8), 0, stream, a);
}

// Whether a die's workgroups take consecutive tiles: where C's rows do not start at whole
// 128-byte lines, tiles side by side share lines, and a line written by two dies goes to
// memory in two pieces. fp32 results: 1321 x 72281 x 128 99 us, tiles in turn 112; 882 x 72178 x
// 640, bound by more steps, 126 and 124; 2000 x 10001 x 4096 166 and 166; rows of whole lines
// 8192 x 8192 x 640 113 and 104. bf16 results: 4000 x 20001 x 256 58 and 62; 1000 x 5001 x 512
// 9.5 and 10.0, x 1024, more bound by its steps, 13.7 and 13.0.
template <int kOut>
bool tiles_in_runs(const ProductArgs& a) {
  return a.c_cols * Elem<kOut>::kSize % 128 != 0 && (kOut == 1 || a.k <= 4 * kBlock);
}

template <int kOut, int kBR, int kAR, int kWB, int kWA, int kSlots, int kPer = 1>
void run_tiles(ProductArgs a, hipStream_t stream) {
  a.tiles_n = (int)ceil_div(a.n, kBR);
  a.tiles = ceil_div(a.m, kAR) * a.tiles_n;
  a.runs = tiles_in_runs<kOut>(a);
  hipLaunchKernelGGL((product_tile_kernel<kOut, kBR, kAR, kWB, kWA, kSlots, kPer>), flat_grid(a.tiles), dim3(64 * kWB * kWA), 0, stream, a);
}

// Small products, however long the contraction: tiles of 16 kBM columns by 16 kAN
// rows of C, whose blocks a workgroup's eight wavefronts share, straight from memory
// into registers, so that many loads are under way with few tiles. A block's
// unscaled sums go to LDS, and each element's chain over the blocks is then walked
// in order by one thread: the bits of the other kernels. kHeld blocks of a wavefront
// are loaded at a time, the next ones while the chain is walked.
constexpr int kFewWaves = 8;

template <int kOut, int kBM, int kAN>
__global__ __launch_bounds__(64 * kFewWaves) void product_few_kernel(ProductArgs a) {
  constexpr int kHeld = 8 / (kBM * kAN), kRound = kHeld * kFewWaves;  // blocks of a round
  constexpr int kEach = kBM * kAN * 256 / (64 * kFewWaves) > 0 ? kBM * kAN * 256 / (64 * kFewWaves) : 1;  // elements per thread
  static_assert(kHeld >= 1, "a wavefront holds a block at least");
  __shared__ floatx4 part[kRound][kBM * kAN][64];
  __shared__ float scales[kRound][16 * kAN];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int quad = lane >> 4, c16 = lane & 15;
  const long long group = flat_group();
  if (group >= a.tiles) return;
  const long long i0 = group / a.tiles_n * 16 * kAN, j0 = group % a.tiles_n * 16 * kBM;
  const int blocks = a.k / kBlock;
  const int at0 = lane_chunk(quad) * 16, at1 = (4 + lane_chunk(quad)) * 16;
  const float* b_scale = a.b_scale + j0 / kBlock * blocks;

  uint4 vb[kHeld][kBM][2], va[kHeld][kAN][2];
  auto load = [&](int first) {
#pragma unroll
    for (int h = 0; h < kHeld; ++h) {
      const int b = first + h * kFewWaves + wave;
#pragma unroll
      for (int i = 0; i < kBM; ++i) {
        const long long row = j0 + 16 * i + c16;
        const uint8_t* p = a.B + row * a.k + (long long)b * kBlock;
        const bool in = b < blocks && row < a.n;
        vb[h][i][0] = in ? *reinterpret_cast<const uint4*>(p + at0) : make_uint4(0u, 0u, 0u, 0u);
        vb[h][i][1] = in ? *reinterpret_cast<const uint4*>(p + at1) : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int i = 0; i < kAN; ++i) {
        const long long row = i0 + 16 * i + c16;
        const uint8_t* p = a.A + row * a.k + (long long)b * kBlock;
        const bool in = b < blocks && row < a.m;
        va[h][i][0] = in ? *reinterpret_cast<const uint4*>(p + at0) : make_uint4(0u, 0u, 0u, 0u);
        va[h][i][1] = in ? *reinterpret_cast<const uint4*>(p + at1) : make_uint4(0u, 0u, 0u, 0u);
      }
    }
  };
  // Element e of this thread: float (64 kFewWaves e + threadIdx.x) of a block's sums.
  float acc[kEach];
#pragma unroll
  for (int e = 0; e < kEach; ++e) acc[e] = 0.0f;

  load(0);
  for (int first = 0; first < blocks; first += kRound) {
    for (int i = threadIdx.x; i < kRound * 16 * kAN; i += 64 * kFewWaves) {
      const int b = first + i / (16 * kAN);
      const long long row = i0 + i % (16 * kAN);
      (&scales[0][0])[i] = b < blocks && row < a.m ? a.a_scale[b * a.scale_rows + row] * b_scale[b] : 0.0f;
    }
#pragma unroll
    for (int h = 0; h < kHeld; ++h) {
      Operand<kOut> fa[kAN];
#pragma unroll
      for (int i = 0; i < kAN; ++i) fa[i].set(va[h][i][0], va[h][i][1]);
#pragma unroll
      for (int j = 0; j < kBM; ++j) {
        Operand<kOut> fb;
        fb.set(vb[h][j][0], vb[h][j][1]);
        floatx4 p[kAN];
        Operand<kOut>::products(fb, fa, p);
#pragma unroll
        for (int i = 0; i < kAN; ++i) part[h * kFewWaves + wave][j * kAN + i][lane] = p[i];
      }
    }
    if (first + kRound < blocks) load(first + kRound);
    __syncthreads();
    const int count = min(kRound, blocks - first);
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int f = 64 * kFewWaves * e + threadIdx.x;
      if (f < kBM * kAN * 256) {
        const float* p = reinterpret_cast<const float*>(part) + f;
        const float* s = &scales[0][16 * ((f >> 8) % kAN) + ((f >> 2) & 15)];
#pragma unroll 8
        for (int b = 0; b < count; ++b) acc[e] = __builtin_fmaf(p[b * kBM * kAN * 256], s[b * 16 * kAN], acc[e]);
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int f = 64 * kFewWaves * e + threadIdx.x, which = f >> 8;
    const long long row = i0 + 16 * (which % kAN) + ((f >> 2) & 15), col = j0 + 16 * (which / kAN) + 4 * ((f >> 6) & 3) + (f & 3);
    if (f < kBM * kAN * 256 && row < a.m && col < a.n)
      static_cast<typename Elem<kOut>::T*>(a.C)[row * a.c_cols + col] = Elem<kOut>::from_f(acc[e]);
  }
}

template <int kOut, int kBM, int kAN>
void run_few(ProductArgs a, hipStream_t stream) {
  a.tiles_n = (int)ceil_div(a.n, 16 * kBM);
  a.tiles = ceil_div(a.m, 16 * kAN) * a.tiles_n;
  hipLaunchKernelGGL((product_few_kernel<kOut, kBM, kAN>), flat_grid(a.tiles), dim3(64 * kFewWaves), 0, stream, a);
}

// Rows first .. first + count of a product.
ProductArgs rows_of(ProductArgs a, long long first, long long count, size_t elem) {
  a.A += first * a.k;
  a.a_scale += first;
  a.C = static_cast<char*>(a.C) + (size_t)first * a.c_cols * elem;
  a.m = count;
  return a;
}

// Columns first .. first + count, first a multiple of 128.
ProductArgs columns_of(ProductArgs a, long long first, long long count, size_t elem) {
  a.B += first * a.k;
  a.b_scale += first / kBlock * (a.k / kBlock);
  a.C = static_cast<char*>(a.C) + (size_t)first * elem;
  a.n = count;
  return a;
}

// Which kernel: all give the same bits. us measured on both sides of each border
// (bf16 results where not said otherwise; m x n x k; operands of normally distributed values).
template <int kOut>
void run_product(const ProductArgs& a, hipStream_t stream) {
  auto tiles = [&](int cols, int rows) { return ceil_div(a.n, cols) * ceil_div(a.m, rows); };
  // No more tiles of 16 to 64 columns by 16 or 32 rows than CUs (the smallest that are
  // so few: larger ones read less): the wavefronts share the blocks. 16 x 2560 x 7168
  // 10.0, in 64 x 64 tiles 20.3; 16 x 10240 x 7168 19.5 and 21.1; 16 x 20480 x 7168
  // 35.6 and 26.7; 128 x 2048 x 16384 35.5 and 43.8; 256 x 2048 x 16384 63.2 and 44.2.
  if (tiles(16, 16) <= kCUs) return run_few<kOut, 1, 1>(a, stream);
  if (tiles(32, 16) <= kCUs) return run_few<kOut, 2, 1>(a, stream);
  if (a.m <= 16 && tiles(64, 16) <= kCUs) return run_few<kOut, 4, 1>(a, stream);
  if (a.m > 16 && tiles(32, 32) <= kCUs) return run_few<kOut, 2, 2>(a, stream);
  // Rows or columns whose tiles fill the CUs a whole number of times, and what is left: a few
  // tiles more than whole rounds take as long as another round, or a third of it in smaller
  // tiles of their own. 6000 x 3000 x 7168 (288 tiles of 256 x 256) 145, all in those 186.
  // Columns where they leave a tenth less, in tiles of 128 x 128: 300 x 70000 x 4096 (by columns
  // 36 of 548 tiles, by rows none whole) 145 and 170, 4096 x 4200 x 4096, fp32 (32 of those and
  // 66) 142 and 150; 2560 x 10240 x 16384, fp32 (600 and 640) 797 and 785.
  struct Rounds {
    long long rounds, rows, columns, left;  // whole rounds, their rows and columns, the tiles left
  };
  auto rounds_of = [&](int size, long long at_once) {
    const long long across = ceil_div(a.n, size), down = ceil_div(a.m, size), all = tiles(size, size);
    const long long rounds = all / at_once, fit = rounds * at_once;
    const long long rows = fit / across * size, columns = fit / down * size;
    const long long rows_left = ceil_div(std::max(a.m - rows, 0LL), 128) * ceil_div(a.n, 128);
    const long long columns_left = ceil_div(std::max(a.n - columns, 0LL), 128) * ceil_div(a.m, 128);
    if (10 * columns_left > 9 * rows_left) return Rounds{rounds, rows, a.n, all - fit / across * across};
    return Rounds{rounds, a.m, columns, all - fit / down * down};
  };
  auto split = [&](const Rounds& r, double most_left, auto&& run) {
    constexpr size_t elem = Elem<kOut>::kSize;
    if (r.rows == 0 || r.columns == 0 || r.left == 0 || r.left > most_left) return run(a);
    if (r.rows < a.m) {
      run(rows_of(a, 0, r.rows, elem));
      run_product<kOut>(rows_of(a, r.rows, a.m - r.rows, elem), stream);
    } else {
      run(columns_of(a, 0, r.columns, elem));
      run_product<kOut>(columns_of(a, r.columns, a.n - r.columns, elem), stream);
    }
  };
  const double steps = (double)(a.k / kBlock);
  // More than half the CUs with a 256 x 256 tile: 2048 x 5120 x 4096 (160 tiles) 52, in
  // 128 x 128 tiles 60; 2048 x 4096 x 4096 (128) 50 and 42.
  // (Left over: a step of a round takes 1.6 us, one of `left` tiles as smaller ones 0.45 +
  // 0.0125 left, and 4 us once.)
  if constexpr (kOut == 0) {
    if (a.m > 128 && a.k >= 3 * kBlock && tiles(kWide, kWide) > kCUs / 2)
      return split(rounds_of(kWide, kCUs), (1.1 - 4.0 / steps) / 0.0125, [&](const ProductArgs& p) { run_wide(p, stream); });
  }
  // Tiles of 64 x 64, two steps per barrier while they run at once, two per CU: 512 x 2048 x
  // 7168 (256) 22.1, with one step 28.8; 196 x 1996 x 9472 (128) 26.7 and 34.9; 1024 x 2560 x
  // 2560 (640) 18.8 and 15.9, in 64 x 128 tiles 17.0; 1280 x 2560 x 7936 (800) 52.0, in 64 x
  // 128 tiles 45.1; 1024 x 4000 x 4096 (1008) 36.6 and 28.2.
  if (tiles(64, 64) <= 2 * kCUs) return run_tiles<kOut, 64, 64, 2, 2, 4, 2>(a, stream);
  if (tiles(64, 64) <= 3 * kCUs) return run_tiles<kOut, 64, 64, 2, 2, 2>(a, stream);
  // Many columns for few rows are a matter of B's bytes: 64 x 61440 x 7168 82.9 in tiles
  // of 128 columns, 95.5 of 64.
  if (a.m <= 64) return run_tiles<kOut, 128, 64, 2, 2, 3>(a, stream);
  // bf16 results: 128 x 128 tiles (of eight wavefronts, two workgroups per CU; of four
  // 2 to 15 % slower) where there are more than CUs: 1024 x 5000 x 4096 (320) 34.2, in 64 x
  // 128 tiles 39.2; 128 x 61440 x 7168 (480) 101 and 141; 1500 x 2600 x 4096 (252) 28.0 and 28.0.
  if constexpr (kOut == 0) {
    if (tiles(128, 128) > kCUs) return run_tiles<kOut, 128, 128, 2, 4, 2>(a, stream);
  }
  // fp32 results: 128 x 128, 64 x 128 or 256 x 256 tiles, of the last the whole rounds at
  // least, whichever end sooner. A step of a round takes 3.2 us with 256 x 256, 2.0 with two
  // of 128 x 128 per CU, 1.2 with one, 0.62 a 64 x 128 tile per CU, and 0.5 + 0.0025 left
  // where 128 x 128 tiles left over become smaller ones; another launch 4.
  // 2048 x 4096 x 4096 in 128 x 128 (512 tiles) 75, in 64 x 128 86; 900 x 5000 x 2560 (320) 42.9
  // and 39.3; 8960 x 1536 x 16384 (210 tiles of 256 x 256) 418, in 128 x 128 tiles 519; 4096 x
  // 4200 x 4096 (256 and 16) 142, all in one size 222 or 172; 2560 x 10240 x 16384 (240 and 160)
  // 835, 852 or 919; 2048 x 10240 x 7168 (256 and 64) 285, 385 or 307.
  if constexpr (kOut == 1) {
    const double most_left = (0.5 - 4.0 / steps) / 0.0025;
    auto in128 = [&](long long n, bool smaller) {  // n tiles of 128 x 128, those left over smaller or not
      const long long over = n % (2 * kCUs);
      return n / (2 * kCUs) * 2.0 + (over == 0 ? 0.0 : smaller && over <= most_left ? 0.5 + 0.0025 * over : over <= kCUs ? 1.2 : 2.0);
    };
    const Rounds r = rounds_of(128, 2 * kCUs), w = rounds_of(kWide, kCUs);
    const double all128 = std::min(in128(tiles(128, 128), false), r.rounds * 2.0 + in128(r.left, r.rounds > 0));
    const double all64 = ceil_div(tiles(64, 128), kCUs) * 0.62;
    const double all256 = ceil_div(tiles(kWide, kWide), kCUs) * 3.2;
    const double parts = w.rounds > 0 ? w.rounds * 3.2 + in128(4 * w.left, true) + 4.0 / steps : all256;
    if (std::min(all256, parts) < std::min(all128, all64))
      return split(w, parts < all256 ? w.left : 0, [&](const ProductArgs& p) { run_tiles<kOut, 256, 256, 2, 4, 2>(p, stream); });
    if (all128 < all64)
      return split(r, most_left, [&](const ProductArgs& p) { run_tiles<kOut, 128, 128, 2, 4, 2>(p, stream); });
  }
  run_tiles<kOut, 64, 128, 2, 2, 2>(a, stream);
}

}  // namespace

hipError_t launch_matmul_fp8_blocks(const MatmulFp8& c, hipStream_t stream) {
  const uintptr_t four = c.out_dtype == 0 ? 7 : 15;
  const ProductArgs a{c.A, c.B, c.a_scale, c.b_scale, c.C, c.m, c.n, c.m, c.n, (int)c.k, 0, 0,
                      c.n % 4 == 0 && (reinterpret_cast<uintptr_t>(c.C) & four) == 0,
                      c.n % (c.out_dtype == 0 ? 8 : 4) == 0 && (reinterpret_cast<uintptr_t>(c.C) & 15) == 0, false};
  if (c.out_dtype == 0) run_product<0>(a, stream);
  else run_product<1>(a, stream);
  return hipGetLastError();
}

}  // namespace itl
