// Cross entropy over the vocabulary and its gradient, through the LM head,
// for the tokens that count.
//
//   z[t, v] = sum_k H[t, k] W[v, k]            fp32 accumulate
//   lse[t]  = log sum_v exp(z[t, v])
//   l[t]    = (1 - e) (lse - z[t, y_t]) + e (lse - mean_v z[t, v]) + lam lse^2
//   loss    = (1 / N) sum_t l[t]               over the N tokens with 0 <= y_t < V
//   G[t, v] = s / N ((1 + 2 lam lse) p[t, v] - (1 - e) [v = y_t] - e / V),  p = exp(z - lse)
//   dH = G W,  dW = G^T H
//
// The logits exist for one chunk of kCeChunk tokens at a time, in the
// workspace. A token whose id is outside [0, V) costs nothing beyond the
// loads of its id: the counted tokens' rows of H are gathered first (their
// number stays on the device; workgroups past it leave at once), and every
// contraction runs over them alone.
//
// With the gradient, for each chunk:
//   1. z = H W^T, kept in fp32: bf16 heads by the logprob forward's
//      contraction and online log-sum-exp folds (the same bits; without the
//      gradient nothing is kept), fp32 heads by 64 x 64 tiles and a pass over
//      z for the log-sum-exp;
//   2. G [chunk, Vpad] in the head's type, like z in blocks of 256 vocabulary
//      entries (all tokens of a block side by side): a tile's rows are then
//      one piece of memory, for its writer and for both contractions;
//   3. dH = G W, K = the vocabulary, split over several workgroups when the
//      chunk has few tiles (fp32 partials added in order);
//   4. dW += G^T H, K = the chunk's tokens.
// 3 and 4 read W, G and H as they lie (tile_engine_km.h): no transposed copy.
// That is three contractions, the least there is (keeping the logits saves
// the fourth: the 8 bytes written and read per logit of z cost less than a
// contraction of 2 d operations each for d > about 1000, the widths here).
//
// Bound by the matrix cores for many tokens: 4096 tokens, three quarters of
// them counted, d = 2560, V = 151936, bf16 take 6.5 ms (forward 2.05, dH 1.88,
// dW 2.08: 1.15 to 1.27 PFLOP/s; G from z 0.52 at 5.4 TB/s), 2188 of 2500, d =
// 7168, V = 129280 11.3 ms. Bound by reading W for few: the loss of 64 tokens, d = 1536, V = 151936
// takes 109 us, 99 of them W at 4.7 TB/s.
//
// Every sum has a fixed order and there are no atomics: token losses depend
// on the token alone, the loss and the gradients are run-to-run
// deterministic.

#include <algorithm>

#include "itl_launch.h"
#include "learner_common.h"
#include "logit_store.h"
#include "lse_fold.h"
#include "tile_engine.h"
#include "tile_engine8.h"
#include "tile_engine_km.h"

namespace itl {

namespace {

constexpr int kCeChunk = 16384;    // tokens per chunk with the gradient (a multiple of kBT)
constexpr int kCeF32Chunk = 4096;  // the same of fp32 heads without it (their logits are kept too)
// bf16 heads without it: the forward's workgroups of 512 threads, up to 256 per
// 256 tokens, and the merge's 16 threads per token then fit a grid dimension
constexpr int kCeLossChunk = 1 << 22;
static_assert(kCeChunk % kBT == 0, "chunks hold whole token blocks");

long long round_up(long long x, long long m) { return (x + m - 1) / m * m; }

// Tiles of the gradient's contractions: 256 x 256 (bf16), 64 x 64 (fp32); K
// steps of 128 bytes.
template <int kDtype>
struct GradTile {
  static constexpr int kRows = kDtype == 0 ? 256 : kF32Tile;
  static constexpr int kStepK = kStepBytes / Elem<kDtype>::kSize;
};

// Workgroups that share the K steps of a tile of dH or dW (each at least 4
// steps): the count that takes the fewest K steps of time, rounds over the CUs
// x steps per workgroup, beside each round's start and end (12 steps' worth)
// and the fp32 partials' traffic (a step's time moves those of about 8 tiles;
// of a single block of tokens, its `rows` of `tile` only). fp32: three
// workgroups fit a CU and share its matrix cores; one alone waits for its loads
// (a step takes 1.6 times as long), starts and ends overlap, and the partials
// are a sixteenth.
struct KSplits {
  uint32_t tiles, nks, rows, tile;
  bool f32;
  // a single block's partials are few: more splits pay
  __host__ __device__ uint32_t most() const { return tiles == 0 ? 1 : rows <= tile ? 64 : 16; }
  __host__ __device__ bool may(uint32_t s) const { return s == 1 || (s <= most() && nks >= 4 * s); }
  __host__ __device__ uint32_t cost(uint32_t s) const {
    const uint32_t rounds = (tiles * s + 255) / 256, steps = (nks + s - 1) / s;
    const uint32_t part = rows < tile ? s * tiles * rows / tile : s * tiles;
    return f32 ? rounds * (steps + 4) + (rounds == 1 ? steps * 3 / 5 : 0) + part / 64 : rounds * (steps + 12) + part / 8;
  }
};

inline int k_splits(const KSplits& k) {
  uint32_t best = 1, least = 0xffffffffu;
  for (uint32_t s = 1; k.may(s); ++s) {
    const uint32_t cost = k.cost(s);
    if (cost < least) best = s, least = cost;
  }
  return (int)best;
}

// The same by a wavefront, a count per lane.
__device__ __forceinline__ int k_splits_wave(const KSplits& k) {
  const uint32_t s = (threadIdx.x & 63) + 1;
  uint64_t key = ((uint64_t)(k.may(s) ? k.cost(s) : 0xffffffffu) << 32) | s;
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) {
    const uint64_t other = (uint64_t)__shfl_xor((unsigned long long)key, off, 64);
    key = other < key ? other : key;
  }
  return (int)(uint32_t)key;
}

// dH's: `live` rows of G in blocks of `tile`, n_dt tiles of d. A single
// block's rows count in quarters of it.
__host__ __device__ inline KSplits dh_split_sizes(uint32_t live, uint32_t n_dt, uint32_t nks, bool f32, uint32_t tile) {
  const uint32_t quarter = tile / 4;
  const uint32_t rows = (live + quarter - 1) / quarter * quarter;
  return KSplits{(live + tile - 1) / tile * n_dt, nks, rows, tile, f32};
}

// Place of (token row t, vocabulary entry v) in a blocked array of `rows`
// token rows: blocks of kBV entries.
__host__ __device__ inline size_t block_at(int t, int v, int rows) {
  return ((size_t)(v / kBV) * rows + t) * kBV + v % kBV;
}

// ---- which tokens count

// One workgroup: rows[j] = the j-th counted token, ids[j] its target,
// slot[t] = token t's place j or -1; *count = N; and each chunk's dH splits.
constexpr int kSelectThreads = 1024;
__global__ __launch_bounds__(kSelectThreads) void ce_select_kernel(const int32_t* __restrict__ targets, int n, int vocab,
                                                                   int32_t* __restrict__ rows, int32_t* __restrict__ ids,
                                                                   int32_t* __restrict__ slot, int32_t* __restrict__ count,
                                                                   int32_t* __restrict__ splits, int chunk, int rows_per_tile,
                                                                   int parts, int n_dt, int nks, int f32) {
  __shared__ int wave_n[kSelectThreads / 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int base = 0;
  for (long long t0 = 0; t0 < n; t0 += kSelectThreads) {
    const long long t = t0 + threadIdx.x;
    const int y = t < n ? targets[t] : -1;
    const bool in = (unsigned)y < (unsigned)vocab;
    const uint64_t mask = __ballot(in);
    if (lane == 0) wave_n[wave] = __popcll(mask);
    __syncthreads();
    int before = base;
    for (int w = 0; w < kSelectThreads / 64; ++w) {
      if (w < wave) before += wave_n[w];
      base += wave_n[w];
    }
    const int j = before + __popcll(mask & ((1ull << lane) - 1ull));
    if (in) {
      rows[j] = (int)t;
      ids[j] = y;
    }
    if (t < n) slot[t] = in ? j : -1;
    __syncthreads();
  }
  if (threadIdx.x == 0) *count = base;
  // dH's splits of every chunk, a wavefront each
  if (splits)
    for (int c = wave; (long long)c * chunk < n; c += kSelectThreads / 64) {
      const int live = parts * max(0, min(base - c * chunk, chunk));
      const int s = k_splits_wave(dh_split_sizes((uint32_t)live, (uint32_t)n_dt, (uint32_t)nks, f32 != 0, (uint32_t)rows_per_tile));
      if (lane == 0) splits[c] = s;
    }
}

// A chunk's share of the count (no count: every token).
__device__ __forceinline__ int chunk_live(const int32_t* count, int c0, int cap) {
  return count ? max(0, min(*count - c0, cap)) : cap;
}

// Hc[j] = H[rows[c0 + j]], 16 bytes per thread; with the first chunk also dH's
// zero rows (nullable), where a token does not count. One workgroup per token
// of the call (chunks past the first: per row of the chunk). parts == 2: the
// rows once more behind themselves (see kPairTokens).
__global__ __launch_bounds__(256) void ce_gather_kernel(const uint4* __restrict__ H, const int32_t* __restrict__ rows,
                                                        const int32_t* __restrict__ slot, const int32_t* __restrict__ count,
                                                        int c0, int cap, int parts, int row_chunks, uint4* __restrict__ Hc,
                                                        uint4* __restrict__ dH, int grad_chunks, long long n) {
  const long long j = flat_group();
  if (j >= n) return;
  if (dH && slot[j] < 0)
    for (int i = threadIdx.x; i < grad_chunks; i += 256) dH[(size_t)j * grad_chunks + i] = make_uint4(0u, 0u, 0u, 0u);
  const int live = chunk_live(count, c0, cap);
  if (j >= live) return;
  const uint4* src = H + (size_t)rows[c0 + j] * row_chunks;
  uint4* dst = Hc + (size_t)j * row_chunks;
  for (int i = threadIdx.x; i < row_chunks; i += 256) {
    const uint4 v = src[i];
    dst[i] = v;
    if (parts == 2) dst[(size_t)live * row_chunks + i] = v;
  }
}

// ---- the forward's contraction over the gathered rows

// lmhead_lse_partial8_kernel's walk with the number of rows on the device;
// the partials' row stride is `stride`.
template <int kDtype, bool kKeep, bool kBFar>
__global__ __launch_bounds__(kThreads8, 1) void ce_partial_kernel(
    const char* __restrict__ H, const char* __restrict__ W, const int32_t* __restrict__ ids,
    const int32_t* __restrict__ count, int c0, int cap, int stride, int row_bytes, int vocab, int n_slices, int group,
    float2* __restrict__ part, float* __restrict__ zy_out, float* __restrict__ logits) {
  __shared__ uint4 smem[kEngineSmemChunks];
  const Lanes8 L = lanes8();
  const int wv = L.wv, tq = L.tq, quad = L.quad, c16 = L.c16;

  const int S = n_slices;
  const int n_tok = __builtin_amdgcn_readfirstlane(chunk_live(count, c0, cap));
  // The walk is that of the live token blocks, workgroups past it leave: dead
  // blocks in between would leave some XCDs idle (three quarters of 4096 tokens
  // counted: 2.32 ms so, 2.0 ms without).
  const int n_tb = (n_tok + kBT - 1) / kBT;
  if ((long long)blockIdx.x >= (long long)n_tb * ((S + group - 1) / group)) return;
  const WideWork work = wide_work(blockIdx.x, n_tb, S, group);
  const int t0 = work.tb * kBT;
  const int n_vt = (vocab + kBV - 1) / kBV;
  const int tile_begin = slice_tile(work.slice_first, n_vt, S);
  const int tile_end = slice_tile(work.slice_end, n_vt, S);
  const int nks = row_bytes / kStepBytes;

  Col16 c[4];
#pragma unroll
  for (int bn = 0; bn < 4; ++bn) {
    const int tok = t0 + tq * 64 + bn * 16 + c16;
    c[bn] = Col16{tok < n_tok ? ids[tok] : -1, -INFINITY, 0.0f};
  }
  auto w_rsrc = [&](int tile) {
    const int v0 = tile * kBV;
    return rsrc_words(W + (size_t)v0 * row_bytes, (uint32_t)min(kBV, vocab - v0) * row_bytes);
  };
  const int4v hr = rsrc_words(H + (size_t)t0 * row_bytes, (uint32_t)min(kBT, n_tok - t0) * row_bytes);

  int slice = work.slice_first;
  int slice_last_tile = slice_tile(slice + 1, n_vt, S) - 1;
  auto epilogue = [&](int tile, floatx4 (&acc)[8][4]) {
    const int vw = tile * kBV + wv * 128;
    int lt = L.lane;  // made opaque: formed here, not kept live across the K loop
    asm volatile("" : "+v"(lt));
    lt = tq * 64 + (lt & 15);
    auto fold_tile = [&](auto partial, auto pick) {
#pragma unroll
      for (int bn = 0; bn < 4; ++bn) {
        if constexpr (kKeep) {
          // (entries past the vocabulary are zeros and have their place)
          const LogitRows rows = logit_rows(logits + (size_t)tile * kBV * cap, kBV, t0 + tq * 64, 64, n_tok, c16, quad);
#pragma unroll
          for (int bm = 0; bm < 8; ++bm)
            store_logits(rows, bn, wv * 128 + bm * 16, quad, kBV, acc[bm][bn], std::false_type{});
        }
        floatx4 z[8];
#pragma unroll
        for (int bm = 0; bm < 8; ++bm) z[bm] = acc[bm][bn];
        if constexpr (decltype(pick)::value) pick_sampled(c[bn], z, vw, quad, zy_out + (t0 + lt + bn * 16));
        fold_column16(c[bn], z, vw, quad, vocab, partial);
        __builtin_amdgcn_sched_barrier(0);  // one token column at a time (register pressure)
      }
    };
    bool mine = false;
#pragma unroll
    for (int bn = 0; bn < 4; ++bn) {
      int y = c[bn].y;
      asm volatile("" : "+v"(y));
      mine = mine || (unsigned)(y - vw) < 128u;
    }
    if (tile * kBV + kBV > vocab) fold_tile(std::true_type{}, std::true_type{});
    else if (__builtin_amdgcn_ballot_w64(mine) != 0) fold_tile(std::false_type{}, std::true_type{});
    else fold_tile(std::false_type{}, std::false_type{});
    if (tile == slice_last_tile) {
#pragma unroll
      for (int bn = 0; bn < 4; ++bn) {
        const int tok = t0 + lt + bn * 16;
        flush_slice16(c[bn], tok, n_tok, quad, ((size_t)slice * 2 + wv) * stride + tok, part);
      }
      ++slice;
      int Sx = S;
      asm volatile("" : "+s"(Sx));
      slice_last_tile = slice_tile(slice + 1, n_vt, Sx) - 1;
    }
  };
  run_tiles8<kDtype, kBFar>(smem, L, row_bytes, tile_begin, tile_end, nks, w_rsrc, hr, epilogue);
}

// The same for few tokens or small vocabularies: blocks of kBRows tokens, one
// workgroup per (token block, slice), the arithmetic and bits as above
// (lmhead_lse_partial_narrow_kernel's walk).
template <int kDtype, bool kKeep, int kBRows>
__global__ __launch_bounds__(kThreads, 1) void ce_partial_narrow_kernel(
    const char* __restrict__ H, const char* __restrict__ W, const int32_t* __restrict__ ids,
    const int32_t* __restrict__ count, int c0, int cap, int stride, int row_bytes, int vocab, int n_slices,
    float2* __restrict__ part, float* __restrict__ zy_out, float* __restrict__ logits) {
  __shared__ uint4 smem[kEngineSmemChunks];
  const Lanes L = lanes();
  const int wv = L.wv, wt = L.wt, quad = L.lane >> 4, c16 = L.lane & 15;
  const int S = n_slices;
  const int slice = blockIdx.x % S;
  constexpr int kBN = kBRows / 32;
  constexpr int kWaveToks = kBRows / 2;
  const int t0 = (blockIdx.x / S) * kBRows;
  const int n_tok = __builtin_amdgcn_readfirstlane(chunk_live(count, c0, cap));
  if (t0 >= n_tok) return;
  const int n_vt = (vocab + kBV - 1) / kBV;
  const int tile_begin = slice_tile(slice, n_vt, S);
  const int tile_end = slice_tile(slice + 1, n_vt, S);
  const int nks = row_bytes / kStepBytes;
  Col16 c[kBN];
#pragma unroll
  for (int bn = 0; bn < kBN; ++bn) {
    const int tok = t0 + wt * kWaveToks + bn * 16 + c16;
    c[bn] = Col16{tok < n_tok ? ids[tok] : -1, -INFINITY, 0.0f};
  }
  auto w_rsrc = [&](int tile) {
    const int v0 = tile * kBV;
    return rsrc_words(W + (size_t)v0 * row_bytes, (uint32_t)min(kBV, vocab - v0) * row_bytes);
  };
  const int4v hr = rsrc_words(H + (size_t)t0 * row_bytes, (uint32_t)min(kBRows, n_tok - t0) * row_bytes);
  auto epilogue = [&](int tile, floatx4 (&acc)[8][kBN]) {
    const int vw = tile * kBV + wv * 128;
    auto fold_tile = [&](auto partial) {
      if constexpr (kKeep) {
        const LogitRows rows =
            logit_rows(logits + (size_t)tile * kBV * cap, kBV, t0 + wt * kWaveToks, kWaveToks, n_tok, c16, quad);
#pragma unroll
        for (int bn = 0; bn < kBN; ++bn)
#pragma unroll
          for (int bm = 0; bm < 8; ++bm)
            store_logits(rows, bn, wv * 128 + bm * 16, quad, kBV, acc[bm][bn], std::false_type{});
      }
#pragma unroll
      for (int bn = 0; bn < kBN; ++bn) {
        floatx4 z[8];
#pragma unroll
        for (int bm = 0; bm < 8; ++bm) z[bm] = acc[bm][bn];
        pick_sampled(c[bn], z, vw, quad, zy_out + (t0 + wt * kWaveToks + bn * 16 + c16));
        fold_column16(c[bn], z, vw, quad, vocab, partial);
      }
    };
    if (tile * kBV + kBV > vocab) fold_tile(std::true_type{});
    else fold_tile(std::false_type{});
  };
  run_tiles_narrow<kDtype, kBRows>(smem, L, row_bytes, tile_begin, tile_end, nks, w_rsrc, hr, epilogue);
#pragma unroll
  for (int bn = 0; bn < kBN; ++bn) {
    const int tok = t0 + wt * kWaveToks + bn * 16 + c16;
    flush_slice16(c[bn], tok, n_tok, quad, ((size_t)slice * 2 + wv) * stride + tok, part);
  }
}

// fp32 heads: z in 64 x 64 tiles (vocabulary tiles fastest).
__global__ __launch_bounds__(kF32Threads, 1) void ce_logits_f32_kernel(const char* __restrict__ Hc,
                                                                       const char* __restrict__ W,
                                                                       const int32_t* __restrict__ count, int c0, int cap,
                                                                       int row_bytes, int vocab, int n_vt,
                                                                       float* __restrict__ z) {
  __shared__ __align__(1024) uint4 smem[kF32SmemChunks];
  const int live = __builtin_amdgcn_readfirstlane(chunk_live(count, c0, cap));
  const int vt = blockIdx.x % n_vt, t0 = blockIdx.x / n_vt * kF32Tile, v0 = vt * kF32Tile;
  if (t0 >= live) return;
  const KmOperand A{W + (size_t)v0 * row_bytes, (uint32_t)row_bytes, min(kF32Tile, vocab - v0), 0u};
  const KmOperand B{Hc + (size_t)t0 * row_bytes, (uint32_t)row_bytes, min(kF32Tile, live - t0), 0u};
  run_tile_f32<false, false>(smem, A, B, row_bytes / kStepBytes, [&](floatx4 (&acc)[2][2], int wave, int quad, int c16) {
#pragma unroll
    for (int bn = 0; bn < 2; ++bn) {
      const int t = t0 + 32 * (wave >> 1) + 16 * bn + c16;
      if (t >= live) continue;
#pragma unroll
      for (int bm = 0; bm < 2; ++bm) {
        const floatx4& o = acc[bm][bn];
        *reinterpret_cast<float4*>(z + block_at(t, v0 + 32 * (wave & 1) + 16 * bm + 4 * quad, cap)) =
            make_float4(o[0], o[1], o[2], o[3]);
      }
    }
  });
}

// G is held in units of u = (1 - e) s / N, which the contractions' epilogues
// apply in fp32: a p - [v = y] - c with a = (1 + 2 lam lse) / (1 - e) and
// c = e / (V (1 - e)). The target's entry is then near -1, which bf16 holds
// to 2^-10 or better; with u folded in, every target's entry would carry the
// same rounding error of u, up to 2^-9 of the whole gradient (measured:
// dH and dW 0.0027 off at d = 2560, V = 151936 with 16-bit results; 0.0020 so).
// The -1 is taken off in fp32, before any rounding to bf16: for a sure token p
// is near 1, and rounded first it would leave of p - 1 its rounding error alone.
struct GradScale {
  float smoothing, z_weight, scale, inv_vocab;
  int mean;
};

__device__ __forceinline__ float grad_unit(const GradScale& g, const int32_t* count) {
  const double u = (double)g.scale * (1.0 - (double)g.smoothing);
  return (float)(g.mean ? u / (double)max(1, *count) : u);
}

// One token's row of G from its logits.
struct GradRow {
  float l2e_lse, a, cc;
  __device__ __forceinline__ GradRow(const GradScale& gs, float lse) {
    const float rest = 1.0f / (1.0f - gs.smoothing);
    l2e_lse = lse * kLog2e;
    a = rest * (1.0f + 2.0f * gs.z_weight * lse);
    cc = gs.smoothing * gs.inv_vocab * rest;
  }
  __device__ __forceinline__ float at(float z) const { return a * fast_exp2(z * kLog2e - l2e_lse) - cc; }
};

// lse and logprob of a row of z: each thread folds entries 4 (tid + 256 i) .. +
// 3 into its (max, sum), then a fixed tree. kGrad: then the row's G too (as
// ce_grad_logits_kernel writes it), of vocabularies up to kGradRowVocab: a
// launch less (177 tokens, d = 128, V = 1024: 37 -> 35 us); larger ones
// want more than a workgroup per token for it.
constexpr int kGradRowVocab = 4096;
template <bool kGrad>
__global__ __launch_bounds__(256) void ce_lse_f32_kernel(const float* __restrict__ z,
                                                         const int32_t* __restrict__ ids, const int32_t* __restrict__ count,
                                                         int c0, int cap, int vocab, float* __restrict__ logprob,
                                                         float* __restrict__ lse, GradScale gs, float* __restrict__ Gd) {
  __shared__ float2 lds[4];
  const int t = blockIdx.x;
  if (t >= chunk_live(count, c0, cap)) return;
  float m = -INFINITY, s = 0.0f;
  for (int v = 4 * threadIdx.x; v < vocab; v += 1024) {
    const float4 q = *reinterpret_cast<const float4*>(z + block_at(t, v, cap));
    float x[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = v + i < vocab ? x[i] : -INFINITY;
    const float top = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), m);
    const float ref = top == -INFINITY ? 0.0f : top;
    float e = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) e += fast_exp2((x[i] - ref) * kLog2e);
    s = __builtin_fmaf(s, fast_exp2((m - ref) * kLog2e), e);
    m = top;
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) {
    const float m2 = __shfl_xor(m, off, 64), s2 = __shfl_xor(s, off, 64);
    lse_merge(m, s, m2, s2);
  }
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = make_float2(m, s);
  __syncthreads();
  if (!kGrad && threadIdx.x != 0) return;
  m = lds[0].x, s = lds[0].y;
  for (int w = 1; w < 4; ++w) lse_merge(m, s, lds[w].x, lds[w].y);
  // (z_y - m) - ln s: lse itself is rounded to a step of its size, which may be
  // many times the loss. s >= 1, the maximum's own term is 1.
  const float ln_s = fast_log2(s) * kLn2;
  const int y = ids[t];  // (not gathered: it may not count)
  if (threadIdx.x == 0) {
    logprob[t] = ((unsigned)y < (unsigned)vocab ? z[block_at(t, y, cap)] - m : 0.0f) - ln_s;
    lse[t] = m + ln_s;
  }
  if constexpr (kGrad) {
    const GradRow row(gs, m + ln_s);
    for (int v = 4 * threadIdx.x; v < (vocab + kBV - 1) / kBV * kBV; v += 1024) {
      const float4 q = *reinterpret_cast<const float4*>(z + block_at(t, v, cap));
      const float x[4] = {q.x, q.y, q.z, q.w};
      float o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float e = row.at(x[i]);
        if (v + i == y) e -= 1.0f;
        o[i] = v + i < vocab ? e : 0.0f;
      }
      *reinterpret_cast<float4*>(Gd + block_at(t, v, cap)) = make_float4(o[0], o[1], o[2], o[3]);
    }
  }
}

// ---- mean of the logits (label smoothing): z's mean over v is H . mean_v W[v]

constexpr int kMeanRows = 128;  // rows of W per partial sum

// part[b, k] = sum of W[v, k] over kMeanRows rows v: 512 columns per workgroup,
// 8 per thread, four wavefronts on rows v, v + 4, ... each, then added in
// order. One pass over W at the memory's rate.
template <int kDtype>
__global__ __launch_bounds__(256) void ce_colsum_kernel(const typename Elem<kDtype>::T* __restrict__ W, int vocab, int d,
                                                        float* __restrict__ part) {
  using E = Elem<kDtype>;
  __shared__ float lds[3][512];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int k = blockIdx.y * 512 + 8 * lane;  // (d is a multiple of 8)
  const int v0 = blockIdx.x * kMeanRows, v1 = min(vocab, v0 + kMeanRows);
  float s[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  if (k < d) {
#pragma unroll 16
    for (int v = v0 + wave; v < v1; v += 4) {
      const uint4* row = reinterpret_cast<const uint4*>(W + (size_t)v * d + k);
      uint4 w[E::kSize / 2];
#pragma unroll
      for (int i = 0; i < E::kSize / 2; ++i) w[i] = row[i];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t x = (&w[0].x)[kDtype == 0 ? j >> 1 : j];
        s[j] += kDtype == 1 ? __uint_as_float(x) : __uint_as_float((j & 1) ? (x & 0xffff0000u) : (x << 16));
      }
    }
  }
  if (wave > 0) {
#pragma unroll
    for (int j = 0; j < 8; ++j) lds[wave - 1][j * 64 + lane] = s[j];
  }
  __syncthreads();
  if (wave > 0 || k >= d) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) s[j] = ((s[j] + lds[0][j * 64 + lane]) + lds[1][j * 64 + lane]) + lds[2][j * 64 + lane];
  float4* out = reinterpret_cast<float4*>(part + (size_t)blockIdx.x * d + k);
  out[0] = make_float4(s[0], s[1], s[2], s[3]);
  out[1] = make_float4(s[4], s[5], s[6], s[7]);
}

// The partial sums in a fixed order (16 wavefronts on every 16th, then the
// wavefronts), over V.
__global__ __launch_bounds__(1024) void ce_colmean_kernel(const float* __restrict__ part, int n_part, int d, int vocab,
                                                          float* __restrict__ wmean) {
  __shared__ double lds[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int k = blockIdx.x * 64 + lane;  // (d is a multiple of 64)
  double s = 0.0;
#pragma unroll 8
  for (int b = wave; b < n_part; b += 16) s += (double)part[(size_t)b * d + k];
  lds[wave][lane] = s;
  __syncthreads();
  if (wave > 0) return;
  for (int w = 1; w < 16; ++w) s += lds[w][lane];
  wmean[k] = (float)(s / (double)vocab);
}

// ---- the tokens' losses

// One wavefront per token of the call: its loss (0 where it does not count)
// and its lse, and per workgroup the fp64 sum of four losses.
template <int kDtype>
__global__ __launch_bounds__(256) void ce_token_loss_kernel(const typename Elem<kDtype>::T* __restrict__ H, int n, int d,
                                                            const int32_t* __restrict__ slot,
                                                            const float* __restrict__ logprob, const float* __restrict__ lse,
                                                            const float* __restrict__ wmean, float smoothing, float z_weight,
                                                            float* __restrict__ token_loss, float* __restrict__ lse_out,
                                                            double* __restrict__ part) {
  using E = Elem<kDtype>;
  __shared__ double lds[4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const long long group = flat_group(), t = group * 4 + wave;
  const int j = t < n ? slot[t] : -1;
  float l = 0.0f, s = 0.0f;
  if (j >= 0) {
    s = lse[j];
    l = -(1.0f - smoothing) * logprob[j];
    if (wmean) {
      float zm = 0.0f;
      // (d is a multiple of 64: 8 values per lane while whole groups of 512 last, then one)
      int k = 8 * lane;
#pragma unroll 2
      for (; k - 8 * lane + 512 <= d; k += 512) {
        const uint4* hr = reinterpret_cast<const uint4*>(H + (size_t)t * d + k);
        uint4 w[E::kSize / 2];
#pragma unroll
        for (int i = 0; i < E::kSize / 2; ++i) w[i] = hr[i];
        const float4 m0 = *reinterpret_cast<const float4*>(wmean + k), m1 = *reinterpret_cast<const float4*>(wmean + k + 4);
        const float m[8] = {m0.x, m0.y, m0.z, m0.w, m1.x, m1.y, m1.z, m1.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t x = (&w[0].x)[kDtype == 0 ? j >> 1 : j];
          zm += (kDtype == 1 ? __uint_as_float(x) : __uint_as_float((j & 1) ? (x & 0xffff0000u) : (x << 16))) * m[j];
        }
      }
      for (k = k - 8 * lane + lane; k < d; k += 64) zm += E::to_f(H[(size_t)t * d + k]) * wmean[k];
      l += smoothing * (s - wave_sum(zm));
    }
    l += z_weight * s * s;
  }
  if (lane == 0) {
    if (t < n) {
      token_loss[t] = l;
      if (lse_out) lse_out[t] = s;
    }
    lds[wave] = (double)l;
  }
  __syncthreads();
  if (threadIdx.x == 0 && group * 4 < n) part[group] = ((lds[0] + lds[1]) + lds[2]) + lds[3];
}

// The fp64 sums in a fixed order, over N (0 when no token counts).
__global__ __launch_bounds__(1024) void ce_loss_kernel(const double* __restrict__ part, int n_part,
                                                       const int32_t* __restrict__ count, int mean,
                                                       float* __restrict__ loss) {
  __shared__ double lds[16];
  double s = 0.0;
  for (int i = threadIdx.x; i < n_part; i += 1024) s += part[i];
  s = wave_sum_d(s);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int w = 1; w < 16; ++w) s += lds[w];
  *loss = (float)(mean ? s / (double)max(1, *count) : s);
}

// Both of the above for at most kSmallTokens tokens without smoothing, in one
// launch: a thread takes four consecutive tokens (the additions are the same,
// so the loss's bits are). slot == nullptr: the tokens were not gathered, a
// token's place is its own and N is counted here.
constexpr int kSmallTokens = 4096;
__global__ __launch_bounds__(1024) void ce_small_loss_kernel(const int32_t* __restrict__ targets, int n, int vocab,
                                                             const int32_t* __restrict__ slot,
                                                             const int32_t* __restrict__ count,
                                                             const float* __restrict__ logprob, const float* __restrict__ lse,
                                                             float z_weight, int mean, float* __restrict__ token_loss,
                                                             float* __restrict__ lse_out, float* __restrict__ loss) {
  __shared__ double lds[16];
  __shared__ int lds_n[16];
  float l[4];
  int live = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = 4 * threadIdx.x + i;
    l[i] = 0.0f;
    float s = 0.0f;
    if (t < n) {
      const int j = slot ? slot[t] : (unsigned)targets[t] < (unsigned)vocab ? t : -1;
      if (j >= 0) {
        ++live;
        s = lse[j];
        l[i] = -logprob[j];
        l[i] += z_weight * s * s;
      }
      token_loss[t] = l[i];
      if (lse_out) lse_out[t] = s;
    }
  }
  double sum = (((double)l[0] + (double)l[1]) + (double)l[2]) + (double)l[3];
  sum = wave_sum_d(sum);
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) live += __shfl_xor(live, off, 64);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = sum, lds_n[threadIdx.x >> 6] = live;
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int w = 1; w < 16; ++w) sum += lds[w], live += lds_n[w];
  if (count) live = *count;
  *loss = (float)(mean ? sum / (double)max(1, live) : sum);
}

// ---- G

// G from the kept logits: 8 vocabulary entries of one token per thread; past
// the vocabulary zeros. rest (bf16, nullable): what the target's entry lost to
// its rounding, which fp32 gradients then take in fp32.
constexpr int kGradVec = 8;

// Up to this many tokens (bf16), G is held as two bf16 rows per token, its
// rounding and the rounding of what that leaves, the second one's rows behind
// all of the first's: both contractions are bound by W and dW then, so the
// second row costs nothing and G's error falls from 2^-8 to 2^-16 of an entry.
// (With few tokens one entry's rounding can be all of a gradient's error;
// with many they average out.)
constexpr int kPairTokens = 128;

template <int kDtype>
__global__ __launch_bounds__(256) void ce_grad_logits_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ ids, const int32_t* __restrict__ count,
    int c0, int cap, int parts, int vocab, int g_rows, const float* __restrict__ lse, GradScale gs,
    typename Elem<kDtype>::T* __restrict__ Gd, float* __restrict__ rest) {
  using E = Elem<kDtype>;
  // a workgroup takes 8 tokens of one block: 8 KiB of z side by side
  const int t = blockIdx.y * (256 * kGradVec / kBV) + threadIdx.x / (kBV / kGradVec);
  const int v = blockIdx.x * kBV + threadIdx.x % (kBV / kGradVec) * kGradVec;
  const int live = chunk_live(count, c0, cap);
  if (t >= live) return;
  const GradRow row(gs, lse[t]);
  const int y = ids[t];
  float z[kGradVec];
  const floatx4* at = reinterpret_cast<const floatx4*>(logits + block_at(t, v, cap));
  const floatx4 lo = __builtin_nontemporal_load(at), hi = __builtin_nontemporal_load(at + 1);
#pragma unroll
  for (int r = 0; r < 4; ++r) z[r] = lo[r], z[4 + r] = hi[r];
#pragma unroll
  for (int r = 0; r < kGradVec; ++r) {
    float x = row.at(z[r]);
    if (v + r == y) x -= 1.0f;
    z[r] = v + r < vocab ? x : 0.0f;
  }
  typename E::T* out = Gd + block_at(t, v, g_rows);
  if constexpr (kDtype == 0) {
    for (int part = 0; part < parts; ++part) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w[j] = (uint32_t)E::from_f(z[2 * j]) | ((uint32_t)E::from_f(z[2 * j + 1]) << 16);
        z[2 * j] -= __uint_as_float(w[j] << 16);
        z[2 * j + 1] -= __uint_as_float(w[j] & 0xffff0000u);
      }
      *reinterpret_cast<uint4*>(out) = make_uint4(w[0], w[1], w[2], w[3]);
      out += (size_t)live * kBV;
    }
    if (rest) {
#pragma unroll
      for (int r = 0; r < kGradVec; ++r)
        if (v + r == y) rest[t] = z[r];
    }
  } else {
    reinterpret_cast<float4*>(out)[0] = make_float4(z[0], z[1], z[2], z[3]);
    reinterpret_cast<float4*>(out)[1] = make_float4(z[4], z[5], z[6], z[7]);
  }
}

// The chunk's live tokens' rest in the gradient's unit, 0 (and id -1) past
// them: the targets' term of the fp32 gradients.
__global__ __launch_bounds__(256) void ce_rest_kernel(const int32_t* __restrict__ ids, const int32_t* __restrict__ count,
                                                      int c0, int cap, GradScale gs, float* __restrict__ coef,
                                                      int32_t* __restrict__ chunk_ids) {
  const int j = blockIdx.x * 256 + threadIdx.x;
  if (j >= cap) return;
  const bool in = j < chunk_live(count, c0, cap);
  coef[j] = in ? coef[j] * grad_unit(gs, count) : 0.0f;
  chunk_ids[j] = in ? ids[j] : -1;
}

// ---- dH

__device__ __forceinline__ void store_grad4(void* out, int grad_f32, size_t at, const float (&o)[4]) {
  if (grad_f32) {
    *reinterpret_cast<float4*>(static_cast<float*>(out) + at) = make_float4(o[0], o[1], o[2], o[3]);
  } else {
    uint2 pk;
    pk.x = (uint32_t)Elem<0>::from_f(o[0]) | ((uint32_t)Elem<0>::from_f(o[1]) << 16);
    pk.y = (uint32_t)Elem<0>::from_f(o[2]) | ((uint32_t)Elem<0>::from_f(o[3]) << 16);
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) = pk;
  }
}

// Partial sp of dH for the chunk: A = W (columns d0 .. of rows v), B = rows of
// Gd, K = the vocabulary steps [nks sp / splits, nks (sp + 1) / splits). Writes
// fp32 rows part[sp, t, :] (the live tokens' rows per split). Token
// blocks fastest: workgroups that run together share W's rows.
template <int kDtype>
__global__ __launch_bounds__(kDtype == 0 ? kThreads8 : kF32Threads, 1) void ce_dh_kernel(
    const char* __restrict__ W, const char* __restrict__ Gd, int vocab, int vpad, int d, const int32_t* __restrict__ count,
    int c0, int cap, int parts, int g_rows, int n_dt, const int32_t* __restrict__ splits_of, float* __restrict__ part) {
  constexpr int kT = GradTile<kDtype>::kRows, kStepK = GradTile<kDtype>::kStepK, es = Elem<kDtype>::kSize;
  __shared__ __align__(1024) uint4 smem[kDtype == 0 ? kEngineSmemChunks : kF32SmemChunks];
  const int live = __builtin_amdgcn_readfirstlane(parts * chunk_live(count, c0, cap));
  const int splits = __builtin_amdgcn_readfirstlane(*splits_of);
  const int n_tb = (live + kT - 1) / kT;
  if ((long long)blockIdx.x >= (long long)n_tb * n_dt * splits) return;
  const int tb = blockIdx.x % n_tb, rest = blockIdx.x / n_tb;
  const int dt = rest % n_dt, sp = rest / n_dt;
  const int t0 = tb * kT;
  const int nks_all = vpad / kStepK;
  const int ks0 = (int)((long long)nks_all * sp / splits), ks1 = (int)((long long)nks_all * (sp + 1) / splits);
  const uint32_t w_row = (uint32_t)d * es, g_row = kBV * es, d_off = (uint32_t)dt * kT * es;
  const char* w_rows = W + (size_t)ks0 * kStepK * w_row;
  const int w_left = vocab - ks0 * kStepK;
  const KmOperand B{Gd + (size_t)t0 * g_row, g_row, min(kT, live - t0), 0u, kDtype == 0 ? 2 : 3, ks0,
                    (size_t)g_rows * g_row};
  static_assert(kBV / kStepK == (kDtype == 0 ? 4 : 8), "K steps of a block of G");
  float* out = part + (size_t)sp * live * d;
  auto store = [&](int t, int k, const floatx4& o) {
    if (t < live && k < d) *reinterpret_cast<float4*>(out + (size_t)t * d + k) = make_float4(o[0], o[1], o[2], o[3]);
  };
  if constexpr (kDtype == 0) {
    const Lanes8 L = lanes8();
    run_tiles_km<false, false>(smem, L, KmOperand{w_rows, w_row, w_left, 0u}, B, dt, dt + 1, ks1 - ks0,
                        [&](int, floatx4 (&acc)[8][4]) {
#pragma unroll
      for (int bn = 0; bn < 4; ++bn)
#pragma unroll
        for (int bm = 0; bm < 8; ++bm)
          store(t0 + L.tq * 64 + bn * 16 + L.c16, dt * kT + L.wv * 128 + bm * 16 + 4 * L.quad, acc[bm][bn]);
    });
  } else {
    run_tile_f32<true, false>(smem, KmOperand{w_rows + d_off, w_row, w_left, d_off}, B, ks1 - ks0, [&](floatx4 (&acc)[2][2], int wave, int quad, int c16) {
#pragma unroll
      for (int bn = 0; bn < 2; ++bn)
#pragma unroll
        for (int bm = 0; bm < 2; ++bm)
          store(t0 + 32 * (wave >> 1) + 16 * bn + c16, dt * kT + 32 * (wave & 1) + 16 * bm + 4 * quad, acc[bm][bn]);
    });
  }
}

// dH rows: the splits added in order (plus, with coef, the target's rest
// coef[j] W[y]), four values per thread, to the token's own row. 256
// columns per workgroup: with few tokens and many splits, waiting for the
// partials is all there is (2 tokens, d = 3904, 16 splits: 39 us by one
// workgroup per token).
constexpr int kDhFinish = 64;
template <int kDtype>
__global__ __launch_bounds__(kDhFinish) void ce_dh_finish_kernel(
    const float* __restrict__ part, const int32_t* __restrict__ splits_of, int cap, int parts, int d,
    const int32_t* __restrict__ rows, const int32_t* __restrict__ ids, const int32_t* __restrict__ count, int c0, GradScale gs,
    const float* __restrict__ coef, const typename Elem<kDtype>::T* __restrict__ W, int grad_f32, void* __restrict__ dH) {
  using E = Elem<kDtype>;
  const int j = blockIdx.x, k = (blockIdx.y * kDhFinish + threadIdx.x) * 4;
  const int live = chunk_live(count, c0, cap);
  if (j >= live || k >= d) return;
  const int splits = *splits_of;
  const size_t per_split = (size_t)(parts * live) * d;
  const float unit = grad_unit(gs, count);
  const float* at = part + (size_t)j * d + k;
  float o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  auto add = [&](const float* p) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    o[0] += v.x, o[1] += v.y, o[2] += v.z, o[3] += v.w;
  };
  if (parts == 2) {
#pragma unroll 8
    for (int s = 0; s < splits; ++s) {
      add(at + s * per_split);
      add(at + s * per_split + (size_t)live * d);
    }
  } else {
#pragma unroll 8
    for (int s = 0; s < splits; ++s) add(at + s * per_split);
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) o[r] *= unit;
  if (coef) {
    const float c = coef[j];
    const typename E::T* w = W + (size_t)ids[j] * d + k;
#pragma unroll
    for (int r = 0; r < 4; ++r) o[r] += c * E::to_f(w[r]);
  }
  store_grad4(dH, grad_f32, (size_t)rows[c0 + j] * d + k, o);
}

// ---- dW

// Columns v0 .. of G as a K-major operand (within one block), `live` rows.
__device__ __forceinline__ KmOperand g_columns(const char* Gd, int v0, int g_rows, int es, int live) {
  const uint32_t off = (uint32_t)(v0 % kBV * es);
  return KmOperand{Gd + (size_t)(v0 / kBV) * g_rows * (kBV * es) + off, (uint32_t)(kBV * es), live, off};
}

// Tile of workgroup b of dW's contraction. Workgroups go to the 8 XCDs in
// turn; XCD x takes the vocabulary tiles x, x + 8, ..., in blocks of 5 of them
// by 3 walks of two tiles of d, so that the 30 or so workgroups it runs
// together (two blocks) share few columns of G and H through its L2, and G
// comes from memory once for every 6 tiles of d or so. (With 32 vocabulary
// tiles side by side, each XCD read G once per tile of d: 16 GB in 3.9 ms at d
// = 7168, the memory's limit. Blocks of 4 x 4, 8 x 4 and walks of one measured
// within 1.5 %.)
constexpr int kDwWalk = 2;  // tiles of d a workgroup walks (fp32: one)
constexpr int kDwVocabTiles = 5, kDwWidthTiles = 3;  // of walks

__host__ __device__ inline bool dw_work(int b, int n_vt, int n_dt, int& vt, int& dt) {
  const int x = b & 7, i = b >> 3;
  const int rows = kDwVocabTiles * n_dt;
  const int rem = i % rows, g = rem / (kDwVocabTiles * kDwWidthTiles);
  const int left = n_dt - g * kDwWidthTiles, w = left < kDwWidthTiles ? left : kDwWidthTiles;
  const int r = rem - g * kDwVocabTiles * kDwWidthTiles;
  dt = g * kDwWidthTiles + r % w;
  vt = x + 8 * (i / rows * kDwVocabTiles + r / w);
  return vt < n_vt;
}

// Workgroups that cover every tile (a few of them past the last).
inline long long dw_groups(long long n_vt, long long n_dt) {
  return 8 * ceil_div(ceil_div(n_vt, 8), kDwVocabTiles) * kDwVocabTiles * n_dt;
}

// The chunk's part of dW: A = Hc (columns d0 ..), B = Gd (columns v0 ..), K =
// the chunk's live tokens.
// A workgroup walks up to `walk` tiles of d (fp32: one), so that a
// tile's first loads and last stores run under its neighbours' products.
// Where there are few tiles (small vocabularies) the tokens are split over
// gridDim.x / tiles workgroups each: partial sums [split, vocab, d] in fp32,
// without the unit.
enum { kDwRound = 0, kDwWrite = 1, kDwAdd = 2, kDwPart = 3 };  // bf16 results; fp32; fp32 on top of dW; partials

template <int kDtype, int kMode>
__global__ __launch_bounds__(kDtype == 0 ? kThreads8 : kF32Threads, 1) void ce_dw_kernel(
    const char* __restrict__ Gd, const char* __restrict__ Hc, int g_rows, const int32_t* __restrict__ count, int c0, int cap,
    int vocab, int d, int n_vt, int n_dt, int walk, GradScale gs, void* __restrict__ dW) {
  constexpr int kT = GradTile<kDtype>::kRows, kStepK = GradTile<kDtype>::kStepK, es = Elem<kDtype>::kSize;
  __shared__ __align__(1024) uint4 smem[kDtype == 0 ? kEngineSmemChunks : kF32SmemChunks];
  const int live = __builtin_amdgcn_readfirstlane(chunk_live(count, c0, cap));
  if (live == 0 && c0 > 0 && kMode != kDwPart) return;  // (the first chunk writes its zeros; partials are read)
  int vt, dt;
  int split = 0;
  if constexpr (kMode == kDwPart) {  // one tile each, in turn over the XCDs: few vocabulary tiles would fill few of them
    const int tiles = n_vt * n_dt;
    split = blockIdx.x / tiles;
    vt = blockIdx.x % tiles / n_dt, dt = blockIdx.x % n_dt;
  } else {
    if (!dw_work(blockIdx.x, n_vt, (n_dt + walk - 1) / walk, vt, dt)) return;
    dt *= walk;
  }
  const int dt_end = min(dt + walk, n_dt);
  const int nks_all = (live + kStepK - 1) / kStepK;
  int ks0 = 0, ks1 = nks_all;
  if constexpr (kMode == kDwPart) {
    const int splits = gridDim.x / (n_vt * n_dt);
    ks0 = (int)((long long)nks_all * split / splits);
    ks1 = (int)((long long)nks_all * (split + 1) / splits);
  }
  const int nks = max(1, ks1 - ks0);  // (a split without steps sums zeros: its range of rows is empty)
  const int first = ks0 * kStepK, left = min(live, ks1 * kStepK) - first;
  const uint32_t h_row = (uint32_t)d * es;
  const uint32_t d_off = (uint32_t)dt * kT * es;
  KmOperand B = g_columns(Gd, vt * kT, g_rows, es, left);
  B.base += (size_t)first * B.row_bytes;
  Hc += (size_t)first * h_row;
  const float unit = kMode == kDwPart ? 1.0f : grad_unit(gs, count);
  auto store = [&](int v, int k, const floatx4& o) {
    if (v >= vocab || k >= d) return;
    if constexpr (kMode == kDwPart) {
      char* part = static_cast<char*>(dW) + (size_t)split * vocab * d * 4;  // (one split's is less than 2^31 bytes)
      *reinterpret_cast<floatx4*>(part + ((uint32_t)v * (uint32_t)d + (uint32_t)k) * 4u) = o;
      return;
    }
    const size_t at = (size_t)v * d + k;
    float x[4] = {o[0] * unit, o[1] * unit, o[2] * unit, o[3] * unit};
    if constexpr (kMode == kDwAdd) {
      const float4 old = *reinterpret_cast<const float4*>(static_cast<const float*>(dW) + at);
      x[0] += old.x, x[1] += old.y, x[2] += old.z, x[3] += old.w;
    }
    store_grad4(dW, kMode != kDwRound, at, x);
  };
  if constexpr (kDtype == 0) {
    const Lanes8 L = lanes8();
    run_tiles_km<true, true>(smem, L, KmOperand{Hc, h_row, left, 0u}, B, dt, dt_end, nks, [&](int tile, floatx4 (&acc)[8][4]) {
      int lane = L.lane;  // made opaque: addresses formed here, not kept live across the K loop
      asm volatile("" : "+v"(lane));
      const int v0 = vt * kT + L.tq * 64 + (lane & 15), k0 = tile * kT + L.wv * 128 + 4 * (lane >> 4);
#pragma unroll
      for (int bn = 0; bn < 4; ++bn) {
#pragma unroll
        for (int bm = 0; bm < 8; ++bm) store(v0 + bn * 16, k0 + bm * 16, acc[bm][bn]);
        __builtin_amdgcn_sched_barrier(0);
      }
    });
  } else {
    run_tile_f32<true, true>(smem, KmOperand{Hc + d_off, h_row, left, d_off}, B, nks, [&](floatx4 (&acc)[2][2], int wave, int quad, int c16) {
#pragma unroll
      for (int bn = 0; bn < 2; ++bn)
#pragma unroll
        for (int bm = 0; bm < 2; ++bm)
          store(vt * kT + 32 * (wave >> 1) + 16 * bn + c16, dt * kT + 32 * (wave & 1) + 16 * bm + 4 * quad, acc[bm][bn]);
    });
  }
}

// The splits' partials added in order, times the unit: as kMode says.
template <int kMode>
__global__ __launch_bounds__(256) void ce_dw_finish_kernel(const float* __restrict__ part, int splits, long long n,
                                                           const int32_t* __restrict__ count, GradScale gs,
                                                           void* __restrict__ dW) {
  const long long i = ((long long)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= n) return;
  const float unit = grad_unit(gs, count);
  float o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
  for (int s = 0; s < splits; ++s) {
    const float4 v = *reinterpret_cast<const float4*>(part + s * n + i);
    o[0] += v.x, o[1] += v.y, o[2] += v.z, o[3] += v.w;
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) o[r] *= unit;
  if constexpr (kMode == kDwAdd) {
    const float4 old = *reinterpret_cast<const float4*>(static_cast<const float*>(dW) + i);
    o[0] += old.x, o[1] += old.y, o[2] += old.z, o[3] += old.w;
  }
  store_grad4(dW, kMode != kDwRound, i, o);
}

// dW of a chunk of few tokens (bf16): 128 x 128 tiles, the tiles of d fastest.
// d = 2560, V = 50000: 500 tokens 188 us in 256 x 256 tiles, 156 so; 1020 282
// and 267. 705 (449 counted), d = 4864, V = 340: 26 us split, 16 so. 2 tokens, d =
// 3904, V = 87112: 125 us, dW written at 5.4 TB/s.
constexpr int kFewTokens = 1024;
template <int kMode>
__global__ __launch_bounds__(kFewThreads, 4) void ce_dw_few_kernel(const char* __restrict__ Gd, const char* __restrict__ Hc,
                                                                   int g_rows, const int32_t* __restrict__ count, int c0,
                                                                   int cap, int parts, int vocab, int d, int n_dt,
                                                                   GradScale gs, void* __restrict__ dW) {
  __shared__ __align__(1024) uint4 smem[kFewSmemChunks];
  const int live = __builtin_amdgcn_readfirstlane(parts * chunk_live(count, c0, cap));
  const int dt = blockIdx.x % n_dt, vt = blockIdx.x / n_dt;
  const uint32_t d_off = (uint32_t)dt * kFewTile * 2;
  const float unit = grad_unit(gs, count);
  run_tile_few(smem, KmOperand{Hc + d_off, (uint32_t)d * 2, live, d_off},
               g_columns(Gd, vt * kFewTile, g_rows, 2, live),
               [&](floatx4 (&acc)[4][4], int wave, int quad, int c16) {
    if constexpr (kMode == kDwRound) {
      // Through LDS (the operands are done with): rows of 256 bytes, 16-byte
      // piece P of row r at P ^ (r mod 16), so that a store moves whole rows.
      // Straight from the accumulators it moves 32 bytes of 16 rows.
      char* tile = reinterpret_cast<char*>(smem);
#pragma unroll
      for (int bn = 0; bn < 4; ++bn)
#pragma unroll
        for (int bm = 0; bm < 4; ++bm) {
          const floatx4& o = acc[bm][bn];
          const int row = 64 * (wave >> 1) + 16 * bn + c16, col = 64 * (wave & 1) + 16 * bm + 4 * quad;
          *reinterpret_cast<uint2*>(tile + row * 256 + (((col >> 3) ^ c16) << 4) + (col & 4) * 2) =
              make_uint2((uint32_t)Elem<0>::from_f(o[0] * unit) | ((uint32_t)Elem<0>::from_f(o[1] * unit) << 16),
                         (uint32_t)Elem<0>::from_f(o[2] * unit) | ((uint32_t)Elem<0>::from_f(o[3] * unit) << 16));
        }
      __syncthreads();
      const int piece = threadIdx.x & 15, k = dt * kFewTile + piece * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int row = 16 * i + (threadIdx.x >> 4), v = vt * kFewTile + row;
        if (v < vocab && k < d)
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(dW) + (size_t)v * d + k) =
              *reinterpret_cast<const uint4*>(tile + row * 256 + ((piece ^ (row & 15)) << 4));
      }
      return;
    }
#pragma unroll
    for (int bn = 0; bn < 4; ++bn) {
      const int v = vt * kFewTile + 64 * (wave >> 1) + 16 * bn + c16;
      if (v >= vocab) continue;
#pragma unroll
      for (int bm = 0; bm < 4; ++bm) {
        const int k = dt * kFewTile + 64 * (wave & 1) + 16 * bm + 4 * quad;
        if (k >= d) continue;
        const size_t at = (size_t)v * d + k;
        const floatx4& o = acc[bm][bn];
        float x[4] = {o[0] * unit, o[1] * unit, o[2] * unit, o[3] * unit};
        if constexpr (kMode == kDwAdd) {
          const float4 old = *reinterpret_cast<const float4*>(static_cast<const float*>(dW) + at);
          x[0] += old.x, x[1] += old.y, x[2] += old.z, x[3] += old.w;
        }
        store_grad4(dW, kMode != kDwRound, at, x);
      }
    }
  });
}

// The accumulated fp32 dW rounded to bf16.
__global__ __launch_bounds__(256) void ce_round_kernel(const float4* __restrict__ in, long long n4, uint2* __restrict__ out) {
  const long long i = flat_group() * 256 + threadIdx.x;
  if (i >= n4) return;
  const float4 v = in[i];
  out[i] = make_uint2((uint32_t)Elem<0>::from_f(v.x) | ((uint32_t)Elem<0>::from_f(v.y) << 16),
                      (uint32_t)Elem<0>::from_f(v.z) | ((uint32_t)Elem<0>::from_f(v.w) << 16));
}

__global__ __launch_bounds__(256) void ce_add_kernel(const float4* __restrict__ in, long long n4, float4* __restrict__ out) {
  const long long i = flat_group() * 256 + threadIdx.x;
  if (i >= n4) return;
  const float4 v = in[i];
  float4 o = out[i];
  o.x += v.x, o.y += v.y, o.z += v.z, o.w += v.w;
  out[i] = o;
}

// out = 0 in 16-byte pieces; *one = 0 where given.
__global__ __launch_bounds__(256) void ce_clear_kernel(uint4* __restrict__ out, long long n16, float* __restrict__ one) {
  const long long i = flat_group() * 256 + threadIdx.x;
  if (i < n16) out[i] = make_uint4(0u, 0u, 0u, 0u);
  if (one && i == 0) *one = 0.0f;
}

// ---- workspace

// The most workgroups, and fp32 partial rows, that a chunk of up to `cap` rows
// of G can take in dH's contraction, over all live counts.
void dh_most(long long cap, long long d, long long vpad, int dtype, long long* groups, long long* rows) {
  const long long tile = dtype == 0 ? GradTile<0>::kRows : GradTile<1>::kRows;
  const long long nks = vpad / (dtype == 0 ? GradTile<0>::kStepK : GradTile<1>::kStepK), n_dt = ceil_div(d, tile);
  *groups = *rows = 0;
  auto take = [&](long long live) {
    const long long s = k_splits(dh_split_sizes((uint32_t)live, (uint32_t)n_dt, (uint32_t)nks, dtype == 1, (uint32_t)tile));
    *groups = std::max(*groups, ceil_div(live, tile) * n_dt * s);
    *rows = std::max(*rows, live * s);
  };
  for (int quarter = 1; quarter < 4; ++quarter) take(quarter * tile / 4);
  for (long long n_tb = 1; n_tb <= ceil_div(cap, tile); ++n_tb) take(n_tb * tile);
}

// Splits of the tokens of a chunk of cap in dW's contraction.
int dw_splits(long long cap, long long d, long long vocab, int dtype) {
  const long long tile = dtype == 0 ? GradTile<0>::kRows : GradTile<1>::kRows;
  const long long nks = ceil_div(cap, dtype == 0 ? GradTile<0>::kStepK : GradTile<1>::kStepK);
  const long long tiles = ceil_div(d, tile) * ceil_div(vocab, tile);
  if (tiles > 512 * (dtype == 0 ? 1 : 3)) return 1;  // the CUs have two rounds without
  return k_splits(KSplits{(uint32_t)tiles, (uint32_t)nks, 2 * (uint32_t)tile, (uint32_t)tile, dtype == 1});
}

struct CeLayout {
  int cap, vpad, parts;
  long long dh_groups;
  size_t rows, ids, slot, count, splits, lp, lse, zy, part, loss, wmean, wpart, hc, z, gd, dhp, dwp, coef, cids, dwacc,
      sampled, total;
};

CeLayout ce_layout(long long n_tok, long long d, long long vocab, int dtype, bool grad, int grad_dtype) {
  CeLayout L{};
  const int es = dtype == 0 ? 2 : 4;
  L.vpad = (int)round_up(vocab, kBV);
  L.cap = (int)std::min<long long>(grad ? kCeChunk : dtype == 1 ? kCeF32Chunk : kCeLossChunk, n_tok);
  L.parts = dtype == 0 && grad && n_tok <= kPairTokens ? 2 : 1;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += align256(bytes);
    return at;
  };
  L.rows = take((size_t)n_tok * 4);
  L.ids = take((size_t)n_tok * 4);
  L.slot = take((size_t)n_tok * 4);
  L.count = take(4);
  L.lp = take((size_t)n_tok * 4);
  L.lse = take((size_t)n_tok * 4);
  if (dtype == 0) {
    L.zy = take((size_t)L.cap * 4);
    L.part = take((size_t)2 * n_slices(vocab) * L.cap * sizeof(float2));
  }
  L.loss = take((size_t)ceil_div(n_tok, 4) * 8);
  L.wmean = take((size_t)d * 4);
  L.wpart = take((size_t)ceil_div(vocab, kMeanRows) * d * 4);
  L.hc = take((size_t)L.parts * L.cap * d * es);
  if (grad || dtype == 1) L.z = take((size_t)L.cap * L.vpad * 4);
  if (grad) {
    long long rows;
    dh_most(L.parts * L.cap, d, L.vpad, dtype, &L.dh_groups, &rows);
    L.splits = take((size_t)ceil_div(n_tok, L.cap) * 4);
    L.gd = take((size_t)L.parts * L.cap * L.vpad * es);
    L.dhp = take((size_t)rows * d * 4);
    if (dtype == 1 || n_tok > kFewTokens) {
      const long long last = n_tok % L.cap ? n_tok % L.cap : L.cap;
      const int s = std::max(dw_splits(L.cap, d, vocab, dtype), dw_splits(last, d, vocab, dtype));
      if (s > 1) L.dwp = take((size_t)s * vocab * d * 4);
    }
    if (dtype == 0 && grad_dtype == 1) {
      L.coef = take((size_t)L.cap * 4);
      L.cids = take((size_t)L.cap * 4);
      L.sampled = take(sampled_dw_workspace_bytes(L.cap, d, vocab));
    }
    if (dtype == 0 && n_tok > L.cap) L.dwacc = take((size_t)vocab * d * 4);
  }
  L.total = off;
  return L;
}

#define ITL_CHECK_LAUNCH()         \
  do {                             \
    e = hipGetLastError();         \
    if (e != hipSuccess) return e; \
  } while (0)

template <bool kKeep>
void launch_ce_partial(const char* Hc, const char* W, const int32_t* ids, const int32_t* count, int c0, int cap, int d,
                       int vocab, float2* part, float* zy, float* logits, hipStream_t stream) {
  const int row_bytes = d * 2;
  const int S = n_slices(vocab), G = slices_per_group(cap, vocab), ntb = (int)ceil_div(cap, kBT);
  // Few workgroups: the narrow walk's blocks are a quarter of the wide one's
  // (two rounds of them over the CUs still half its time). The bits are the
  // same.
  const long long narrow = ceil_div(cap, kNarrowBRows) * S;
  if (narrow <= 512) {
    hipLaunchKernelGGL((ce_partial_narrow_kernel<0, kKeep, kNarrowBRows>), dim3((unsigned)narrow), dim3(kThreads), 0,
                       stream, Hc, W, ids, count, c0, cap, cap, row_bytes, vocab, S, part, zy, logits);
    return;
  }
  const dim3 grid((unsigned)ntb * (unsigned)n_slice_groups(cap, vocab));
  // the load schedule's rule as in the logprob's forward
  if (row_bytes / kStepBytes > kNearBMaxSteps)
    hipLaunchKernelGGL((ce_partial_kernel<0, kKeep, true>), grid, dim3(kThreads8), 0, stream, Hc, W, ids, count, c0,
                       cap, cap, row_bytes, vocab, S, G, part, zy, logits);
  else
    hipLaunchKernelGGL((ce_partial_kernel<0, kKeep, false>), grid, dim3(kThreads8), 0, stream, Hc, W, ids, count, c0,
                       cap, cap, row_bytes, vocab, S, G, part, zy, logits);
}

template <int kDtype>
hipError_t run_cross_entropy(const CeCall& c, hipStream_t stream) {
  using E = Elem<kDtype>;
  using T = typename E::T;
  const bool grad = c.dW != nullptr;
  if (c.n_tok == 0) {  // no token: loss 0, dW zeros
    hipLaunchKernelGGL(ce_clear_kernel, dim3(1), dim3(256), 0, stream, reinterpret_cast<uint4*>(c.loss), 0LL, c.loss);
    if (grad) {
      const long long n16 = c.vocab * c.d * (c.grad_dtype == 0 ? 2 : 4) / 16;
      hipLaunchKernelGGL(ce_clear_kernel, flat_grid(ceil_div(n16, 256)), dim3(256), 0, stream,
                         static_cast<uint4*>(c.dW), n16, nullptr);
    }
    return hipGetLastError();
  }
  const CeLayout L = ce_layout(c.n_tok, c.d, c.vocab, kDtype, grad, c.grad_dtype);
  char* ws = static_cast<char*>(c.workspace);
  auto at = [&](size_t off) { return ws + off; };
  int32_t* rows = reinterpret_cast<int32_t*>(at(L.rows));
  int32_t* ids = reinterpret_cast<int32_t*>(at(L.ids));
  int32_t* slot = reinterpret_cast<int32_t*>(at(L.slot));
  int32_t* count = reinterpret_cast<int32_t*>(at(L.count));
  float* lp = reinterpret_cast<float*>(at(L.lp));
  float* lse = reinterpret_cast<float*>(at(L.lse));
  float* zy = reinterpret_cast<float*>(at(L.zy));
  float2* part = reinterpret_cast<float2*>(at(L.part));
  double* loss_part = reinterpret_cast<double*>(at(L.loss));
  float* wmean = c.smoothing > 0.0f ? reinterpret_cast<float*>(at(L.wmean)) : nullptr;
  float* wpart = reinterpret_cast<float*>(at(L.wpart));
  char* Hc = at(L.hc);
  const T* H = static_cast<const T*>(c.H);
  const T* W = static_cast<const T*>(c.W);
  const int n = (int)c.n_tok, d = (int)c.d, vocab = (int)c.vocab, S = n_slices(vocab);
  const int row_chunks = d * E::kSize / 16;
  hipError_t e;

  // A few tokens without their gradient: a block or two hold them all, counted
  // or not, so nothing is gathered.
  const bool direct = !grad && !wmean && n <= kNarrow128MaxTokens;
  if (!direct) {
    hipLaunchKernelGGL(ce_select_kernel, dim3(1), dim3(kSelectThreads), 0, stream, c.targets, n, vocab, rows, ids, slot,
                         count, grad ? reinterpret_cast<int32_t*>(at(L.splits)) : nullptr, L.cap, GradTile<kDtype>::kRows,
                       L.parts, (int)ceil_div(d, GradTile<kDtype>::kRows), L.vpad / GradTile<kDtype>::kStepK, kDtype);
    ITL_CHECK_LAUNCH();
  }
  if (wmean) {
    const int nb = (int)ceil_div(vocab, kMeanRows);
    hipLaunchKernelGGL(ce_colsum_kernel<kDtype>, dim3((unsigned)nb, (unsigned)ceil_div(d, 512)), dim3(256), 0, stream, W,
                       vocab, d, wpart);
    hipLaunchKernelGGL(ce_colmean_kernel, dim3((unsigned)(d / 64)), dim3(1024), 0, stream, wpart, nb, d, vocab,
                       wmean);
    ITL_CHECK_LAUNCH();
  }
  GradScale gs{c.smoothing, c.z_weight, c.grad_scale, 1.0f / (float)vocab, c.mean};
  const bool exact = grad && kDtype == 0 && c.grad_dtype == 1;
  const bool row_grad = grad && kDtype == 1 && vocab <= kGradRowVocab;
  for (long long first = 0; first < n; first += L.cap) {
    const int c0 = (int)first;
    const int cap = std::min(L.cap, n - c0);
    if (!direct)
      hipLaunchKernelGGL(ce_gather_kernel, flat_grid(c0 == 0 ? n : cap), dim3(256), 0, stream,
                         reinterpret_cast<const uint4*>(H), rows, slot, count, c0, cap, L.parts, row_chunks,
                         reinterpret_cast<uint4*>(Hc), c0 == 0 ? static_cast<uint4*>(c.dH) : nullptr,
                         d * (c.grad_dtype == 0 ? 2 : 4) / 16, (long long)(c0 == 0 ? n : cap));
    float* z = reinterpret_cast<float*>(at(L.z));
    const char* h_rows = direct ? reinterpret_cast<const char*>(H) : Hc;
    const char* w_rows = reinterpret_cast<const char*>(W);
    const int32_t* y = direct ? c.targets : ids + c0;
    const int32_t* counted = direct ? nullptr : count;
    if constexpr (kDtype == 0) {
      if (grad) launch_ce_partial<true>(h_rows, w_rows, y, counted, c0, cap, d, vocab, part, zy, z, stream);
      else launch_ce_partial<false>(h_rows, w_rows, y, counted, c0, cap, d, vocab, part, zy, nullptr, stream);
      ITL_CHECK_LAUNCH();
      e = launch_lse_combine(part, zy, cap, 2 * S, lp + c0, lse + c0, stream);
      if (e != hipSuccess) return e;
    } else {
      const int n_vt = (int)ceil_div(vocab, kF32Tile);
      hipLaunchKernelGGL(ce_logits_f32_kernel, dim3((unsigned)(n_vt * ceil_div(cap, kF32Tile))), dim3(kF32Threads), 0, stream,
                         h_rows, w_rows, counted, c0, cap, d * 4, vocab, n_vt, z);
      if (row_grad)
        hipLaunchKernelGGL((ce_lse_f32_kernel<true>), dim3((unsigned)cap), dim3(256), 0, stream, z, y, counted, c0, cap, vocab,
                           lp + c0, lse + c0, gs, reinterpret_cast<float*>(at(L.gd)));
      else
        hipLaunchKernelGGL((ce_lse_f32_kernel<false>), dim3((unsigned)cap), dim3(256), 0, stream, z, y, counted, c0, cap, vocab,
                           lp + c0, lse + c0, gs, nullptr);
      ITL_CHECK_LAUNCH();
    }
    if (!grad) continue;

    T* Gd = reinterpret_cast<T*>(at(L.gd));
    const int g_rows = L.parts * cap;
    float* coef = exact ? reinterpret_cast<float*>(at(L.coef)) : nullptr;
    if (!row_grad) {
      hipLaunchKernelGGL(ce_grad_logits_kernel<kDtype>,
                         dim3((unsigned)(L.vpad / kBV), (unsigned)ceil_div(cap, 256 * kGradVec / kBV)), dim3(256), 0, stream,
                         z, ids + c0, count, c0, cap, L.parts, vocab, g_rows, lse + c0, gs, Gd, coef);
      ITL_CHECK_LAUNCH();
    }
    int32_t* cids = reinterpret_cast<int32_t*>(at(L.cids));
    if (exact) {
      hipLaunchKernelGGL(ce_rest_kernel, dim3((unsigned)ceil_div(cap, 256)), dim3(256), 0, stream, ids + c0, count, c0,
                         cap, gs, coef, cids);
      ITL_CHECK_LAUNCH();
    }
    // dH
    float* dhp = reinterpret_cast<float*>(at(L.dhp));
    constexpr int kT = GradTile<kDtype>::kRows;
    const dim3 g_block(kDtype == 0 ? kThreads8 : kF32Threads);
    const int n_dt = (int)ceil_div(d, kT), n_vt = (int)ceil_div(vocab, kT);
    // (a walk each for fewer than four rounds over the CUs leaves some idle at the end)
    const int walk = kDtype == 0 && (long long)n_vt * ceil_div(n_dt, kDwWalk) >= 1024 ? kDwWalk : 1;
    const int32_t* splits = reinterpret_cast<const int32_t*>(at(L.splits)) + c0 / L.cap;
    hipLaunchKernelGGL(ce_dh_kernel<kDtype>, dim3((unsigned)L.dh_groups), g_block, 0, stream,
                       reinterpret_cast<const char*>(W), reinterpret_cast<const char*>(Gd), vocab, L.vpad, d, count, c0, cap,
                       L.parts, g_rows, n_dt, splits, dhp);
    ITL_CHECK_LAUNCH();
    hipLaunchKernelGGL(ce_dh_finish_kernel<kDtype>, dim3((unsigned)cap, (unsigned)ceil_div(d, 4 * kDhFinish)),
                       dim3(kDhFinish), 0, stream, dhp, splits, cap, L.parts, d, rows,
                       ids + c0, count, c0, gs, coef, W, c.grad_dtype, c.dH);
    ITL_CHECK_LAUNCH();
    // dW
    const bool single = n <= L.cap;
    float* acc = single ? nullptr : c.grad_dtype == 1 && !exact ? static_cast<float*>(c.dW) : reinterpret_cast<float*>(at(L.dwacc));
    void* out = c.dW;
    int add = 0, out_f32 = c.grad_dtype;
    if (exact) {
      // the chunk's targets' rests first (every row of the target is written), then the contraction on top
      float* target = single ? static_cast<float*>(c.dW) : c0 == 0 ? static_cast<float*>(c.dW) : acc;
      e = launch_sampled_dw(Hc, kDtype, cap, d, vocab, cids, coef, target, at(L.sampled), stream);
      if (e != hipSuccess) return e;
      out = target, add = 1;
    } else if (!single) {
      out = acc, out_f32 = 1, add = c0 > 0;
    }
    auto dw = [&](auto mode) {
      if constexpr (kDtype == 0 && decltype(mode)::value != kDwWrite) {  // (kDwWrite: of several chunks)
        if (n <= kFewTokens) {
          const int n_dt2 = (int)ceil_div(d, kFewTile), n_vt2 = (int)ceil_div(vocab, kFewTile);
          hipLaunchKernelGGL((ce_dw_few_kernel<decltype(mode)::value>), dim3((unsigned)(n_vt2 * n_dt2)), dim3(kFewThreads), 0,
                             stream, reinterpret_cast<const char*>(Gd), Hc, g_rows, count, c0, cap, L.parts, vocab, d, n_dt2, gs,
                             out);
          return;
        }
      }
      const int splits = dw_splits(cap, d, vocab, kDtype);
      if (splits > 1) {
        float* dwp = reinterpret_cast<float*>(at(L.dwp));
        hipLaunchKernelGGL((ce_dw_kernel<kDtype, kDwPart>), dim3((unsigned)(n_vt * n_dt * splits)), g_block, 0,
                           stream, reinterpret_cast<const char*>(Gd), Hc, g_rows, count, c0, cap, vocab, d, n_vt, n_dt, 1, gs,
                           dwp);
        hipLaunchKernelGGL((ce_dw_finish_kernel<decltype(mode)::value>),
                           dim3((unsigned)ceil_div((long long)vocab * d, 1024)), dim3(256), 0, stream, dwp, splits,
                           (long long)vocab * d, count, gs, out);
        return;
      }
      hipLaunchKernelGGL((ce_dw_kernel<kDtype, decltype(mode)::value>), dim3((unsigned)dw_groups(n_vt, ceil_div(n_dt, walk))),
                         g_block, 0, stream, reinterpret_cast<const char*>(Gd), Hc, g_rows, count, c0, cap, vocab, d, n_vt,
                         n_dt, walk, gs, out);
    };
    if (add) dw(std::integral_constant<int, kDwAdd>{});
    else if (kDtype == 1 || out_f32) dw(std::integral_constant<int, kDwWrite>{});
    else if constexpr (kDtype == 0) dw(std::integral_constant<int, kDwRound>{});
    ITL_CHECK_LAUNCH();
    if (exact && !single && c0 > 0) {
      hipLaunchKernelGGL(ce_add_kernel, flat_grid(ceil_div((long long)vocab * d / 4, 256)), dim3(256), 0, stream,
                         reinterpret_cast<const float4*>(acc), (long long)vocab * d / 4, static_cast<float4*>(c.dW));
      ITL_CHECK_LAUNCH();
    }
    if (!exact && !single && first + L.cap >= n && c.grad_dtype == 0) {
      hipLaunchKernelGGL(ce_round_kernel, flat_grid(ceil_div((long long)vocab * d / 4, 256)), dim3(256), 0, stream,
                         reinterpret_cast<const float4*>(acc), (long long)vocab * d / 4, static_cast<uint2*>(c.dW));
      ITL_CHECK_LAUNCH();
    }
  }
  if (!wmean && n <= kSmallTokens) {
    hipLaunchKernelGGL(ce_small_loss_kernel, dim3(1), dim3(1024), 0, stream, c.targets, n, vocab, direct ? nullptr : slot,
                       direct ? nullptr : count, lp, lse, c.z_weight, c.mean, c.token_loss, c.lse, c.loss);
  } else {
    hipLaunchKernelGGL(ce_token_loss_kernel<kDtype>, flat_grid(ceil_div(n, 4)), dim3(256), 0, stream, H, n, d, slot, lp,
                       lse, wmean, c.smoothing, c.z_weight, c.token_loss, c.lse, loss_part);
    hipLaunchKernelGGL(ce_loss_kernel, dim3(1), dim3(1024), 0, stream, loss_part, (int)ceil_div(n, 4), count, c.mean,
                       c.loss);
  }
  ITL_CHECK_LAUNCH();
  return hipSuccess;
}

}  // namespace

size_t cross_entropy_workspace_bytes(long long n_tok, long long d, long long vocab, int dtype, bool grad, int grad_dtype) {
  return n_tok <= 0 ? 0 : ce_layout(n_tok, d, vocab, dtype, grad, grad_dtype).total;
}

hipError_t launch_cross_entropy(const CeCall& c, hipStream_t stream) {
  return c.dtype == 0 ? run_cross_entropy<0>(c, stream) : run_cross_entropy<1>(c, stream);
}

}  // namespace itl
