// Tile products whose operands lie with the contracted index outermost
// (K-major: row k holds the tile's 256 columns), as a gradient's do: dH = G W
// contracts W's rows, dW = G^T H the rows of both. Transposed copies of W, G
// and H are not made: the operand comes into LDS as it lies, and the fragments
// are read through the transposing LDS read.
//
// bf16 (run_tiles_km): 256 x 256 tiles on the eight-wavefront schedule of
// tile_engine8.h (same wavefront tiles, slots, barriers and load places). A
// K step of a K-major operand is 64 rows of 512 bytes, 32 KiB, one slot. The
// read (ds_read_b64_tr_b16, measured layout): in each group of 16 lanes, lane
// a addresses 8 bytes, row k0 + a / 4, columns 4 (a mod 4) .. + 3, and lane i
// receives column i of rows k0 .. k0 + 3. Two reads give a lane the 8 values
// of k that the K-contiguous operand's 16-byte chunk holds, so both kinds
// meet in one instruction. The 32-byte piece (16 columns) P of row k sits at
// piece P ^ f(k), f(k) = (k mod 4) + 4 (bit 4 of k) + 8 (bit 3 of k): the 8
// rows that lanes 0-31 (or 32-63) read, whose k differ in bits 0, 1 and 4 (see
// lane_chunk), fall on 8 pieces that cover all 64 banks.
//
// fp32 (run_tile_f32): 64 x 64 tiles, four wavefronts of 32 x 32. The fp32
// matrix rate is a sixteenth of bf16's, so such a tile is bound by it all the
// same and small problems fill the chip; lanes read single values, row by
// row, which needs no transposing.
#pragma once

#include "tile_engine.h"
#include "tile_engine8.h"

namespace itl {

typedef short shortx4 __attribute__((ext_vector_type(4)));

// An operand of a tile: `base` its first row k (K-major: at the tile's first
// column; K-contiguous: row 0 of the tile at the first k), rows or columns
// past it never read.
// A K-contiguous operand may lie in blocks of 2^block_shift K steps (rows of one
// block side by side, block_bytes between blocks; 0: whole rows): base is the
// tile's first row in block 0 then, and `first` the first step.
struct KmOperand {
  const char* base;
  uint32_t row_bytes;  // between rows
  int rows;            // K-major: rows k in all; K-contiguous: the tile's rows
  uint32_t skip;       // bytes before base in its row (the range ends with the last row)
  int block_shift = 0, first = 0;
  size_t block_bytes = 0;
};

// Step s of a K-contiguous operand: its buffer range and the offset in a row.
__device__ __forceinline__ int4v contiguous_rsrc(const KmOperand& o, int s, uint32_t* off) {
  const uint32_t n = (uint32_t)o.rows * o.row_bytes - o.skip;
  if (o.block_shift == 0) {
    *off = (uint32_t)s * kStepBytes;
    return rsrc_words(o.base, n);
  }
  const uint32_t at = (uint32_t)(o.first + s), block = at >> o.block_shift;
  *off = (at - (block << o.block_shift)) * kStepBytes;
  return rsrc_words(o.base + block * o.block_bytes, n);
}

// K-major rows 64 s .. of a K step as a buffer range: rows past the end load
// zeros.
__device__ __forceinline__ int4v km_step_rsrc(const KmOperand& o, int s, int step_rows) {
  const int left = o.rows - s * step_rows;
  const uint32_t n = left <= 0 ? 0u : (uint32_t)(left < step_rows ? left : step_rows) * o.row_bytes - o.skip;
  return rsrc_words(o.base + (size_t)s * step_rows * o.row_bytes, n);
}

__device__ __forceinline__ int km_swz(int k) { return (k & 3) | (((k >> 4) & 1) << 2) | (((k >> 3) & 1) << 3); }

// For tiles tile_begin .. tile_end - 1 of A (a tile's columns 512 bytes behind
// the last one's; A is given at column 0, skip 0): acc = A_tile B^T over nks
// steps of 64 k, A K-major, B K-major or K-contiguous (kBMajor). epi(tile, acc)
// as in run_tiles8 (smem 1 KiB aligned): acc[bm][bn][i] is A column 128 wv + 16 bm + 4 quad + i
// against B 64 tq + 16 bn + c16. The next tile's first steps are loaded while
// a tile ends and is stored. All 512 threads call this.
// The far operand (three slots, loaded two steps ahead) is A, with kBFar B.
template <bool kBMajor, bool kBFar, class Epi>
__device__ __forceinline__ void run_tiles_km(uint4* smem, const Lanes8& L, const KmOperand& A, const KmOperand& B,
                                             int tile_begin, int tile_end, int nks, Epi&& epi) {
  constexpr int kAS = kBFar ? kHSlots : kWSlots, kBS = kBFar ? kWSlots : kHSlots;
  const int lane = L.lane, wave = L.wave, quad = L.quad, c16 = L.c16;
  const uint32_t lds0 = (uint32_t)(size_t)((__attribute__((address_space(3))) uint4*)smem);
  const uint32_t my_rows = (uint32_t)wave * 32 * kStepBytes;  // a wavefront's 4 KiB of a slot, either kind

  // Loads. K-major: load j of wavefront w fetches rows 8 w + 2 j + (lane / 32)
  // at the chunk that belongs at position lane mod 32. K-contiguous: as in
  // run_tiles8. Offsets less 1024 j for dma16x4, which underflow only for
  // rows of less than 512 bytes: those are loaded one by one.
  auto offsets = [&](uint32_t (&voff)[4], bool major, uint32_t row_bytes) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (major) {
        const int k = 8 * wave + 2 * j + (lane >> 5);
        voff[j] = (uint32_t)k * row_bytes + (uint32_t)(((lane & 31) ^ (2 * km_swz(k))) * 16);
      } else {
        const int lr = lane >> 3;
        voff[j] = (uint32_t)(wave * 32 + j * kDmaRows + lr) * row_bytes + (((lane & 7) ^ lr ^ (j & 1)) * 16);
      }
    }
  };
  uint32_t avoff[4], bvoff[4];
  offsets(avoff, true, A.row_bytes);
  offsets(bvoff, kBMajor, B.row_bytes);
  const bool a_four = A.row_bytes >= 512, b_four = !kBMajor || B.row_bytes >= 512;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (a_four) avoff[j] -= 1024u * j;
    if (b_four) bvoff[j] -= 1024u * j;
  }
  auto load = [&](const int4v& r, const uint32_t (&voff)[4], uint32_t soff, uint32_t lds, bool four) {
    if (four) {
      dma16x4(r, voff, soff, lds);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) dma16(r, voff[j], soff, lds + 1024u * j);
    }
  };
  // Each operand's loads come in step order: running counts of the step
  // within the tile. A step past the end loads the last one again into a slot
  // nothing reads.
  int a_tile = tile_begin, a_ks = 0, b_ks = 0, b_left = (tile_end - tile_begin) * nks;
  auto a_load = [&](int s) {
    const uint32_t at = (uint32_t)a_tile * 512u;
    load(km_step_rsrc(KmOperand{A.base + at, A.row_bytes, A.rows, at}, a_ks, 64), avoff, 0u,
         lds0 + (uint32_t)(s % kAS) * kSlotBytes + my_rows, a_four);
    if (a_ks + 1 < nks) ++a_ks;
    else if (a_tile + 1 < tile_end) a_ks = 0, ++a_tile;
    a_ks = __builtin_amdgcn_readfirstlane(a_ks);
    a_tile = __builtin_amdgcn_readfirstlane(a_tile);
  };
  auto b_load = [&](int s) {
    const uint32_t lds = lds0 + (uint32_t)(kAS + s % kBS) * kSlotBytes + my_rows;
    if constexpr (kBMajor) {
      load(km_step_rsrc(B, b_ks, 64), bvoff, 0u, lds, b_four);
    } else {
      uint32_t off;
      const int4v r = contiguous_rsrc(B, b_ks, &off);
      load(r, bvoff, off, lds, true);
    }
    if (--b_left > 0) b_ks = b_ks + 1 < nks ? b_ks + 1 : 0;
    b_ks = __builtin_amdgcn_readfirstlane(b_ks);
  };

  // Fragment addresses within a slot (bytes). K-major block b, half kk, part
  // p: row 32 kk + 8 lane_chunk(quad) + 4 p + c16 / 4, piece b ^ f. A block's
  // number enters bits 5 and up by an exclusive or alone, so one register
  // serves all blocks.
  const int krow = 8 * lane_chunk(quad) + (c16 >> 2);
  const int f = km_swz(krow);  // (bits 2 and 5 of the row do not enter)
  const uint32_t a_off = (uint32_t)(krow * 512 + ((L.wv * 8) ^ f) * 32 + (c16 & 3) * 8);
  const uint32_t b_off = (uint32_t)(krow * 512 + ((L.tq * 4) ^ f) * 32 + (c16 & 3) * 8);
  int bc_off[2];
#pragma unroll
  for (int kk = 0; kk < 2; ++kk) bc_off[kk] = (L.tq * 64 + c16) * kRowChunks + ((4 * kk + lane_chunk(quad)) ^ swz(c16));

  typedef __attribute__((address_space(3))) shortx4 lds_s4;
  auto tr8 = [&](uint32_t at) {
    const shortx4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)(size_t)at);
    const shortx4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)(size_t)(at + 4 * 512));
    const uint2 a = __builtin_bit_cast(uint2, lo), b = __builtin_bit_cast(uint2, hi);
    return make_uint4(a.x, a.y, b.x, b.y);
  };

  auto near_load = [&](int s) {
    if constexpr (kBFar) a_load(s);
    else b_load(s);
  };
  auto far_load = [&](int s) {
    if constexpr (kBFar) b_load(s);
    else a_load(s);
  };
  near_load(0);
  far_load(0);
  near_load(1);
  far_load(1);
  wait_and_barrier<2 * kDma8PerWave>();
  __builtin_amdgcn_sched_barrier(0);

  uint4 FA[2][2], FB[2][4];
  auto read_a = [&](int s, int kk, int bm) {
    FA[(bm >> 1) & 1][bm & 1] = tr8(((lds0 + (uint32_t)(s % kAS) * kSlotBytes + a_off) ^ (uint32_t)(bm * 32)) + (uint32_t)kk * (32 * 512));
  };
  auto read_b = [&](int s, int kk, int bn) {
    if constexpr (kBMajor)
      FB[kk][bn] = tr8(((lds0 + (uint32_t)(kAS + s % kBS) * kSlotBytes + b_off) ^ (uint32_t)(bn * 32)) + (uint32_t)kk * (32 * 512));
    else
      FB[kk][bn] = smem[(kAS + s % kBS) * kSlotChunks + bc_off[kk] + bn * 16 * kRowChunks];
  };
  floatx4 acc[8][4];
  auto zero_acc = [&]() {
#pragma unroll
    for (int bm = 0; bm < 8; ++bm)
#pragma unroll
      for (int bn = 0; bn < 4; ++bn) acc[bm][bn] = floatx4{};
  };
  // the sub-steps of run_tiles8
  auto sub = [&](auto J, auto next, int s) {
    constexpr int j = decltype(J)::value;
    constexpr int kk = j >> 2, p = j & 3;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int b = q >> 2, bn = q & 3;
      Mma16<0>::step(acc[2 * p + b][bn], FA[p & 1][b], FB[kk][bn]);
      if constexpr (j < 6) {
        if (q < 2) read_a(s, (j + 1) >> 2, 2 * ((j + 1) & 3) + q);
        if (j < 4 && q == 2) read_b(s, 1, j);
      } else if constexpr (j == 6) {
        if (q < 2) read_a(s, 1, 6 + q);
        if (q == 5) {
          wait_and_barrier<kDma8PerWave>();
          near_load(s + 2);
        }
        if (decltype(next)::value && q >= 6) read_b(s + 1, 0, q - 6);
      } else {
        if (decltype(next)::value && q < 2) read_a(s + 1, 0, q);
        if (decltype(next)::value && (q == 2 || q == 3)) read_b(s + 1, 0, q);
      }
      if constexpr (j == 0) {
        if (q == 3) far_load(s + 2);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  auto k_step = [&](int s, auto next) {
    sub(std::integral_constant<int, 0>{}, next, s);
    sub(std::integral_constant<int, 1>{}, next, s);
    sub(std::integral_constant<int, 2>{}, next, s);
    sub(std::integral_constant<int, 3>{}, next, s);
    sub(std::integral_constant<int, 4>{}, next, s);
    sub(std::integral_constant<int, 5>{}, next, s);
    sub(std::integral_constant<int, 6>{}, next, s);
    sub(std::integral_constant<int, 7>{}, next, s);
  };
  auto read_first = [&](int s) {
    read_a(s, 0, 0);
    read_a(s, 0, 1);
#pragma unroll
    for (int bn = 0; bn < 4; ++bn) read_b(s, 0, bn);
  };
  zero_acc();
  read_first(0);
  int s = 0;
  for (int tile = tile_begin; tile < tile_end; ++tile) {
    for (int ks = 0; ks + 1 < nks; ++ks, ++s) k_step(s, std::true_type{});
    k_step(s, std::false_type{});
    ++s;
    epi(tile, acc);
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
    zero_acc();
    if (tile + 1 < tile_end) read_first(s);
  }
  // loads of the steps past the end may still be writing LDS
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

// ---- bf16, few k

// A product over few k is bound by its results' stores, not its contraction:
// 128 x 128 tiles (four wavefronts of 64 x 64), 32 KiB of LDS and at most 128
// registers, so that four workgroups per CU have stores and loads in flight
// at once where the 256 x 256 tile has one. Both operands K-major, rows of 256
// bytes in LDS; the 32-byte piece P of row k sits at P ^ g(k), g(k) = (k mod 4)
// + 4 (bit 4 of k).
constexpr int kFewTile = 128;
constexpr int kFewThreads = 256;
constexpr int kFewSmemChunks = 2 * 64 * 256 / 16;

__device__ __forceinline__ int few_swz(int k) { return (k & 3) | (((k >> 4) & 1) << 2); }

// acc = A B^T over the operands' rows, 64 at a time: wavefront w holds A
// columns 64 (w mod 2) .. against B 64 (w / 2) ..; acc[bm][bn][i] is A 64 (w &
// 1) + 16 bm + 4 quad + i, B 64 (w >> 1) + 16 bn + c16.
template <class Epi>
__device__ __forceinline__ void run_tile_few(uint4* smem, const KmOperand& A, const KmOperand& B, Epi&& epi) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int quad = lane >> 4, c16 = lane & 15;
  const uint32_t lds0 = (uint32_t)(size_t)((__attribute__((address_space(3))) uint4*)smem);
  // load j of wavefront w: rows 16 w + 4 j + lane / 16 of either operand
  uint32_t ao[4], bo[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int k = 16 * wave + 4 * j + (lane >> 4);
    const uint32_t chunk = (uint32_t)(((lane & 15) ^ (2 * few_swz(k))) * 16);
    ao[j] = (uint32_t)k * A.row_bytes + chunk;
    bo[j] = (uint32_t)k * B.row_bytes + chunk;
  }
  const int krow = 8 * lane_chunk(quad) + (c16 >> 2);
  const int f = few_swz(krow);
  typedef __attribute__((address_space(3))) shortx4 lds_s4;
  auto tr8 = [&](uint32_t at) {
    const shortx4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)(size_t)at);
    const shortx4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)(size_t)(at + 4 * 256));
    const uint2 a = __builtin_bit_cast(uint2, lo), b = __builtin_bit_cast(uint2, hi);
    return make_uint4(a.x, a.y, b.x, b.y);
  };
  const uint32_t at0 = lds0 + (uint32_t)(krow * 256 + (c16 & 3) * 8);
  floatx4 acc[4][4];
#pragma unroll
  for (int bm = 0; bm < 4; ++bm)
#pragma unroll
    for (int bn = 0; bn < 4; ++bn) acc[bm][bn] = floatx4{};
  const int steps = (A.rows + 63) / 64;
  for (int s = 0; s < steps; ++s) {
    const int4v ar = km_step_rsrc(A, s, 64), br = km_step_rsrc(B, s, 64);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      dma16(ar, ao[j], 0u, lds0 + (uint32_t)(wave * 4096 + j * 1024));
      dma16(br, bo[j], 0u, lds0 + 16384u + (uint32_t)(wave * 4096 + j * 1024));
    }
    wait_and_barrier<0>();
    const int halves = A.rows - 64 * s > 32 ? 2 : 1;
    for (int kk = 0; kk < halves; ++kk) {
      uint4 a[4], b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = tr8(at0 + (uint32_t)(kk * 32 * 256 + ((4 * (wave & 1) + i) ^ f) * 32));
        b[i] = tr8(at0 + 16384u + (uint32_t)(kk * 32 * 256 + ((4 * (wave >> 1) + i) ^ f) * 32));
      }
#pragma unroll
      for (int bm = 0; bm < 4; ++bm)
#pragma unroll
        for (int bn = 0; bn < 4; ++bn) Mma16<0>::step(acc[bm][bn], a[bm], b[bn]);
    }
    __syncthreads();  // every wavefront is done with the step's rows
  }
  epi(acc, wave, quad, c16);
}

// ---- fp32

constexpr int kF32Tile = 64;
constexpr int kF32StepK = 32;                                            // 128 bytes of a K-contiguous row
constexpr int kF32SlotBytes = kF32Tile * kF32StepK * 4;                  // 8 KiB, either kind
constexpr int kF32Slots = 3;                                             // per operand, loaded two steps ahead
constexpr int kF32SmemChunks = 2 * kF32Slots * kF32SlotBytes / 16;       // 48 KiB: three workgroups per CU
constexpr int kF32Threads = 256;

// acc = A B^T over nks steps of 32 k, 64 x 64: wavefront w holds A columns
// 32 (w mod 2) .. against B 32 (w / 2) .., as 2 x 2 blocks; acc[bm][bn][i] is
// A 32 (w & 1) + 16 bm + 4 quad + i, B 32 (w >> 1) + 16 bn + c16. Each operand
// is K-major or K-contiguous. K-major rows are 256 bytes; their 64-byte piece
// (16 columns) P of row k sits at P ^ ((k / 4) mod 4).
// Sums of kF32Fold steps (64 k) are added to the total one by one: one chain
// of k / 4 dependent additions of a growing sum lost up to 8e-6 of a logit at
// 5056 k where the terms agree in sign; 16 additions, then k / 64 do not.
constexpr int kF32Fold = 2;
template <bool kAMajor, bool kBMajor, class Epi>
__device__ __forceinline__ void run_tile_f32(uint4* smem, const KmOperand& A, const KmOperand& B, int nks, Epi&& epi) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int quad = lane >> 4, c16 = lane & 15;
  const uint32_t lds0 = (uint32_t)(size_t)((__attribute__((address_space(3))) uint4*)smem);
  // two loads per operand, step and wavefront: 2 KiB of the 8 KiB slot
  auto offset = [&](int j, bool major, uint32_t row_bytes) -> uint32_t {
    if (major) {  // rows 8 w + 4 j + lane / 16
      const int k = 8 * wave + 4 * j + (lane >> 4);
      return (uint32_t)k * row_bytes + (uint32_t)(((lane & 15) ^ (4 * ((k >> 2) & 3))) * 16);
    }
    const int lr = lane >> 3;  // rows 16 w + 8 j + lane / 8
    return (uint32_t)(16 * wave + 8 * j + lr) * row_bytes + (((lane & 7) ^ lr ^ (j & 1)) * 16);
  };
  const uint32_t ao[2] = {offset(0, kAMajor, A.row_bytes), offset(1, kAMajor, A.row_bytes)};
  const uint32_t bo[2] = {offset(0, kBMajor, B.row_bytes), offset(1, kBMajor, B.row_bytes)};
  auto load = [&](int s) {
    const int st = s < nks ? s : nks - 1;
    const uint32_t slot = (uint32_t)(s % kF32Slots) * kF32SlotBytes + (uint32_t)wave * 2048u;
    uint32_t a_off = 0u, b_off = 0u;
    const int4v ar = kAMajor ? km_step_rsrc(A, st, kF32StepK) : contiguous_rsrc(A, st, &a_off);
    const int4v br = kBMajor ? km_step_rsrc(B, st, kF32StepK) : contiguous_rsrc(B, st, &b_off);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      dma16(ar, ao[j], a_off, lds0 + slot + 1024u * j);
      dma16(br, bo[j], b_off, lds0 + kF32Slots * kF32SlotBytes + slot + 1024u * j);
    }
  };
  const float* lds_f = reinterpret_cast<const float*>(smem);
  floatx4 acc[2][2], total[2][2];
#pragma unroll
  for (int bm = 0; bm < 2; ++bm)
#pragma unroll
    for (int bn = 0; bn < 2; ++bn) acc[bm][bn] = total[bm][bn] = floatx4{};
  load(0);
  load(1);
  for (int s = 0; s < nks; ++s) {
    if (s % kF32Fold == 0 && s > 0) {
#pragma unroll
      for (int bm = 0; bm < 2; ++bm)
#pragma unroll
        for (int bn = 0; bn < 2; ++bn) {
          total[bm][bn] += acc[bm][bn];
          acc[bm][bn] = floatx4{};
        }
    }
    // step s landed (step s + 1 may be in flight); every wavefront is done
    // with step s - 1, whose slot takes step s + 2
    wait_and_barrier<4>();
    load(s + 2);
    const int slot = (s % kF32Slots) * (kF32SlotBytes / 4);
    const float* sa = lds_f + slot;
    const float* sb = lds_f + kF32Slots * (kF32SlotBytes / 4) + slot;
    // the four values of a block's column (or row) c16 in half kk: k = 16 kk +
    // 4 lane_chunk(quad) + j
    auto fragment = [&](auto major, const float* t, int block, int kk, float (&v)[4]) {
      if constexpr (decltype(major)::value) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int k = 16 * kk + 4 * lane_chunk(quad) + j;
          v[j] = t[k * 64 + ((block ^ ((k >> 2) & 3)) * 16) + c16];
        }
      } else {
        const int row = 16 * block + c16;
        const float4 w = reinterpret_cast<const float4*>(t)[row * kRowChunks + ((4 * kk + lane_chunk(quad)) ^ swz(c16))];
        v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w;
      }
    };
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      float a[2][4], b[2][4];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        fragment(std::integral_constant<bool, kAMajor>{}, sa, 2 * (wave & 1) + t, kk, a[t]);
        fragment(std::integral_constant<bool, kBMajor>{}, sb, 2 * (wave >> 1) + t, kk, b[t]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int bm = 0; bm < 2; ++bm)
#pragma unroll
          for (int bn = 0; bn < 2; ++bn)
            acc[bm][bn] = __builtin_amdgcn_mfma_f32_16x16x4f32(a[bm][j], b[bn][j], acc[bm][bn], 0, 0, 0);
    }
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#pragma unroll
  for (int bm = 0; bm < 2; ++bm)
#pragma unroll
    for (int bn = 0; bn < 2; ++bn) total[bm][bn] += acc[bm][bn];
  epi(total, wave, quad, c16);
}

}  // namespace itl
