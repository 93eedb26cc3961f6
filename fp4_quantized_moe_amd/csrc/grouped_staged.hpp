// LDS-staged grouped GEMM for MXFP4 and bf16 operands.  The contraction runs
// along the rows of the routed operand and along the weights' rows (weights
// [E, N, K]) or, with kOpBf16T, down their columns (weights [E, K, N]).
//
// A stage is 128 bytes of K (256 MXFP4 or 64 bf16 elements) of TN weight and
// TM routed rows; two stages in LDS.  128 bytes are one cache line, so every
// staging instruction reads whole lines (8 rows of 8 chunks).  Row r keeps its
// chunk c in slot c ^ (r / 2 % 8): 16 consecutive rows of a fragment read then
// take each of the 16-byte groups of the 64 banks (two rows of 128 bytes)
// once, and the permutation is applied to the source address of the DMA,
// within the line.
//
// With kOpBf16T the weights' part of a stage is 64 rows k of TN columns, and
// fragments are gathered by the transposing LDS read: a group of 16 lanes
// reads 4 rows of 16 columns, and each lane receives one column's 4 values.
// Chunk c of row k sits in slot c ^ 4 (k % 4), so that the 4 rows of a group
// and the two groups of a 32-column fragment lie in different banks.
//
// One stage is four MFMA steps; in step s lanes 0-31 contract chunk s and
// lanes 32-63 chunk 4 + s, so a lane's four MXFP4 block scales of the stage
// are one dword, whose byte s the matrix instruction selects.
//
// Pipeline: step s + 1's fragments are read while step s is multiplied.  The
// last step of a stage is held back: its fragments are in registers, so after
// one barrier the stage's LDS is free (the DMA of the next but one stage
// starts) and the next stage has landed (its first fragments are read under
// the held-back step's MFMAs).  One barrier a stage, no exposed LDS latency.
#pragma once

#include <type_traits>
#include <utility>

#include "grouped_dma.hpp"
#include "grouped_direct.hpp"

namespace quads {

template <class F, int... I>
__device__ __forceinline__ void each_index(F &&f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
// f(integral_constant<int, 0>), ..., f(integral_constant<int, N - 1>).
template <int N, class F>
__device__ __forceinline__ void each(F &&f) {
  each_index(static_cast<F &&>(f), std::make_integer_sequence<int, N>{});
}

template <int OP_, int TM_, int TN_, int WM_, int WN_, bool ODD_ = false>
struct StagedCfg {
  static constexpr int OP = OP_, TM = TM_, TN = TN_, WM = WM_, WN = WN_;
  static constexpr int WAVES = WM * WN, THREADS = 64 * WAVES;
  static constexpr int MI = TM / WM / 32, NI = TN / WN / 32;  // 32 x 32 tiles of a wave
  static constexpr int ROWS = TM + TN;
  static constexpr int LOADS = ROWS / 8 / WAVES;       // staging instructions of a wave and stage
  static constexpr int WLOADS = TN / 8 / WAVES;        // the weights' part of them
  static constexpr bool MX = OP == kOpMx, TRANS = OP == kOpBf16T;
  // MXFP4 scale rows that are not dword-aligned (K % 128 != 0): the DMA does
  // not take them, and each lane loads its fragments' scales to registers.
  static constexpr bool ODD = ODD_, SLDS = MX && !ODD;
  static constexpr int KROWS = 512 / TN;  // kOpBf16T: weight rows of one staging instruction
  static constexpr int SLOADS = SLDS ? ROWS / 32 / WAVES : 0;  // scale instructions (32 rows each)
  static constexpr int STAGE = ROWS * 128 + (SLDS ? ROWS * 8 : 0);
  static constexpr int TURN = 2 * STAGE;  // LDS: two stages, then the epilogue's blocks,
  // Rows of the blocks that the epilogue turns around: whole lines, or half
  // ones for the small tile, of which two workgroups then fit a CU.
  static constexpr int RB = NI >= 4 ? 128 : 64, TURN_BYTES = 32 * RB;
  static constexpr int TOKENS = TURN + WAVES * TURN_BYTES;             // then the next tile's token ids
  static constexpr int LDS = TOKENS + 256 * WAVES;
  static constexpr int ALL = LOADS + SLOADS;
  // Staging instructions issued in a stage's last step and in the next
  // stage's first.  Three quarters and a quarter measured best (8192 x 8192 x
  // 16384 MXFP4: all in the last 518 us, 3 : 1 504, half and half 545).
  static constexpr int LATE = ALL * 3 / 4;
  static_assert(!MX || (TN % (32 * WAVES) == 0 && TM % (32 * WAVES) == 0), "a scale instruction reads one operand");
  static_assert(WAVES * KROWS % 4 == 0 || !TRANS, "slots of kOpBf16T");
  static_assert(64 * WAVES >= TM, "token ids of a tile");
  static_assert(TN % (8 * WAVES) == 0 && TM % (8 * WAVES) == 0 && (!MX || ROWS % (32 * WAVES) == 0), "staging split");
};

// Transposing LDS read of 16-bit values (see above).
__device__ __forceinline__ uint2 read_tr(const uint8_t *at) {
  typedef short s16x4 __attribute__((ext_vector_type(4)));
  typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
  const s16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(const_cast<uint8_t *>(at)));
  return __builtin_bit_cast(uint2, v);
}

// ---- epilogue ----------------------------------------------------------------
//
// A lane's four consecutive columns are 8 or 16 bytes of one row: stored from
// registers, an instruction touches 32 rows in 16-byte pieces (measured: the
// down projection's 537 MB of bf16 took 190 of its 352 us that way).  Each
// wave turns 32-row blocks around in LDS of its own instead and stores whole
// 128-byte lines, 8 rows an instruction.  Block row r keeps its 16-byte chunk
// c in slot c ^ (r / 2 % chunks); a wave's LDS accesses are in order, so no
// barrier is needed.

template <int RB>  // bytes of a block row: 64 or 128
__device__ __forceinline__ int turn_at(int row, int c) {
  return row * RB + 16 * (c ^ ((row >> 1) & (RB / 16 - 1)));
}

// One 32 x 32 tile as bf16 columns [32 i, 32 i + 32) of the block.
template <int RB>
__device__ __forceinline__ void turn_put_bf16(uint8_t *turn, int lane, int i, const float (&v)[16]) {
  const int half = lane >> 5, fr = lane & 31;
#pragma unroll
  for (int q = 0; q < 4; ++q)
    *reinterpret_cast<uint2 *>(turn + turn_at<RB>(fr, 4 * i + q) + 8 * half) =
        make_uint2(pack_bf16(v[4 * q], v[4 * q + 1]), pack_bf16(v[4 * q + 2], v[4 * q + 3]));
}

// The block's rows < rows to out (stride bytes apart); bytes at and behind
// `limit` of a row lie behind the last column and are not stored.  Stores that
// stream past the L2 leave it to the operands: 1060 -> 905 us for 8192 x
// 16384 x 8192 in bf16, 240 -> 200 us for the 537 MB of a down projection,
// and nowhere slower, down to outputs of 8 MB (17.5 -> 16.9 us).
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
template <int RB>
__device__ __forceinline__ void turn_store(const uint8_t *turn, int lane, uint8_t *out, int64_t stride, int rows, int limit) {
  constexpr int CH = RB / 16, PER = 64 / CH;  // rows of one instruction
#pragma unroll
  for (int j = 0; j < 32 / PER; ++j) {
    const int row = j * PER + lane / CH, c = (lane % CH) ^ ((row >> 1) & (CH - 1));
    const u32x4 v = *reinterpret_cast<const u32x4 *>(turn + row * RB + 16 * (lane % CH));
    if (row < rows && 16 * c < limit) __builtin_nontemporal_store(v, reinterpret_cast<u32x4 *>(out + row * stride + 16 * c));
  }
  __builtin_amdgcn_sched_barrier(0);  // block after block: all accumulators at once do not fit the other registers
}

// The reverse: global rows into the block (rows and columns outside: not loaded).
template <int RB>
struct TurnLoad {
  static constexpr int CH = RB / 16, PER = 64 / CH, N = 32 / PER;
  uint4 v[N];
  __device__ __forceinline__ void load(const uint8_t *in, int lane, int64_t stride, int rows, int limit) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int row = j * PER + lane / CH, c = (lane % CH) ^ ((row >> 1) & (CH - 1));
      v[j] = make_uint4(0, 0, 0, 0);
      if (row < rows && 16 * c < limit) v[j] = *reinterpret_cast<const uint4 *>(in + row * stride + 16 * c);
    }
  }
  __device__ __forceinline__ void put(uint8_t *turn, int lane) const {
#pragma unroll
    for (int j = 0; j < N; ++j) *reinterpret_cast<uint4 *>(turn + (j * PER + lane / CH) * RB + 16 * (lane % CH)) = v[j];
  }
};

// This lane's 16 values of the block's tile i.
template <int RB>
__device__ __forceinline__ void turn_get_bf16(const uint8_t *turn, int lane, int i, float (&v)[16]) {
  const int half = lane >> 5, fr = lane & 31;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint2 w = *reinterpret_cast<const uint2 *>(turn + turn_at<RB>(fr, 4 * i + q) + 8 * half);
    v[4 * q] = __uint_as_float(w.x << 16);
    v[4 * q + 1] = __uint_as_float(w.x & 0xFFFF0000u);
    v[4 * q + 2] = __uint_as_float(w.y << 16);
    v[4 * q + 3] = __uint_as_float(w.y & 0xFFFF0000u);
  }
}

// The lane's number, computed anew: what is derived from it is not kept in
// registers from before the loops, which have none to spare.
__device__ __forceinline__ int fresh_lane() {
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));
  return lane;
}

// A wave's accumulators a[i] (i-th 32 columns) of 32 rows: row0 is the first
// row's index in the output, rows how many exist, n0 the wave's first column.
// RB: bytes of a row of the block that is turned around.
template <int EPI, int NI, int RB>
__device__ __forceinline__ void store_block(const GroupedParams &p, const f32x16 (&a)[NI], uint8_t *turn, int lane,
                                            int64_t row0, int rows, int32_t n0) {
  if (rows <= 0) return;
  constexpr int TILES = RB / 64;  // 32-column bf16 tiles of a block
  float v[16];
  if constexpr (EPI == kEpiF32) {
    const int half = lane >> 5, fr = lane & 31;
    constexpr int COLS = RB / 4;
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int part = 0; part < 32 / COLS; ++part) {
#pragma unroll
        for (int q = 0; q < COLS / 8; ++q) {
          const int r = 4 * (q + part * (COLS / 8));
          *reinterpret_cast<float4 *>(turn + turn_at<RB>(fr, 2 * q + half)) =
              make_float4(a[i][r], a[i][r + 1], a[i][r + 2], a[i][r + 3]);
        }
        const int32_t n = n0 + 32 * i + COLS * part;
        turn_store<RB>(turn, lane, static_cast<uint8_t *>(p.y) + 4 * (row0 * p.width + n),
                       4 * static_cast<int64_t>(p.width), rows, 4 * (p.width - n));
      }
  } else if constexpr (EPI == kEpiBf16) {
#pragma unroll
    for (int i = 0; i < NI; i += TILES) {
#pragma unroll
      for (int t = 0; t < TILES; ++t) {
#pragma unroll
        for (int r = 0; r < 16; ++r) v[r] = a[i + t][r];
        turn_put_bf16<RB>(turn, lane, t, v);
      }
      const int32_t n = n0 + 32 * i;
      turn_store<RB>(turn, lane, static_cast<uint8_t *>(p.y) + 2 * (row0 * p.width + n),
                     2 * static_cast<int64_t>(p.width), rows, 2 * (p.width - n));
    }
  } else if constexpr (EPI == kEpiSwiglu) {
    constexpr int PAIRS = NI / 2;
    static_assert(PAIRS == TILES, "a block holds the wave's columns");
    const int64_t stride = 2 * static_cast<int64_t>(p.width);
    const int limit = 2 * (p.width - n0);
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) {
#pragma unroll
      for (int r = 0; r < 16; ++r) v[r] = silu(a[i][r]) * a[PAIRS + i][r];
      turn_put_bf16<RB>(turn, lane, i, v);
    }
    turn_store<RB>(turn, lane, static_cast<uint8_t *>(p.y) + row0 * stride + 2 * n0, stride, rows, limit);
    if (p.y2) {
#pragma unroll
      for (int part = 0; part < 2; ++part) {
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
#pragma unroll
          for (int r = 0; r < 16; ++r) v[r] = a[part * PAIRS + i][r];
          turn_put_bf16<RB>(turn, lane, i, v);
        }
        turn_store<RB>(turn, lane, static_cast<uint8_t *>(p.y2) + row0 * 2 * stride + part * stride + 2 * n0, 2 * stride,
                       rows, limit);
      }
    }
  } else {
    static_assert(EPI == kEpiSwigluMx, "kEpiGatedBwd has an epilogue of its own");
    constexpr int PAIRS = NI / 2;
    const int fr = lane & 31;
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) {
#pragma unroll
      for (int r = 0; r < 16; ++r) v[r] = silu(a[i][r]) * a[PAIRS + i][r];
      store_mx_block(v, lane, true, turn + fr * 16 * PAIRS + 16 * i, turn + 32 * 16 * PAIRS + fr * PAIRS + i);
    }
    const int row = lane / PAIRS, i = lane % PAIRS;
    const uint4 c = *reinterpret_cast<const uint4 *>(turn + 16 * (lane & (32 * PAIRS - 1)));
    const uint8_t s = turn[32 * 16 * PAIRS + (lane & (32 * PAIRS - 1))];
    if (lane < 32 * PAIRS && row < rows && n0 + 32 * i < p.width) {
      *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(p.y) + (row0 + row) * (p.width >> 1) + (n0 >> 1) + 16 * i) = c;
      static_cast<uint8_t *>(p.y2)[(row0 + row) * (p.width >> 5) + (n0 >> 5) + i] = s;
    }
    __builtin_amdgcn_sched_barrier(0);
  }
}

// The backward's epilogue: a[i] is dh; du and dg take the place of u and g.
// (Sending for the next block's gate and up while one is computed, from a
// second set of registers or from this one, measured slower: 515 - 535
// against 505 us for the layer.)
template <int RB>
struct GatedBlock {
  TurnLoad<RB> g, u;
  __device__ __forceinline__ void load(const GroupedParams &p, int lane, int64_t row0, int rows, int32_t n) {
    const int64_t stride = 4 * static_cast<int64_t>(p.width);  // bytes of a row [gate | up]
    const uint8_t *in = reinterpret_cast<const uint8_t *>(p.gu) + row0 * stride + 2 * n;
    g.load(in, lane, stride, rows, 2 * (p.width - n));
    u.load(in + 2 * static_cast<int64_t>(p.width), lane, stride, rows, 2 * (p.width - n));
  }
};

template <int RB>
__device__ __forceinline__ void store_gated_grad(const GroupedParams &p, const f32x16 (&d)[RB / 64], uint8_t *turn,
                                                 int lane, int64_t row0, int rows, int32_t n) {
  GatedBlock<RB> in;
  in.load(p, lane, row0, rows, n);
  constexpr int TILES = RB / 64;
  const int64_t stride = 4 * static_cast<int64_t>(p.width);
  uint8_t *out = static_cast<uint8_t *>(p.y) + row0 * stride + 2 * n;
  const int limit = 2 * (p.width - n);
  float g[TILES][16], u[TILES][16];
  in.g.put(turn, lane);
#pragma unroll
  for (int t = 0; t < TILES; ++t) turn_get_bf16<RB>(turn, lane, t, g[t]);
  in.u.put(turn, lane);
#pragma unroll
  for (int t = 0; t < TILES; ++t) turn_get_bf16<RB>(turn, lane, t, u[t]);
#pragma unroll
  for (int t = 0; t < TILES; ++t)
#pragma unroll
    for (int r = 0; r < 16; ++r) gated_grad(d[t][r], g[t][r], u[t][r]);
#pragma unroll
  for (int t = 0; t < TILES; ++t) turn_put_bf16<RB>(turn, lane, t, g[t]);
  turn_store<RB>(turn, lane, out, stride, rows, limit);
#pragma unroll
  for (int t = 0; t < TILES; ++t) turn_put_bf16<RB>(turn, lane, t, u[t]);
  turn_store<RB>(turn, lane, out + 2 * static_cast<int64_t>(p.width), stride, rows, limit);
}

// One workgroup's tiles.  Tiles are numbered columns fastest, each XCD owns a
// contiguous eighth (workgroups are dealt to the 8 XCDs in turn), so that the
// tiles running together on an XCD share an expert's weights and few row
// tiles in its L2; a workgroup takes every step-th tile of its XCD's.
struct StagedTile {
  int e;         // expert, or -1: no tile
  int32_t r0, rows, n0;
};

template <class C, int EPI>
__device__ __forceinline__ void staged_tiles(const GroupedParams &p, uint8_t *lds, uint32_t col_tiles) {
  constexpr bool PAIR = EPI == kEpiSwiglu || EPI == kEpiSwigluMx;
  constexpr int COLS = PAIR ? C::TN / 2 : C::TN;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), half = lane >> 5;
  const int wn = wave / C::WM, wm = wave % C::WM;

  // The tiles of this workgroup: at, at + step, ... below end.
  const uint32_t tiles = count_tiles<C::TM>(p.offsets, p.E) * col_tiles, per = (tiles + 7) / 8;
  const uint32_t step_tiles = gridDim.x / 8, end = min(tiles, ((blockIdx.x & 7) + 1) * per);
  uint32_t at = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
  if (at >= end) return;
  const TileAt t0 = find_tile<C::TM>(p.offsets, p.E, static_cast<int>(at / col_tiles));
  Walker walk(p.offsets, t0);
  StagedTile t{t0.e, t0.r0, t0.rows, static_cast<int32_t>(at % col_tiles) * COLS};
  const auto advance = [&](StagedTile &u) {
    at += step_tiles;
    u = StagedTile{-1, 0, 0, 0};
    if (at >= end) return;
    walk.to<C::TM>(static_cast<int32_t>(at / col_tiles), u.r0, u.rows);
    u.e = walk.e;
    u.n0 = static_cast<int32_t>(at % col_tiles) * COLS;
  };

  // Rows of a tile that a wave takes: with at most half of the large tile's
  // rows (an expert's last ones) the waves halve those, and do half the
  // products (512 rows an expert on average: 689 -> 660 us for the gated
  // forward).  There only: in the others the second form of the loops makes
  // the compiler spill (the backward 478 -> 531 us, MXFP4 547 -> 555).
  constexpr bool HALVES = PAIR && C::MI >= 4 && !C::MX;
  const auto wave_rows = [](const StagedTile &u) {
    return HALVES && u.rows <= C::TM / 2 ? C::TM / C::WM / 2 : C::TM / C::WM;
  };

  // This lane's staging sources; each moves on by one stage when it is used.
  const uint8_t *from[C::LOADS], *sfrom[C::SLOADS + 1];
  const uint8_t *zero = reinterpret_cast<const uint8_t *>(g_zero_chunk);
  const int chunk = (lane & 7) ^ ((4 * wave + (lane >> 4)) & 7);
  // kOpBf16T: weight row of the stage and column chunk that this lane stages.
  // Instructions are 4 rows or a multiple apart, so the slot does not depend on j.
  const int wk = wave * C::KROWS + lane / (64 / C::KROWS);
  // ODD: the scale rows of this lane's fragment rows.
  const uint8_t *arows[C::ODD ? C::NI : 1], *brows[C::ODD ? C::MI : 1];
  int32_t limit = p.chunks;  // chunks of the staged tile (0: there is none, and zeros are staged)
  const auto aim = [&](const StagedTile &u, auto token) {
    const int lane = fresh_lane(), lr = lane >> 3, chunk = (lane & 7) ^ ((4 * wave + (lr >> 1)) & 7);
    const int wk = wave * C::KROWS + lane / (64 / C::KROWS);
    // Weight row of tile row r.  With a gate/up pair the first half of each
    // wave's rows are gate columns, the second half the same up columns.
    const auto weight_row = [&](int r) -> int64_t {
      if constexpr (PAIR) {
        constexpr int PER = C::TN / C::WN, HALF = PER / 2;
        const int q = r % PER;
        const int32_t col = min(u.n0 + (r / PER) * HALF + q % HALF, p.width - 1);
        return col + (q >= HALF ? p.width : 0);
      }
      return min(u.n0 + r, p.N - 1);
    };
    const uint8_t *we = p.w + u.e * p.w_expert;
    const int wcol = min(u.n0 + 8 * ((lane % (64 / C::KROWS)) ^ ((wk & 3) << 2)), p.width - 8);
#pragma unroll
    for (int j = 0; j < C::LOADS; ++j) {
      if (j < C::WLOADS && C::TRANS)
        from[j] = we + (wk + j * C::WAVES * C::KROWS) * p.w_row + 2 * wcol;
      else if (j < C::WLOADS)
        from[j] = we + weight_row((j * C::WAVES + wave) * 8 + lr) * p.w_row + 16 * chunk;
      else
        from[j] = p.x + token(((j - C::WLOADS) * C::WAVES + wave) * 8 + lr) * p.x_row + 16 * chunk;
    }
    if constexpr (C::ODD) {
      const int fr = lane & 31;
#pragma unroll
      for (int i = 0; i < C::NI; ++i)
        arows[i] = p.w_scales + (static_cast<int64_t>(u.e) * p.N + weight_row(wn * (C::TN / C::WN) + 32 * i + fr)) * p.chunks;
#pragma unroll
      for (int i = 0; i < C::MI; ++i)
        brows[i] = p.x_scales + token(wm * (C::TM / C::WM) + 32 * i + fr) * p.chunks;
    }
#pragma unroll
    for (int j = 0; j < C::SLOADS; ++j) {
      const int r = (j * C::WAVES + wave) * 32 + (lane >> 1);
      if (j * C::WAVES * 32 < C::TN)
        sfrom[j] = p.w_scales + (static_cast<int64_t>(u.e) * p.N + weight_row(r)) * p.chunks + 4 * (lane & 1);
      else
        sfrom[j] = p.x_scales + token(r - C::TN) * p.chunks + 4 * (lane & 1);
    }
  };

  // Instruction j of stage s (the scales' behind the operands').  Lanes whose
  // chunk lies behind K stage zeros (a scale byte 0 is 2^-127).
  const auto fetch_one = [&](int s, uint8_t *base, auto jc) {
    constexpr int j = decltype(jc)::value;
    if constexpr (j >= C::LOADS) {
      constexpr int k = j - C::LOADS;
      dma_wave(8 * s + 4 * (lane & 1) < limit ? sfrom[k] : zero, base + C::ROWS * 128 + (k * C::WAVES + wave) * 256, 4);
      sfrom[k] += 8;
    } else if constexpr (C::TRANS && j < C::WLOADS) {
      dma_wave(64 * s + wk + j * C::WAVES * C::KROWS < 8 * limit ? from[j] : zero, base + (j * C::WAVES + wave) * 1024, 16);
      from[j] += 64 * p.w_row;
    } else {
      dma_wave(8 * s + chunk < limit ? from[j] : zero, base + (j * C::WAVES + wave) * 1024, 16);
      from[j] += 128;
    }
  };
  // Token ids of a tile's rows into LDS: wave w brings rows 64 w ...
  int32_t *tokens = reinterpret_cast<int32_t *>(lds + C::TOKENS);
  const auto fetch_tokens = [&](const StagedTile &u) {
    if (p.row_token == nullptr || u.e < 0) return;
    dma_wave(p.row_token + u.r0 + min(64 * wave + lane, u.rows - 1), tokens + 64 * wave, 4);
  };

  // Fragment addresses: row (lane % 32) of a 32-row group, chunk 4 half + s.
  const int fr = lane & 31;
  const int arow = wn * (C::TN / C::WN) + fr;
  const auto first_brow = [&](const StagedTile &u) { return C::TN + wm * wave_rows(u) + fr; };
  int brow = first_brow(t);  // of the fragments that are read
  // kOpBf16T: lane 16 g + 4 j + b of a transposing read addresses row j and
  // columns 16 (g % 2) + 4 b .. + 3 of the fragment's 32, in half g / 2.
  int tcol[C::NI];
#pragma unroll
  for (int i = 0; i < C::NI; ++i) {
    const int j = (lane >> 2) & 3;
    const int c = (wn * (C::TN / C::WN) + 32 * i) / 8 + 2 * ((lane >> 4) & 1) + ((lane >> 1) & 1);
    tcol[i] = (32 * half + j) * (2 * C::TN) + 16 * (c ^ (j << 2)) + 8 * (lane & 1);
  }
  struct Frag {
    uint4 a[C::NI], b[C::MI];
  };
  struct Scales {
    uint32_t a[C::NI], b[C::MI];
  };
  constexpr int FRAGS = C::NI + C::MI;
  // Item r of a step's fragment reads, in the order the products need them:
  // a[0], all of b, then the other a; behind them a stage's scales.
  const auto read_item = [&](Frag &f, Scales &sf, const uint8_t *base, int s, auto rc) {
    constexpr int r = decltype(rc)::value;
    if constexpr (r >= FRAGS) {
      constexpr int k = r - FRAGS;
      const uint8_t *sb = base + C::ROWS * 128 + 4 * half;
      if constexpr (k < C::NI)
        sf.a[k] = *reinterpret_cast<const uint32_t *>(sb + (arow + 32 * k) * 8);
      else
        sf.b[k - C::NI] = *reinterpret_cast<const uint32_t *>(sb + (brow + 32 * (k - C::NI)) * 8);
    } else if constexpr (r >= 1 && r <= C::MI) {
      f.b[r - 1] = *reinterpret_cast<const uint4 *>(base + (brow + 32 * (r - 1)) * 128 + 16 * ((4 * half + s) ^ ((fr >> 1) & 7)));
    } else {
      constexpr int i = r == 0 ? 0 : r - C::MI;
      if constexpr (C::TRANS) {
        const uint8_t *src = base + tcol[i] + 8 * s * (2 * C::TN);
        const uint2 lo = read_tr(src), hi = read_tr(src + 4 * (2 * C::TN));
        f.a[i] = make_uint4(lo.x, lo.y, hi.x, hi.y);
      } else {
        f.a[i] = *reinterpret_cast<const uint4 *>(base + (arow + 32 * i) * 128 + 16 * ((4 * half + s) ^ ((fr >> 1) & 7)));
      }
    }
  };

  f32x16 acc[C::NI][C::MI];
  Scales sc;
  // ODD: the scales of a stage as loaded (a dword at any byte; near the end of
  // a row its last four bytes), the shift that brings the stage's first byte
  // down, and whether there is one.  Bytes behind K become 0 (2^-127).
  struct Raw {
    Scales v;
    int shift;
    bool any;
  };
  Raw raw;
  const auto load_scales = [&](int s) {
    const int at = 8 * s + 4 * half, valid = min(limit - at, 4);
    const int off = valid >= 4 ? at : valid > 0 ? limit - 4 : 0;
    raw.any = valid > 0;
    raw.shift = 8 * (4 - max(valid, 1));
#pragma unroll
    for (int i = 0; i < C::NI; ++i) __builtin_memcpy(&raw.v.a[i], arows[C::ODD ? i : 0] + off, 4);
#pragma unroll
    for (int i = 0; i < C::MI; ++i) __builtin_memcpy(&raw.v.b[i], brows[C::ODD ? i : 0] + off, 4);
  };
  const auto take_scales = [&](Scales &to) {
#pragma unroll
    for (int i = 0; i < C::NI; ++i) to.a[i] = raw.any ? raw.v.a[i] >> raw.shift : 0u;
#pragma unroll
    for (int i = 0; i < C::MI; ++i) to.b[i] = raw.any ? raw.v.b[i] >> raw.shift : 0u;
  };
  Frag f0, f1;
  // One step: its products of `f`, with the reads of `g` (step gs of the stage
  // at gbase) and, in a stage's last step, the next stage's scales and the
  // staging of stage ds between them, in exactly this order.  Left to itself
  // the compiler puts the reads last, where the next step waits for them.
  // MA: row groups of 32 that the tile has for each wave.
  const auto step = [&](auto ma, auto sel, const Frag &f, Frag &g, Scales &gsc, const uint8_t *gbase, int gs, int ds,
                        uint8_t *dbase) {
    constexpr int S = decltype(sel)::value, MA = decltype(ma)::value, SLOTS = C::NI * MA;
    constexpr int MR = S == 3 ? C::MI : MA;  // the last step's reads may be for another tile
    constexpr int DF = S == 3 ? 0 : C::LATE, DN = S == 3 ? C::LATE : S == 0 ? C::ALL - C::LATE : 0;
    constexpr int READS = C::NI + MR + (C::SLDS && S == 3 ? FRAGS : 0);
    constexpr int RPS = (READS + SLOTS - 1) / SLOTS, DPS = (DN + SLOTS - 1) / SLOTS;
    each<SLOTS>([&](auto slot) {
      constexpr int n = decltype(slot)::value, i = n / MA, k = n % MA;
      if constexpr (C::MX)
        acc[i][k] = mfma_mx<S>(f.a[i], f.b[k], acc[i][k], sc.a[i], sc.b[k]);
      else
        acc[i][k] = mfma_bf16(f.a[i], f.b[k], acc[i][k]);
      each<RPS>([&](auto q) {
        constexpr int r = n * RPS + decltype(q)::value;
        if constexpr (r < READS)
          read_item(g, gsc, gbase, gs, std::integral_constant<int, (r <= MR ? r : r + C::MI - MR)>{});
      });
      each<DPS>([&](auto q) {
        constexpr int d = n * DPS + decltype(q)::value;
        if constexpr (d < DN) fetch_one(ds, dbase, std::integral_constant<int, DF + d>{});
      });
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  // One stage.  The rest of stage `now`, which the step before began to bring,
  // follows in its first step, and stage `ds` begins in its last; `between` may
  // aim at another tile.
  uint8_t *cur = lds;
  const auto stage = [&](auto ma, int now, int ds, auto between, int next_brow) {
    uint8_t *nxt = lds + (cur == lds ? C::STAGE : 0);
    step(ma, std::integral_constant<int, 0>{}, f0, f1, sc, cur, 1, now, nxt);
    step(ma, std::integral_constant<int, 1>{}, f1, f0, sc, cur, 2, 0, cur);
    between();
    step(ma, std::integral_constant<int, 2>{}, f0, f1, sc, cur, 3, 0, cur);
    wait_lgkm0();  // step 3's fragments are in registers: this wave is done with the stage's LDS
    wait_vm<0>();  // and its part of the next stage has landed
    barrier_no_fence();
    Scales next;
    if constexpr (C::ODD) {  // the next stage's have landed with its operands
      take_scales(next);
      load_scales(ds);
    }
    brow = next_brow;
    step(ma, std::integral_constant<int, 3>{}, f1, f0, next, nxt, 0, ds, cur);
    if constexpr (C::MX) sc = next;
    cur = nxt;
  };

  const int stages = max((p.chunks + 7) / 8, 2);  // at least both buffers: one of zeros for a short K
  aim(t, [&](int r) -> int64_t { return source_row(p, t.r0 + min(r, t.rows - 1)); });
  if constexpr (C::ODD) {
    load_scales(0);
    take_scales(sc);
    load_scales(1);
  }
  each<C::ALL>([&](auto j) { fetch_one(0, lds, j); });
  each<C::LATE>([&](auto j) { fetch_one(1, lds + C::STAGE, j); });
  StagedTile nt;
  advance(nt);
  wait_vm<C::LATE>();
  barrier_no_fence();
  each<FRAGS + (C::SLDS ? FRAGS : 0)>([&](auto r) { read_item(f0, sc, lds, 0, r); });
  fetch_tokens(nt);

#pragma unroll
  for (int i = 0; i < C::NI; ++i)
#pragma unroll
    for (int k = 0; k < C::MI; ++k) acc[i][k] = f32x16{};
  // Names every accumulator as an accumulation register where the loops meet
  // (no instruction): the compiler otherwise carries them in ordinary
  // registers and copies all of them twice a stage.
  const auto pin = [&] {
#pragma unroll
    for (int i = 0; i < C::NI; ++i)
#pragma unroll
      for (int k = 0; k < C::MI; ++k) asm volatile("" : "+a"(acc[i][k]));
  };
  // All stages of a tile.  A stage is one block of code without branches: with
  // one inside, the compiler sinks the products past all the reads.
  const auto contract = [&](auto ma) {
    for (int s = 2; s < stages; ++s) {
      pin();
      stage(ma, s - 1, s, [] {}, brow);
    }
    pin();
    if (stages == 2) {  // no barrier since the tokens were sent for
      wait_vm<0>();
      barrier_no_fence();
    }
    // The last two stages bring the next tile's first two.
    stage(ma, stages - 1, 0, [&] {
      limit = nt.e < 0 ? 0 : p.chunks;
      if (nt.e >= 0)
        aim(nt, [&](int r) -> int64_t {
          const int m = min(r, nt.rows - 1);
          return p.row_token ? tokens[m] : nt.r0 + m;
        });
    }, brow);
    pin();
    stage(ma, 0, 1, [] {}, first_brow(nt));
    pin();
  };
  while (true) {
    if constexpr (HALVES) {
      if (t.rows <= C::TM / 2)
        contract(std::integral_constant<int, C::MI / 2>{});
      else
        contract(std::integral_constant<int, C::MI>{});
    } else {
      contract(std::integral_constant<int, C::MI>{});
    }
    uint8_t *turn = lds + C::TURN + wave * C::TURN_BYTES;
    const int fl = fresh_lane();
    const int32_t wn0 = t.n0 + wn * (C::TN / C::WN) / (PAIR ? 2 : 1);
    const int64_t wrow = static_cast<int64_t>(t.r0) + wm * wave_rows(t);
    const int wrows = min(t.rows - wm * wave_rows(t), wave_rows(t));
    if constexpr (EPI == kEpiGatedBwd) {
      constexpr int TILES = C::RB / 64, ACROSS = C::NI / TILES, BLOCKS = C::MI * ACROSS;
      each<BLOCKS>([&](auto bc) {
        constexpr int b = decltype(bc)::value, k = b / ACROSS, i = b % ACROSS * TILES;
        f32x16 d[TILES];
#pragma unroll
        for (int q = 0; q < TILES; ++q) {
          asm volatile("" : "+a"(acc[i + q][k]));  // not read before its turn
          d[q] = acc[i + q][k];
        }
        if (wrows > 32 * k)
          store_gated_grad<C::RB>(p, d, turn, fl, wrow + 32 * k, wrows - 32 * k, wn0 + 32 * i);
#pragma unroll
        for (int q = 0; q < TILES; ++q) acc[i + q][k] = f32x16{};
        __builtin_amdgcn_sched_barrier(0);
      });
    } else {
#pragma unroll
      for (int k = 0; k < C::MI; ++k) {
        f32x16 col[C::NI];
#pragma unroll
        for (int i = 0; i < C::NI; ++i) {
          asm volatile("" : "+a"(acc[i][k]));  // not read before its turn
          col[i] = acc[i][k];
        }
        store_block<EPI, C::NI, C::RB>(p, col, turn, fl, wrow + 32 * k, wrows - 32 * k, wn0);
#pragma unroll
        for (int i = 0; i < C::NI; ++i) acc[i][k] = f32x16{};
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if (nt.e < 0) break;
    t = nt;
    advance(nt);
    fetch_tokens(nt);
  }
  wait_vm<0>();  // nothing of this workgroup writes LDS after its end
}

template <class C, int EPI>
__global__ __launch_bounds__(C::THREADS, 1) void k_grouped_staged(GroupedParams p, int col_tiles) {
  __shared__ __attribute__((aligned(128))) uint8_t lds[C::LDS];
  staged_tiles<C, EPI>(p, lds, static_cast<uint32_t>(col_tiles));
}

// Workgroups: as many as run at once (PER_CU on each of the 256 CUs), or one
// for each tile if there are fewer.
template <class C, int EPI>
hipError_t launch_staged(const GroupedParams &p, int64_t R, hipStream_t stream) {
  constexpr int COLS = EPI == kEpiSwiglu || EPI == kEpiSwigluMx ? C::TN / 2 : C::TN;
  constexpr int PER_CU = C::LDS <= 81920 ? 2 : 1;
  const int64_t cols = (p.width + COLS - 1) / COLS;
  const int64_t tiles = (max_row_tiles(R, p.E, C::TM) * cols + 7) / 8 * 8;
  if (tiles > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
  const int64_t grid = tiles < 256 * PER_CU ? tiles : 256 * PER_CU;
  hipLaunchKernelGGL((k_grouped_staged<C, EPI>), dim3(static_cast<unsigned>(grid)), dim3(C::THREADS), 0, stream, p,
                     static_cast<int>(cols));
  return hipGetLastError();
}

// The large and the small tile.  256 x 256 reads each operand half as often
// and its waves read LDS least per product (8192 x 8192 x 8192 MXFP4: 282 us
// against 422 us with 128 x 128), but wants rows to fill it, from 128 an
// expert on, and fills the card in coarse rounds of 256 tiles.  Small tiles
// run two a CU, one's stores under the other's products, in rounds of 512
// that take 0.5 to 0.6 of a large one's with short contractions and in the
// backward, 0.6 to 0.75 from 16 stages on.  An expert adds half a row tile.
// Large against small, with the rounds: 4096 x 1536 x 2048 22.0 and 16.1 us (1,
// 1); 32768 x 800 x 992 in 16 groups 48 and 36 (3, 4); 131072 x 1536 x 2048 in
// 64 groups 265 and 306 (13, 25); backward of 32032 x 1408 x 1152 in 16 groups
// 234 and 187 (4, 6), of 65536 x 1456 x 2048 in 32 632 and 684 (7, 13).
template <int EPI>
bool staged_large(const GroupedParams &p, int64_t R) {
  constexpr int PAIRED = EPI == kEpiSwiglu || EPI == kEpiSwigluMx ? 2 : 1;
  const auto rounds = [&](int64_t tile, int64_t places) {
    const int64_t rows = (R + tile * p.E / 2 + tile - 1) / tile, cols = (PAIRED * static_cast<int64_t>(p.width) + tile - 1) / tile;
    return (rows * cols + places - 1) / places;
  };
  const int64_t percent = p.chunks >= 16 * 8 && EPI != kEpiGatedBwd ? 65 : 57;
  return R >= 128 * static_cast<int64_t>(p.E) && 100 * rounds(256, 256) <= percent * rounds(128, 512);
}

template <int OP, int EPI, bool ODD = false>
hipError_t launch_staged_tiles(const GroupedParams &p, int64_t R, hipStream_t stream) {
  if (staged_large<EPI>(p, R))
    return launch_staged<StagedCfg<OP, 256, 256, 2, 2, ODD>, EPI>(p, R, stream);
  return launch_staged<StagedCfg<OP, 128, 128, 2, 2, ODD>, EPI>(p, R, stream);
}

}  // namespace quads
