// LDS-staged products of a batch of fp16 matrices, Y[i, j] = sum_k X[i, k] W[j, k]
// for each, with the epilogues of a Newton-Schulz step.  Either operand may be
// stored with the contraction along its rows (X as [K, M], W as [K, N]).
//
// A stage is 32 of K of TILE rows of X and of W; four stages in LDS, brought by
// DMA three stages before they are read (with the smallest tile two stages, one
// before).  Rows are 64 bytes; row r keeps its chunk c in slot c ^ (r / 4 % 4),
// so that 16 rows of a fragment read take each of the banks once.  (Two stages
// of 64, as in grouped_staged.hpp, are as fast with many matrices and slower
// with few: one 1536 x 2048 361 against 324 us.)
//
// What differs from there besides: fp16; every matrix of the same size; either
// operand by transposing reads; symmetric results, of which only the tiles on
// and below the diagonal are computed and those below it stored twice; and the
// way out.
//
// A step's epilogue moves more of memory's bytes than its stages bring (X comes
// in as hi and lo and leaves as both), so it takes no turn through LDS: X's
// rows are MFMA's first operand and W's the second, so a lane holds one column
// of 16 rows, and the columns are dealt to lanes and fragments so that a
// lane's V fragments of a row are V neighbours (V = 4 with the large tile).  A
// wave's access is then two rows of 256 bytes, 8 a lane.  Where W's rows are
// staged, that is a permutation of the rows that the DMA fetches; where its
// columns are, the transposing reads give a quad of lanes 4 neighbouring
// columns of every fragment, and a 4 x 4 transpose inside the quad follows.
// X's rows are dealt so that a lane's 16 are neighbours too: 32 bytes of a row
// of the transposed tile.
//
// Bound: the loop by the staging and by the card's power limit, then the
// epilogue's bytes.  128 products of 1024 x 1024 x 2048, tiles on and below the
// diagonal, on random data 376 us; without the epilogue 341, of that without
// the matrix instructions 215, without the DMA 254; on zeros, which spare the
// power limit, 284, 250, 212 and 174.  Three or five buffers, workgroups that
// start staggered, no wait for the stores in a tile's first three stages, and
// batches that fit the last-level cache gained nothing.
#pragma once

#include "grouped_staged.hpp"

namespace quads {

// Global-memory-to-LDS DMA from a uniform address and the lane's offset: 16
// bytes a lane, to consecutive LDS addresses.
__device__ __forceinline__ void dma_uniform(uint32_t offset, const uint8_t *base, uint32_t lds) {
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(offset), "s"(base), "s"(lds)
               : "memory", "m0");
#pragma clang diagnostic pop
}

// LDS reads at an address of their own address space.
__device__ __forceinline__ uint4 read_lds16(uint32_t at) {
  typedef __attribute__((address_space(3))) const u32x4 lds_u32x4;
  const u32x4 v = *reinterpret_cast<lds_u32x4 *>(static_cast<uintptr_t>(at));
  return make_uint4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void write_lds16(uint32_t at, const float (&v)[4]) {
  typedef float f32x4 __attribute__((ext_vector_type(4)));
  typedef __attribute__((address_space(3))) f32x4 lds_f32x4;
  *reinterpret_cast<lds_f32x4 *>(static_cast<uintptr_t>(at)) = f32x4{v[0], v[1], v[2], v[3]};
}
__device__ __forceinline__ uint2 read_tr_at(uint32_t at) {
  typedef short s16x4 __attribute__((ext_vector_type(4)));
  typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
  const s16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(static_cast<uintptr_t>(at)));
  return __builtin_bit_cast(uint2, v);
}

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ f32x16 mfma_f16(uint4 a, uint4 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(h8, a), __builtin_bit_cast(h8, b), c, 0, 0, 0);
}

// Two floats -> packed fp16, nearest-even.
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const f16x2 p = {static_cast<_Float16>(lo), static_cast<_Float16>(hi)};
  return __builtin_bit_cast(uint32_t, p);
}

// lo = v less its fp16 rounding (exact in fp32).
template <int N>
__device__ __forceinline__ void split_f16(const float (&v)[N], float (&lo)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) lo[i] = v[i] - static_cast<float>(static_cast<_Float16>(v[i]));
}

// fp16(a - x.lo), fp16(b - x.hi): the differences are exact in fp32.
__device__ __forceinline__ uint32_t residual_f16(uint32_t x, float a, float b) {
  uint32_t d;
  asm("v_fma_mixlo_f16 %0, %1, -1.0, %2 op_sel_hi:[1,0,0]" : "=v"(d) : "v"(x), "v"(a));
  asm("v_fma_mixhi_f16 %0, %1, -1.0, %2 op_sel:[1,0,0] op_sel_hi:[1,0,0]" : "+v"(d) : "v"(x), "v"(b));
  return d;
}

enum BatchedEpi {
  kEpiGram = 0,  // out = alpha Y, symmetric
  kEpiPoly = 1,  // out = beta in + alpha Y, symmetric
  kEpiNext = 2,   // v = beta (in + in2) + Y; out = fp16(v), out2 = fp16(v - out)
  kEpiRound = 3,  // v = beta (in + in2) + Y; out = fp16(v)
  kEpiLast = 4,   // out = bf16(alpha (beta in + Y))
  kEpiOnly = 5    // out = bf16(alpha (beta (in + in2) + Y))
};

struct BatchedParams {
  const uint8_t *x, *w;
  int64_t x_row, w_row, x_mat, w_mat;  // strides in bytes of stored rows and of matrices
  int32_t batch, M, N;                 // multiples of 16
  int32_t K;                           // a multiple of 32, at least 128
  int64_t in_row, in_mat, out_row, out_mat;  // strides in bytes of the arrays below
  const uint16_t *in, *in2;            // [batch, M, N]; in2 may be out2, or null
  uint16_t *out, *out2;                // [batch, M, N]; out2 may be null
  float alpha, beta;
};

// A tile's K is contracted by SPLIT groups of waves, each a part of it.
// TILE 256 and 128: one group of 2 x 2 waves with a quarter of the tile each.
// TILE 64: four groups of one wave, for the whole tile; their sums meet in LDS,
// and each takes a quarter of the rows out.
template <int TILE_, bool XT_, bool WT_>
struct BatchedCfg {
  static constexpr int TILE = TILE_, SPLIT = TILE == 64 ? 4 : 1, WAVES = 4 / SPLIT, SIDE = WAVES == 4 ? 2 : 1;
  static constexpr int HALF = TILE / SIDE;             // a wave's part, each way
  static constexpr bool XT = XT_, WT = WT_;
  static constexpr int MI = HALF / 32;                 // 32 x 32 tiles of a wave, each way
  static constexpr int BUFFERS = TILE == 64 ? 2 : 4;   // (two workgroups of the smallest tile a CU)
  static constexpr int STAGE = 2 * TILE * 64;          // 32 of K: 64 bytes of a row
  static constexpr int LOADS = STAGE / 1024 / WAVES;   // staging instructions of a wave and stage, both operands
  static constexpr int KROWS = 512 / TILE;             // transposed operand: stored rows of an instruction
  static constexpr int RING = BUFFERS * STAGE, LDS = SPLIT * RING;
  static constexpr int ROWS = SPLIT == 1 ? MI : 1;     // row fragments that a wave takes out, and
  static constexpr int REGS = SPLIT == 1 ? 16 : 8;     // registers of each
  // Position p of 32 (a lane of a fragment, or a row of the accumulators) and
  // fragment t of a wave's half tile -> column or row inside the half.
  // W by rows: lane p of fragment t has column MI p + t.  W by columns: in
  // units of 4 columns, unit p / 4 of fragment t is 2 MI (p / 8) + 2 t + p / 4 % 2
  // (two units lie in one 16-byte chunk).  X: position 8 q + 4 h + r (lanes of
  // half h, register 4 q + r) is row 16 h + 4 q + r.
  static __device__ __forceinline__ int w_row(int p, int t) { return MI * p + t; }
  static __device__ __forceinline__ int w_unit(int p4, int t) { return 2 * MI * (p4 >> 1) + 2 * t + (p4 & 1); }
  static __device__ __forceinline__ int x_unit(int p4) { return 4 * (p4 & 1) + (p4 >> 1); }
  // Slot of a chunk of a transposed stage is chunk ^ slot(k): the four rows k
  // that a group of 16 lanes reads lie in different banks than its units.
  // (Rows of the smallest tile are 128 bytes: two of them have banks of their own.)
  static __device__ __forceinline__ int w_slot(int k) {
    return TILE == 256 ? k & 3 : TILE == 128 ? (k & 1) | ((k & 2) << 2) : (k >> 1) & 1;
  }
  static __device__ __forceinline__ int x_slot(int k) { return TILE == 64 ? (k & 2) << 1 : (k & 3) << 2; }
};

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// V neighbouring fp16 (or bf16) values of a row, in V / 2 dwords.
template <int V>
struct Neighbours {
  uint32_t w[V / 2];
};
template <int V>
__device__ __forceinline__ Neighbours<V> load_neighbours(const uint8_t *p) {
  Neighbours<V> n;
  if constexpr (V == 4) {
    const u32x2 v = *reinterpret_cast<const u32x2 *>(p);
    n.w[0] = v[0];
    n.w[1] = v[1];
  } else {
    n.w[0] = *reinterpret_cast<const uint32_t *>(p);
  }
  return n;
}
template <int V>
__device__ __forceinline__ void store_neighbours(uint8_t *p, const Neighbours<V> &n) {
  if constexpr (V == 4) *reinterpret_cast<u32x2 *>(p) = u32x2{n.w[0], n.w[1]};
  else *reinterpret_cast<uint32_t *>(p) = n.w[0];
}

template <int CTRL>
__device__ __forceinline__ float quad_move(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xf, 0xf, true));
}

// v[t] of lane c of a quad -> V neighbours: column 4 t + c becomes lane c's
// column V c + e (V = 4: the 4 x 4 transpose; V = 2: lane c takes two of
// fragment c / 2).
template <int V>
__device__ __forceinline__ void quad_transpose(float (&v)[V], int lane) {
  if constexpr (V == 4) {
    const bool odd = lane & 1, high = lane & 2;
    float w[4];
#pragma unroll
    for (int t = 0; t < 4; t += 2) {
      const float a = quad_move<0xB1>(v[t]), b = quad_move<0xB1>(v[t + 1]);  // lane ^ 1
      w[t] = odd ? b : v[t];
      w[t + 1] = odd ? v[t + 1] : a;
    }
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const float a = quad_move<0x4E>(w[t]), b = quad_move<0x4E>(w[t + 2]);  // lane ^ 2
      v[t] = high ? b : w[t];
      v[t + 2] = high ? w[t + 2] : a;
    }
  } else {
    const bool high = lane & 2;
    const float a0 = quad_move<0x88>(v[0]), a1 = quad_move<0xDD>(v[0]);  // lanes 0 2 0 2, 1 3 1 3
    const float b0 = quad_move<0x88>(v[1]), b1 = quad_move<0xDD>(v[1]);
    v[0] = high ? b0 : a0;
    v[1] = high ? b1 : a1;
  }
}

struct BatchedTile {
  int32_t e, m0, n0;  // matrix (-1: no tile), first row and column
};

template <class C, int EPI>
__device__ __forceinline__ void batched_tiles(const BatchedParams &p, uint8_t *lds, uint32_t per_matrix, uint32_t col_tiles) {
  constexpr bool SYM = EPI == kEpiGram || EPI == kEpiPoly;
  constexpr bool LOW = EPI == kEpiNext || EPI == kEpiRound || EPI == kEpiOnly;  // in2 is read
  const int lane = threadIdx.x & 63, all_waves = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), half = lane >> 5;
  const int wave = all_waves % C::WAVES, group = all_waves / C::WAVES;
  const int wn = wave / C::SIDE, wm = wave % C::SIDE;

  // The tiles of this workgroup: at, at + step, ... below end, out of its XCD's eighth.
  const uint32_t tiles = static_cast<uint32_t>(p.batch) * per_matrix, per = (tiles + 7) / 8;
  const uint32_t step_tiles = gridDim.x / 8, end = min(tiles, ((blockIdx.x & 7) + 1) * per);
  uint32_t at = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
  if (at >= end) return;
  const auto tile_at = [&](uint32_t index) -> BatchedTile {
    if (index >= end) return BatchedTile{-1, 0, 0};
    const uint32_t e = index / per_matrix;
    uint32_t r = index % per_matrix, i = 0;
    if constexpr (SYM) {  // tile r of the rows i = 0, 1, ... of i + 1 tiles
      while (r > i) r -= ++i;
    } else {
      i = r / col_tiles;
      r %= col_tiles;
    }
    return BatchedTile{static_cast<int32_t>(e), static_cast<int32_t>(i) * C::TILE, static_cast<int32_t>(r) * C::TILE};
  };
  BatchedTile t = tile_at(at), nt{-1, 0, 0};
  const auto advance = [&] {
    at += step_tiles;
    nt = tile_at(at);
  };

  // Staging: instruction j < LOADS / 2 brings W, the others X.  A lane's source
  // is a uniform address, which moves on from stage to stage in scalar
  // registers, and an offset that it keeps for the tile: nothing for the vector
  // unit between the products (64-bit addresses and a selected source behind K
  // instead: 128 experts' gate and up 14.3 ms, so 13.9; down 7.2 and 6.8).
  // Behind the matrix rows and columns repeat the last one.
  constexpr int WL = C::LOADS / 2;
  uint32_t from[C::LOADS];
  const uint8_t *wbase, *xbase;
  // The group's stages, at least BUFFERS, and those of the groups before it.
  const int all_stages = p.K / 32, before = group * all_stages / C::SPLIT;
  const int stages = (group + 1) * all_stages / C::SPLIT - before;
  const int64_t wstep = C::WT ? 32 * p.w_row : 64, xstep = C::XT ? 32 * p.x_row : 64;
  const auto aim = [&](const BatchedTile &u) {
    const int lane = fresh_lane(), lr = lane >> 2, chunk = (lane & 3) ^ ((lane >> 4) & 3);
    const int wk = wave * C::KROWS + lane / (64 / C::KROWS);
    const int slot = lane % (64 / C::KROWS);
    wbase = p.w + u.e * p.w_mat + (C::WT ? 2 * static_cast<int64_t>(u.n0) : u.n0 * p.w_row) + before * wstep;
    xbase = p.x + u.e * p.x_mat + (C::XT ? 2 * static_cast<int64_t>(u.m0) : u.m0 * p.x_row) + before * xstep;
#pragma unroll
    for (int j = 0; j < C::LOADS; ++j) {
      const bool weight = j < WL;
      const uint32_t stride = static_cast<uint32_t>(weight ? p.w_row : p.x_row);
      const int32_t left = weight ? p.N - u.n0 : p.M - u.m0;
      const int jj = weight ? j : j - WL;
      if (weight ? C::WT : C::XT) {
        const int column = 8 * (slot ^ (weight ? C::w_slot(wk) : C::x_slot(wk)));
        from[j] = (wk + jj * C::WAVES * C::KROWS) * stride + 2 * min(column, left - 8);
      } else {
        const int r = (jj * C::WAVES + wave) * 16 + lr, part = r & ~(C::HALF - 1), t = r % C::HALF / 32, q = r & 31;
        const int row = part + (weight ? C::w_row(q, t) : 32 * t + 4 * C::x_unit(q >> 2) + (q & 3));
        from[j] = min(row, left - 1) * stride + 16 * chunk;
      }
    }
  };
  const uint32_t lds0 = lds_address(lds) + group * C::RING;
  // Instruction j of the stage that wbase and xbase point at, into the buffer at `to`.
  const auto fetch_one = [&](uint32_t to, auto jc) {
    constexpr int j = decltype(jc)::value, jj = j < WL ? j : j - WL;
    dma_uniform(from[j], j < WL ? wbase : xbase, to + (j < WL ? 0 : C::TILE * 64) + (jj * C::WAVES + wave) * 1024);
    if constexpr (j == WL - 1) wbase += wstep;
    if constexpr (j == C::LOADS - 1) xbase += xstep;
  };

  // This lane's fragment addresses inside a stage, by step.
  const int fr = lane & 31;
  // Lane 16 g + 4 j + b of a transposing read addresses row j and unit 4 (g % 2) + b
  // of the fragment's 8, in half g / 2.
  uint32_t wat[C::WT ? C::MI : 2], xat[C::XT ? C::MI : 2];
  {
    const int j = (lane >> 2) & 3, unit = 4 * ((lane >> 4) & 1) + (lane & 3);
#pragma unroll
    for (int i = 0; i < (C::WT ? C::MI : 2); ++i) {
      const int wu = wn * (C::HALF / 4) + C::w_unit(unit, i);
      wat[i] = C::WT ? (8 * half + j) * (2 * C::TILE) + 16 * ((wu >> 1) ^ C::w_slot(j)) + 8 * (wu & 1)
                     : (wn * C::HALF + fr) * 64 + 16 * ((2 * i + half) ^ ((fr >> 2) & 3));
    }
#pragma unroll
    for (int i = 0; i < (C::XT ? C::MI : 2); ++i) {
      const int xu = wm * (C::HALF / 4) + 8 * i + C::x_unit(unit);
      xat[i] = C::TILE * 64 + (C::XT ? (8 * half + j) * (2 * C::TILE) + 16 * ((xu >> 1) ^ C::x_slot(j)) + 8 * (xu & 1)
                                     : (wm * C::HALF + fr) * 64 + 16 * ((2 * i + half) ^ ((fr >> 2) & 3)));
    }
  }
  struct Frag {
    uint4 a[C::MI], b[C::MI];
  };
  // Item r of the fragment reads of step S of the stage at `base`, in the order
  // the products need them: a[0], all of b, then the other a.
  const auto read_item = [&](Frag &f, uint32_t base, auto sc, auto rc) {
    constexpr int S = decltype(sc)::value, r = decltype(rc)::value;
    constexpr bool x = r >= 1 && r <= C::MI;
    constexpr int i = x ? r - 1 : r == 0 ? 0 : r - C::MI;
    uint4 v;
    if constexpr (x ? C::XT : C::WT) {
      const uint32_t src = base + (x ? xat[C::XT ? i : 0] : wat[C::WT ? i : 0]) + 16 * S * (2 * C::TILE);
      const uint2 lo = read_tr_at(src), hi = read_tr_at(src + 4 * (2 * C::TILE));
      v = make_uint4(lo.x, lo.y, hi.x, hi.y);
    } else {
      v = read_lds16(base + (x ? xat[C::XT ? 0 : S] : wat[C::WT ? 0 : S]) + 2048 * i);
    }
    if constexpr (x) f.b[i] = v;
    else f.a[i] = v;
  };

  f32x16 acc[C::MI][C::MI];  // [columns][rows]
  Frag f0, f1;
  // One step of 16 of K: the products of `f` with the reads of `g` (step GS of
  // the stage at gbase) and, in a stage's second, the staging of another into
  // its own buffer between them, in exactly this order.
  const auto step = [&](auto gs, auto fetch, const Frag &f, Frag &g, uint32_t gbase, uint32_t to) {
    constexpr int GS = decltype(gs)::value, SLOTS = C::MI * C::MI, DN = GS == 0 && decltype(fetch)::value ? C::LOADS : 0;
    constexpr int READS = 2 * C::MI, RPS = (READS + SLOTS - 1) / SLOTS, DPS = (DN + SLOTS - 1) / SLOTS;
    each<SLOTS>([&](auto slot) {
      constexpr int n = decltype(slot)::value, i = n / C::MI, k = n % C::MI;
      acc[i][k] = mfma_f16(f.b[k], f.a[i], acc[i][k]);
      each<RPS>([&](auto q) {
        constexpr int r = n * RPS + decltype(q)::value;
        if constexpr (r < READS) read_item(g, gbase, gs, std::integral_constant<int, r>{});
      });
      each<DPS>([&](auto q) {  // the later slots: the earlier ones have the reads
        constexpr int d = n * DPS + decltype(q)::value - (SLOTS * DPS - DN);
        if constexpr (d >= 0) fetch_one(to, std::integral_constant<int, d>{});
      });
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  // One stage.  Its second step's fragments are in registers after the first,
  // so behind one barrier its buffer is free for the stage four further on, and
  // the next stage has landed.
  uint32_t cur = lds0;  // the stage's buffer
  const auto stage = [&](auto fetch) {
    constexpr bool FETCH = decltype(fetch)::value;
    const uint32_t nxt = cur == lds0 + (C::BUFFERS - 1) * C::STAGE ? lds0 : cur + C::STAGE;
    step(std::integral_constant<int, 1>{}, fetch, f0, f1, cur, cur);
    wait_lgkm0();
    wait_vm<FETCH ? (C::BUFFERS - 2) * C::LOADS : 0>();  // all but the youngest stages have landed
    if constexpr (C::WAVES > 1) barrier_no_fence();
    step(std::integral_constant<int, 0>{}, fetch, f1, f0, nxt, cur);
    cur = nxt;
  };

  aim(t);
  each<C::BUFFERS>([&](auto b) {
    each<C::LOADS>([&](auto j) { fetch_one(lds0 + decltype(b)::value * C::STAGE, j); });
  });
  if constexpr (C::SPLIT == 1) advance();
  wait_vm<(C::BUFFERS - 1) * C::LOADS>();
  if constexpr (C::WAVES > 1) barrier_no_fence();
  each<2 * C::MI>([&](auto r) { read_item(f0, lds0, std::integral_constant<int, 0>{}, r); });
#pragma unroll
  for (int i = 0; i < C::MI; ++i)
#pragma unroll
    for (int k = 0; k < C::MI; ++k) acc[i][k] = f32x16{};
  const auto pin = [&] {  // accumulators stay accumulation registers where the loops meet
#pragma unroll
    for (int i = 0; i < C::MI; ++i)
#pragma unroll
      for (int k = 0; k < C::MI; ++k) asm volatile("" : "+a"(acc[i][k]));
  };

  while (true) {
    for (int s = C::BUFFERS; s < stages; ++s) {
      pin();
      stage(std::true_type{});
    }
    if constexpr (C::SPLIT == 1) {
      // The last stages bring the next tile's first (there being none, this one's again).
      aim(nt.e >= 0 ? nt : t);
      for (int s = 0; s < C::BUFFERS; ++s) {
        pin();
        stage(std::true_type{});
      }
    } else {  // one tile a workgroup
      for (int s = 0; s < C::BUFFERS; ++s) {
        pin();
        stage(std::false_type{});
      }
      // The waves' sums, a fragment at a time; wave g takes registers 8 (g % 2) ..
      // of row fragment g / 2, from all waves in their order.
      wait_lgkm0();
      barrier_no_fence();  // every wave is done with the stages
      const uint32_t exchange = lds_address(lds) + 16 * lane;
#pragma unroll
      for (int i = 0; i < C::MI; ++i)
#pragma unroll
        for (int k = 0; k < C::MI; ++k)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float v[4] = {acc[i][k][4 * q], acc[i][k][4 * q + 1], acc[i][k][4 * q + 2], acc[i][k][4 * q + 3]};
            write_lds16(exchange + 16384 * group + 1024 * ((i * C::MI + k) * 4 + q), v);
          }
      wait_lgkm0();
      barrier_no_fence();
#pragma unroll
      for (int i = 0; i < C::MI; ++i)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          float sum[4] = {};
#pragma unroll
          for (int g = 0; g < C::SPLIT; ++g) {
            const uint4 v = read_lds16(exchange + 16384 * g + 1024 * ((i * C::MI + (group >> 1)) * 4 + 2 * (group & 1) + q));
            sum[0] += __uint_as_float(v.x);
            sum[1] += __uint_as_float(v.y);
            sum[2] += __uint_as_float(v.z);
            sum[3] += __uint_as_float(v.w);
          }
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[i][0][4 * q + r] = sum[r];
        }
    }
    pin();

    // ---- the tile's results, 4 registers' rows of all fragments at a time
    constexpr int V = C::MI, PER = C::REGS / 4, GROUPS = PER * C::ROWS;  // group g: row fragment g / PER, registers 4 (g % PER) ..
    constexpr int AHEAD = GROUPS > 3 ? 3 : GROUPS - 1;
    const int fl = fresh_lane(), fh = fl >> 5, fp = fl & 31;
    const int32_t wm0 = t.m0 + wm * C::HALF + 32 * (group >> 1), wn0 = t.n0 + wn * C::HALF;
    // The lane's V columns.
    const int32_t col = wn0 + (!C::WT ? V * fp
                               : V == 4 ? 4 * C::w_unit(fp >> 2, fp & 3)
                                        : 4 * C::w_unit(fp >> 2, (fp >> 1) & 1) + 2 * (fp & 1));
    const bool col_ok = col < p.N;
    const uint32_t at_col = 2 * static_cast<uint32_t>(col_ok ? col : 0);
    // Addresses are a uniform row (in scalar registers) and the lane's offset
    // from it: its columns, and 16 rows with half 1.  A row fragment's halves
    // lie inside the matrix or behind it (sizes are multiples of 16); lanes
    // behind it read other rows, and store nothing.  No branch around loads:
    // where paths with different numbers of loads meet, the compiler can only
    // wait for all of them, also for those sent ahead.
    const auto rows_left = [&](int k) { return p.M - (wm0 + 32 * k); };
    const auto offset = [&](int k, int64_t row) {
      return at_col + (fh != 0 && rows_left(k) > 16 ? 16 * static_cast<uint32_t>(row) : 0u);
    };
    // Byte of a group's first row.  Made where the compiler does not see it
    // before: it would compute all groups' at once and has no registers for them.
    const auto group_at = [&](int g, int64_t row_bytes, int64_t mat_bytes) -> int64_t {
      int32_t row = min(wm0 + 32 * (g / PER), p.M - 16) + C::REGS * (group & 1) + 4 * (g % PER);
      asm volatile("" : "+s"(row));
      return t.e * mat_bytes + row * row_bytes;
    };
    struct Group {
      Neighbours<V> in[4], in2[4];
    };
    Group ring[AHEAD + 1];
    const auto load_group = [&](Group &u, int g) {
      if constexpr (EPI != kEpiGram) {
        const uint32_t lane_at = offset(g / PER, p.in_row);
        const int64_t at = group_at(g, p.in_row, p.in_mat);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          u.in[r] = load_neighbours<V>(reinterpret_cast<const uint8_t *>(p.in) + (at + r * p.in_row) + lane_at);
          if constexpr (LOW)
            u.in2[r] = load_neighbours<V>(reinterpret_cast<const uint8_t *>(p.in2) + (at + r * p.in_row) + lane_at);
        }
      }
    };
    each<AHEAD>([&](auto gc) { load_group(ring[decltype(gc)::value], decltype(gc)::value); });
    const bool mirror = SYM && t.m0 != t.n0;
    each<GROUPS>([&](auto gc) {
      constexpr int g = decltype(gc)::value, k = g / PER, r0 = 4 * (g % PER);
      if constexpr (g + AHEAD < GROUPS) load_group(ring[(g + AHEAD) % (AHEAD + 1)], g + AHEAD);
      __builtin_amdgcn_sched_barrier(0);
      {
        const Group &u = ring[g % (AHEAD + 1)];
        Neighbours<V> out[4], out2[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          float v[V];
#pragma unroll
          for (int i = 0; i < V; ++i) {
            v[i] = acc[i][k][r0 + r];
            if constexpr (SYM) v[i] *= p.alpha;
          }
          if constexpr (C::WT) quad_transpose<V>(v, fl);
#pragma unroll
          for (int i = 0; i < V; i += 2) {
            if constexpr (EPI != kEpiGram) {
              const f16x2 x = __builtin_bit_cast(f16x2, u.in[r].w[i / 2]);
              v[i] = __builtin_fmaf(static_cast<float>(x[0]), p.beta, v[i]);
              v[i + 1] = __builtin_fmaf(static_cast<float>(x[1]), p.beta, v[i + 1]);
            }
            if constexpr (LOW) {
              const f16x2 x = __builtin_bit_cast(f16x2, u.in2[r].w[i / 2]);
              v[i] = __builtin_fmaf(static_cast<float>(x[0]), p.beta, v[i]);
              v[i + 1] = __builtin_fmaf(static_cast<float>(x[1]), p.beta, v[i + 1]);
            }
            if constexpr (EPI == kEpiLast || EPI == kEpiOnly) {
              out[r].w[i / 2] = pack_bf16(p.alpha * v[i], p.alpha * v[i + 1]);
            } else {
              const f16x2 x = {static_cast<_Float16>(v[i]), static_cast<_Float16>(v[i + 1])};
              out[r].w[i / 2] = __builtin_bit_cast(uint32_t, x);
              if constexpr (EPI == kEpiNext) out2[r].w[i / 2] = residual_f16(out[r].w[i / 2], v[i], v[i + 1]);
            }
          }
          if constexpr (EPI == kEpiPoly) {  // for the transposed tile
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i][k][r0 + r] = v[i];
          }
        }
        const uint32_t lane_at = offset(k, p.out_row);
        if (col_ok && rows_left(k) > 16 * fh) {
          const int64_t at = group_at(g, p.out_row, p.out_mat);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            store_neighbours<V>(reinterpret_cast<uint8_t *>(p.out) + (at + r * p.out_row) + lane_at, out[r]);
            if constexpr (EPI == kEpiNext)
              store_neighbours<V>(reinterpret_cast<uint8_t *>(p.out2) + (at + r * p.out_row) + lane_at, out2[r]);
          }
        }
      }
      if constexpr (SYM && g % PER == PER - 1) {
        if (mirror) {
          const int32_t at_row = wm0 + 32 * k + 16 * fh + C::REGS * (group & 1);
#pragma unroll
          for (int i = 0; i < V; ++i) {  // a lane's rows of column i are neighbours in a row
            const int32_t row = wn0 + (C::WT ? 4 * C::w_unit(fp >> 2, i) + (fp & 3) : C::w_row(fp, i));
            if (row < p.N && at_row < p.M) {
              uint8_t *to = reinterpret_cast<uint8_t *>(p.out) + t.e * p.out_mat + row * p.out_row + 2 * at_row;
              const float scale = EPI == kEpiGram ? p.alpha : 1.0f;
#pragma unroll
              for (int r = 0; r < C::REGS; r += 8) {
                uint32_t w[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) w[q] = pack_f16(scale * acc[i][k][r + 2 * q], scale * acc[i][k][r + 2 * q + 1]);
                *reinterpret_cast<uint4 *>(to + 2 * r) = make_uint4(w[0], w[1], w[2], w[3]);
              }
            }
          }
        }
      }
      if constexpr (g % PER == PER - 1) {
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i][k] = f32x16{};
      }
      __builtin_amdgcn_sched_barrier(0);
    });
    if (C::SPLIT > 1 || nt.e < 0) break;
    t = nt;
    advance();
  }
  wait_vm<0>();  // nothing of this workgroup writes LDS after its end
}

template <class C, int EPI>
__global__ __launch_bounds__(256, 1) void k_batched(BatchedParams p, uint32_t per_matrix, uint32_t col_tiles) {
  __shared__ __attribute__((aligned(128))) uint8_t lds[C::LDS];
  batched_tiles<C, EPI>(p, lds, per_matrix, col_tiles);
}

template <class C, int EPI>
hipError_t launch_batched_tiles(const BatchedParams &p, hipStream_t stream) {
  constexpr bool SYM = EPI == kEpiGram || EPI == kEpiPoly;
  constexpr int PER_CU = C::LDS <= 81920 ? 2 : 1;
  const int64_t r = (p.M + C::TILE - 1) / C::TILE, c = (p.N + C::TILE - 1) / C::TILE;
  const int64_t per_matrix = SYM ? r * (r + 1) / 2 : r * c;
  const int64_t tiles = (p.batch * per_matrix + 7) / 8 * 8;
  if (tiles > 0x3FFFFFFF) return hipErrorInvalidConfiguration;
  const int64_t grid = C::SPLIT > 1 ? tiles : std::min<int64_t>(tiles, 256 * PER_CU);  // with SPLIT one tile a workgroup
  hipLaunchKernelGGL((k_batched<C, EPI>), dim3(static_cast<unsigned>(grid)), dim3(256), 0, stream, p,
                     static_cast<uint32_t>(per_matrix), static_cast<uint32_t>(c));
  return hipGetLastError();
}

// The large tile reads each operand half as often; smaller ones, two a CU, fill
// the card with few matrices: a round of the large one over the card has to cost
// no more than 0.6 of the smaller's rounds (five steps, every product by 128 and
// by 256: 4 of 2048 x 2048 1090 and 892 us, 16 of 1024 x 2048 1095 and 1000, 64
// of 512 x 1024 744 and 746; but 2 of 2048 x 2048 595 and 725, 4 of 1024 x 2048
// 326 and 547, 64 of 528 x 784 755 and 902; 8 of 1024 x 2048 573 and 632, 530 with
// each product by the rule; 128 of 528 x 784 1737 and 1673, which it misses).
// The smallest where all of them run at once: one matrix of 1024 x 1024 in five
// steps 198 -> 140 us, of 512 x 512 138 -> 98, 8 of 512 x 512 144 -> 128; beyond,
// one of 2048 x 2048 takes 375 us with 128 x 128 and 653 with it.
template <bool XT, bool WT, int EPI>
hipError_t launch_batched(const BatchedParams &p, hipStream_t stream) {
  constexpr bool SYM = EPI == kEpiGram || EPI == kEpiPoly;
  const auto tiles = [&](int64_t tile) {
    const int64_t r = (p.M + tile - 1) / tile, c = (p.N + tile - 1) / tile;
    return p.batch * (SYM ? r * (r + 1) / 2 : r * c);
  };
  if (100 * ((tiles(256) + 255) / 256) <= 60 * ((tiles(128) + 511) / 512))
    return launch_batched_tiles<BatchedCfg<256, XT, WT>, EPI>(p, stream);
  if (tiles(64) <= 512 && p.K >= 256) return launch_batched_tiles<BatchedCfg<64, XT, WT>, EPI>(p, stream);
  return launch_batched_tiles<BatchedCfg<128, XT, WT>, EPI>(p, stream);
}

}  // namespace quads
