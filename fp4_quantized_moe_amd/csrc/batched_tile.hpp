// LDS-staged products of a batch of fp16 matrices, Y[i, j] = sum_k X[i, k] W[j, k]
// for each, with the epilogues of a Newton-Schulz step.  Either operand may be
// stored with the contraction along its rows (X as [K, M], W as [K, N]).
//
// A stage is 32 of K of TILE rows of X and of W; four stages in LDS, brought by
// DMA three stages before they are read.  Rows are 64 bytes; row r keeps its
// chunk c in slot c ^ (r / 4 % 4), so that 16 rows of a fragment read take each
// of the banks once.  (Two stages of 64, as in grouped_staged.hpp, are as fast
// with many matrices and slower with few: one 1536 x 2048 361 against 324 us.)
//
// What differs from there besides: fp16; every matrix of the same size; either
// operand by transposing reads; symmetric results, of which only the tiles on
// and below the diagonal are computed and those below it stored twice; and the
// way out.
//
// A step's epilogue reads and writes more bytes than its stages bring (X comes
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
#pragma once

#include "grouped_staged.hpp"

namespace quads {

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
  kEpiNext = 2,  // v = beta (in + in2) + Y; out = fp16(v), out2 = fp16(v - out)
  kEpiLast = 3   // out = bf16(alpha (beta (in + in2) + Y))
};

struct BatchedParams {
  const uint8_t *x, *w;
  int64_t x_row, w_row, x_mat, w_mat;  // strides in bytes of stored rows and of matrices
  int32_t batch, M, N;                 // multiples of 16
  int32_t chunks;                      // K / 8
  const uint16_t *in, *in2;            // [batch, M, N]; in2 may be out2
  uint16_t *out, *out2;                // [batch, M, N]
  float alpha, beta;
};

template <int TILE_, bool XT_, bool WT_>
struct BatchedCfg {
  static constexpr int TILE = TILE_, HALF = TILE / 2;  // 2 x 2 waves
  static constexpr bool XT = XT_, WT = WT_;
  static constexpr int MI = HALF / 32;                 // 32 x 32 tiles of a wave, each way
  static constexpr int BUFFERS = 4;
  static constexpr int STAGE = 2 * TILE * 64;          // 32 of K: 64 bytes of a row
  static constexpr int LOADS = TILE / 32;              // staging instructions of a wave and stage, both operands
  static constexpr int KROWS = 512 / TILE;             // transposed operand: stored rows of an instruction
  static constexpr int LDS = BUFFERS * STAGE;
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
  static __device__ __forceinline__ int w_slot(int k) { return MI == 4 ? k & 3 : (k & 1) | ((k & 2) << 2); }
  static __device__ __forceinline__ int x_slot(int k) { return (k & 3) << 2; }
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
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), half = lane >> 5;
  const int wn = wave / 2, wm = wave % 2;

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
  BatchedTile t = tile_at(at), nt;
  const auto advance = [&] {
    at += step_tiles;
    nt = tile_at(at);
  };

  // Staging: instruction j < LOADS / 2 brings weights, the others rows of X.
  constexpr int WL = C::LOADS / 2;
  const uint8_t *from[C::LOADS];
  const uint8_t *zero = reinterpret_cast<const uint8_t *>(g_zero_chunk);
  const int chunk = (lane & 3) ^ ((lane >> 4) & 3);
  const int wk = wave * C::KROWS + lane / (64 / C::KROWS);
  int32_t limit = p.chunks;  // 0: no tile, zeros are staged
  const auto aim = [&](const BatchedTile &u) {
    const int lane = fresh_lane(), lr = lane >> 2, chunk = (lane & 3) ^ ((lane >> 4) & 3);
    const int wk = wave * C::KROWS + lane / (64 / C::KROWS);
    const int slot = lane % (64 / C::KROWS);
    const uint8_t *we = p.w + u.e * p.w_mat, *xe = p.x + u.e * p.x_mat;
#pragma unroll
    for (int j = 0; j < C::LOADS; ++j) {
      const bool weight = j < WL;
      const uint8_t *base = weight ? we : xe;
      const int64_t stride = weight ? p.w_row : p.x_row;
      const int32_t first = weight ? u.n0 : u.m0, size = weight ? p.N : p.M;
      const int jj = weight ? j : j - WL;
      if (weight ? C::WT : C::XT) {
        const int column = first + 8 * (slot ^ (weight ? C::w_slot(wk) : C::x_slot(wk)));
        from[j] = base + (wk + jj * 4 * C::KROWS) * stride + 2 * min(column, size - 8);
      } else {
        const int r = (jj * 4 + wave) * 16 + lr, part = r & ~(C::HALF - 1), t = r % C::HALF / 32, q = r & 31;
        const int row = first + part + (weight ? C::w_row(q, t) : 32 * t + 4 * C::x_unit(q >> 2) + (q & 3));
        from[j] = base + min(row, size - 1) * stride + 16 * chunk;
      }
    }
  };
  const auto fetch_one = [&](int s, uint8_t *base, auto jc) {
    constexpr int j = decltype(jc)::value, jj = j < WL ? j : j - WL;
    uint8_t *to = base + (j < WL ? 0 : C::TILE * 64) + (jj * 4 + wave) * 1024;
    if constexpr (j < WL ? C::WT : C::XT) {
      dma_wave(32 * s + wk + jj * 4 * C::KROWS < 8 * limit ? from[j] : zero, to, 16);
      from[j] += 32 * (j < WL ? p.w_row : p.x_row);
    } else {
      dma_wave(4 * s + chunk < limit ? from[j] : zero, to, 16);
      from[j] += 64;
    }
  };

  // Fragment addresses inside an operand's part of a stage.
  const int fr = lane & 31;
  // Lane 16 g + 4 j + b of a transposing read addresses row j and unit 4 (g % 2) + b
  // of the fragment's 8, in half g / 2.
  int wcol[C::WT ? C::MI : 1], xcol[C::XT ? C::MI : 1];
  {
    const int j = (lane >> 2) & 3, unit = 4 * ((lane >> 4) & 1) + (lane & 3);
#pragma unroll
    for (int i = 0; i < C::MI; ++i) {
      const int wu = wn * (C::HALF / 4) + C::w_unit(unit, i), xu = wm * (C::HALF / 4) + 8 * i + C::x_unit(unit);
      if constexpr (C::WT) wcol[i] = (8 * half + j) * (2 * C::TILE) + 16 * ((wu >> 1) ^ C::w_slot(j)) + 8 * (wu & 1);
      if constexpr (C::XT) xcol[i] = (8 * half + j) * (2 * C::TILE) + 16 * ((xu >> 1) ^ C::x_slot(j)) + 8 * (xu & 1);
    }
  }
  struct Frag {
    uint4 a[C::MI], b[C::MI];
  };
  // Item r of a step's fragment reads, in the order the products need them:
  // a[0], all of b, then the other a.
  const auto read_item = [&](Frag &f, const uint8_t *base, int s, auto rc) {
    constexpr int r = decltype(rc)::value;
    constexpr bool x = r >= 1 && r <= C::MI;
    constexpr int i = x ? r - 1 : r == 0 ? 0 : r - C::MI;
    const uint8_t *part = base + (x ? C::TILE * 64 : 0);
    uint4 v;
    if constexpr (x ? C::XT : C::WT) {
      const uint8_t *src = part + (x ? xcol[C::XT ? i : 0] : wcol[C::WT ? i : 0]) + 16 * s * (2 * C::TILE);
      const uint2 lo = read_tr(src), hi = read_tr(src + 4 * (2 * C::TILE));
      v = make_uint4(lo.x, lo.y, hi.x, hi.y);
    } else {
      v = *reinterpret_cast<const uint4 *>(part + ((x ? wm : wn) * C::HALF + 32 * i + fr) * 64 + 16 * ((2 * s + half) ^ ((fr >> 2) & 3)));
    }
    if constexpr (x) f.b[i] = v;
    else f.a[i] = v;
  };

  f32x16 acc[C::MI][C::MI];  // [columns][rows]
  Frag f0, f1;
  // One step of 16 of K: the products of `f` with the reads of `g` (step gs of
  // the stage at gbase) and, in a stage's second, the staging of stage ds
  // between them, in exactly this order.
  const auto step = [&](auto sel, const Frag &f, Frag &g, const uint8_t *gbase, int gs, int ds, uint8_t *dbase) {
    constexpr int SLOTS = C::MI * C::MI, DN = decltype(sel)::value == 1 ? C::LOADS : 0;
    constexpr int READS = 2 * C::MI, RPS = (READS + SLOTS - 1) / SLOTS, DPS = (DN + SLOTS - 1) / SLOTS;
    each<SLOTS>([&](auto slot) {
      constexpr int n = decltype(slot)::value, i = n / C::MI, k = n % C::MI;
      acc[i][k] = mfma_f16(f.b[k], f.a[i], acc[i][k]);
      each<RPS>([&](auto q) {
        constexpr int r = n * RPS + decltype(q)::value;
        if constexpr (r < READS) read_item(g, gbase, gs, std::integral_constant<int, r>{});
      });
      each<DPS>([&](auto q) {
        constexpr int d = n * DPS + decltype(q)::value;
        if constexpr (d < DN) fetch_one(ds, dbase, std::integral_constant<int, d>{});
      });
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  // One stage.  Its second step's fragments are in registers after the first,
  // so behind one barrier its buffer is free for the stage four further on (ds
  // of its tile), and the next stage has landed.
  uint32_t cur = 0;  // the stage's buffer
  const auto stage = [&](int ds) {
    const uint32_t nxt = cur == (C::BUFFERS - 1) * C::STAGE ? 0 : cur + C::STAGE;
    step(std::integral_constant<int, 0>{}, f0, f1, lds + cur, 1, 0, lds);
    wait_lgkm0();
    wait_vm<(C::BUFFERS - 2) * C::LOADS>();  // all but the youngest stages have landed
    barrier_no_fence();
    step(std::integral_constant<int, 1>{}, f1, f0, lds + nxt, 0, ds, lds + cur);
    cur = nxt;
  };

  const int stages = max((p.chunks + 3) / 4, C::BUFFERS);  // a short K: stages of zeros
  aim(t);
  each<C::BUFFERS>([&](auto b) {
    each<C::LOADS>([&](auto j) { fetch_one(decltype(b)::value, lds + decltype(b)::value * C::STAGE, j); });
  });
  advance();
  wait_vm<(C::BUFFERS - 1) * C::LOADS>();
  barrier_no_fence();
  each<2 * C::MI>([&](auto r) { read_item(f0, lds, 0, r); });
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
      stage(s);
    }
    // The last stages bring the next tile's first.
    limit = nt.e < 0 ? 0 : p.chunks;
    if (nt.e >= 0) aim(nt);
    for (int s = 0; s < C::BUFFERS; ++s) {
      pin();
      stage(s);
    }
    pin();

    // ---- the tile's results, 4 registers' rows of all fragments at a time
    constexpr int V = C::MI, GROUPS = 4 * C::MI, AHEAD = 3;  // group g: row fragment g / 4, registers 4 (g % 4) ..
    const int fl = fresh_lane(), fh = fl >> 5, fp = fl & 31;
    const int32_t wm0 = t.m0 + wm * C::HALF, wn0 = t.n0 + wn * C::HALF;
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
    const int64_t stride = 2 * static_cast<int64_t>(p.N);
    const int64_t matrix = 2 * static_cast<int64_t>(t.e) * p.M * p.N;
    const auto rows_left = [&](int k) { return p.M - (wm0 + 32 * k); };
    const auto offset = [&](int k) {
      return at_col + (fh != 0 && rows_left(k) > 16 ? 16 * static_cast<uint32_t>(stride) : 0u);
    };
    // Byte of a group's first row.  Made where the compiler does not see it
    // before: it would compute all groups' at once and has no registers for them.
    const auto group_at = [&](int g) -> int64_t {
      int32_t row = min(wm0 + 32 * (g / 4), p.M - 16) + 4 * (g % 4);
      asm volatile("" : "+s"(row));
      return matrix + row * stride;
    };
    struct Group {
      Neighbours<V> in[4], in2[4];
    };
    Group ring[AHEAD + 1];
    const auto load_group = [&](Group &u, int g) {
      if constexpr (EPI != kEpiGram) {
        const uint32_t lane_at = offset(g / 4);
        const int64_t at = group_at(g);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          u.in[r] = load_neighbours<V>(reinterpret_cast<const uint8_t *>(p.in) + (at + r * stride) + lane_at);
          if constexpr (EPI == kEpiNext || EPI == kEpiLast)
            u.in2[r] = load_neighbours<V>(reinterpret_cast<const uint8_t *>(p.in2) + (at + r * stride) + lane_at);
        }
      }
    };
    each<AHEAD>([&](auto gc) { load_group(ring[decltype(gc)::value], decltype(gc)::value); });
    const bool mirror = SYM && t.m0 != t.n0;
    each<GROUPS>([&](auto gc) {
      constexpr int g = decltype(gc)::value, k = g / 4, r0 = 4 * (g % 4);
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
            if constexpr (EPI == kEpiNext || EPI == kEpiLast) {
              const f16x2 x = __builtin_bit_cast(f16x2, u.in2[r].w[i / 2]);
              v[i] = __builtin_fmaf(static_cast<float>(x[0]), p.beta, v[i]);
              v[i + 1] = __builtin_fmaf(static_cast<float>(x[1]), p.beta, v[i + 1]);
            }
            if constexpr (EPI == kEpiLast) {
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
        const uint32_t lane_at = offset(k);
        if (col_ok && rows_left(k) > 16 * fh) {
          const int64_t at = group_at(g);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            store_neighbours<V>(reinterpret_cast<uint8_t *>(p.out) + (at + r * stride) + lane_at, out[r]);
            if constexpr (EPI == kEpiNext)
              store_neighbours<V>(reinterpret_cast<uint8_t *>(p.out2) + (at + r * stride) + lane_at, out2[r]);
          }
        }
      }
      if constexpr (SYM && g % 4 == 3) {
        if (mirror) {
          const int32_t at_row = wm0 + 32 * k + 16 * fh;
#pragma unroll
          for (int i = 0; i < V; ++i) {  // a lane's 16 rows of column i are neighbours in a row
            const int32_t row = wn0 + (C::WT ? 4 * C::w_unit(fp >> 2, i) + (fp & 3) : C::w_row(fp, i));
            if (row < p.N && at_row < p.M) {
              uint32_t w[8];
#pragma unroll
              for (int r = 0; r < 8; ++r) {
                const float scale = EPI == kEpiGram ? p.alpha : 1.0f;
                w[r] = pack_f16(scale * acc[i][k][2 * r], scale * acc[i][k][2 * r + 1]);
              }
              uint4 *to = reinterpret_cast<uint4 *>(reinterpret_cast<uint8_t *>(p.out) + matrix + row * stride + 2 * at_row);
              to[0] = make_uint4(w[0], w[1], w[2], w[3]);
              to[1] = make_uint4(w[4], w[5], w[6], w[7]);
            }
          }
        }
      }
      if constexpr (g % 4 == 3) {
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i][k] = f32x16{};
      }
      __builtin_amdgcn_sched_barrier(0);
    });
    if (nt.e < 0) break;
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
  const int64_t grid = std::min<int64_t>(tiles, 256 * PER_CU);
  hipLaunchKernelGGL((k_batched<C, EPI>), dim3(static_cast<unsigned>(grid)), dim3(256), 0, stream, p,
                     static_cast<uint32_t>(per_matrix), static_cast<uint32_t>(c));
  return hipGetLastError();
}

// The large tile reads each operand half as often; small ones, two a CU, fill
// the card with few matrices.
template <bool XT, bool WT, int EPI>
hipError_t launch_batched(const BatchedParams &p, hipStream_t stream) {
  constexpr bool SYM = EPI == kEpiGram || EPI == kEpiPoly;
  const auto rounds = [&](int64_t tile, int64_t places) {
    const int64_t r = (p.M + tile - 1) / tile, c = (p.N + tile - 1) / tile;
    return (p.batch * (SYM ? r * (r + 1) / 2 : r * c) + places - 1) / places;
  };
  if (100 * rounds(256, 256) <= 60 * rounds(128, 512)) return launch_batched_tiles<BatchedCfg<256, XT, WT>, EPI>(p, stream);
  return launch_batched_tiles<BatchedCfg<128, XT, WT>, EPI>(p, stream);
}

}  // namespace quads
