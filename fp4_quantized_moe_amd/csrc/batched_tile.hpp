// LDS-staged products of a batch of fp16 matrices, Y[i, j] = sum_k X[i, k] W[j, k]
// for each, with the epilogues of a Newton-Schulz step.  Either operand may be
// stored with the contraction along its rows (X as [K, M], W as [K, N]).
//
// Stages, swizzles, fragment reads and the pipeline are those of
// grouped_staged.hpp (its comments say why); what differs: fp16, every matrix
// of the same size, either operand by transposing reads, and symmetric
// results, of which only the tiles on and below the diagonal are computed and
// those below it stored twice.
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

__device__ __forceinline__ void unpack_f16(uint32_t w, float &lo, float &hi) {
  const f16x2 p = __builtin_bit_cast(f16x2, w);
  lo = static_cast<float>(p[0]);
  hi = static_cast<float>(p[1]);
}

// lo = v less its fp16 rounding (exact in fp32).
template <int N>
__device__ __forceinline__ void split_f16(const float (&v)[N], float (&lo)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) lo[i] = v[i] - static_cast<float>(static_cast<_Float16>(v[i]));
}

enum BatchedEpi {
  kEpiGram = 0,  // out = alpha Y, symmetric
  kEpiPoly = 1,  // out = beta in + alpha Y, symmetric
  kEpiNext = 2,  // v = beta (in + in2) + alpha Y; out = fp16(v), out2 = fp16(v - out)
  kEpiLast = 3   // out = bf16(beta (in + in2) + alpha Y)
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
  static constexpr int STAGE = 2 * TILE * 128;
  static constexpr int LOADS = TILE / 16;              // staging instructions of a wave and stage, both operands
  static constexpr int LATE = LOADS * 3 / 4;
  static constexpr int KROWS = 512 / TILE;             // transposed operand: stored rows of an instruction
  static constexpr int TURN = 2 * STAGE, TURN_BYTES = 32 * 128;
  static constexpr int LDS = TURN + 4 * TURN_BYTES;
};

// One 32 x 32 tile as fp16 columns [32 i, 32 i + 32) of a turned-around block of 32 rows of 64.
__device__ __forceinline__ void turn_put_f16(uint8_t *turn, int lane, int i, const float (&v)[16]) {
  const int half = lane >> 5, fr = lane & 31;
#pragma unroll
  for (int q = 0; q < 4; ++q)
    *reinterpret_cast<uint2 *>(turn + turn_at<128>(fr, 4 * i + q) + 8 * half) =
        make_uint2(pack_f16(v[4 * q], v[4 * q + 1]), pack_f16(v[4 * q + 2], v[4 * q + 3]));
}

// Its transpose, as columns [32 i, 32 i + 32) of the block.
__device__ __forceinline__ void turn_put_f16_t(uint8_t *turn, int lane, int i, const f32x16 &v) {
  const int half = lane >> 5, col = 32 * i + (lane & 31);
#pragma unroll
  for (int r = 0; r < 16; ++r)
    *reinterpret_cast<_Float16 *>(turn + turn_at<128>(8 * (r >> 2) + 4 * half + (r & 3), col >> 3) + 2 * (col & 7)) =
        static_cast<_Float16>(v[r]);
}

__device__ __forceinline__ void turn_get_f16(const uint8_t *turn, int lane, int i, float (&v)[16]) {
  const int half = lane >> 5, fr = lane & 31;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint2 w = *reinterpret_cast<const uint2 *>(turn + turn_at<128>(fr, 4 * i + q) + 8 * half);
    unpack_f16(w.x, v[4 * q], v[4 * q + 1]);
    unpack_f16(w.y, v[4 * q + 2], v[4 * q + 3]);
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
  const int chunk = (lane & 7) ^ ((4 * wave + (lane >> 4)) & 7);
  const int wk = wave * C::KROWS + lane / (64 / C::KROWS);
  int32_t limit = p.chunks;  // 0: no tile, zeros are staged
  const auto aim = [&](const BatchedTile &u) {
    const int lane = fresh_lane(), lr = lane >> 3, chunk = (lane & 7) ^ ((4 * wave + (lr >> 1)) & 7);
    const int wk = wave * C::KROWS + lane / (64 / C::KROWS);
    const int tc = 8 * ((lane % (64 / C::KROWS)) ^ ((wk & 3) << 2));
    const uint8_t *we = p.w + u.e * p.w_mat, *xe = p.x + u.e * p.x_mat;
#pragma unroll
    for (int j = 0; j < C::LOADS; ++j) {
      const bool weight = j < WL;
      const uint8_t *base = weight ? we : xe;
      const int64_t stride = weight ? p.w_row : p.x_row;
      const int32_t first = weight ? u.n0 : u.m0, size = weight ? p.N : p.M;
      const int jj = weight ? j : j - WL;
      if (weight ? C::WT : C::XT)
        from[j] = base + (wk + jj * 4 * C::KROWS) * stride + 2 * min(first + tc, size - 8);
      else
        from[j] = base + min(first + (jj * 4 + wave) * 8 + lr, size - 1) * stride + 16 * chunk;
    }
  };
  const auto fetch_one = [&](int s, uint8_t *base, auto jc) {
    constexpr int j = decltype(jc)::value, jj = j < WL ? j : j - WL;
    uint8_t *to = base + (j < WL ? 0 : C::TILE * 128) + (jj * 4 + wave) * 1024;
    if constexpr (j < WL ? C::WT : C::XT) {
      dma_wave(64 * s + wk + jj * 4 * C::KROWS < 8 * limit ? from[j] : zero, to, 16);
      from[j] += 64 * (j < WL ? p.w_row : p.x_row);
    } else {
      dma_wave(8 * s + chunk < limit ? from[j] : zero, to, 16);
      from[j] += 128;
    }
  };

  // Fragment addresses inside an operand's part of a stage.
  const int fr = lane & 31;
  const auto column = [&](int first) {  // of a transposed operand: of the 32 columns from `first` on
    const int j = (lane >> 2) & 3;
    const int c = first / 8 + 2 * ((lane >> 4) & 1) + ((lane >> 1) & 1);
    return (32 * half + j) * (2 * C::TILE) + 16 * (c ^ (j << 2)) + 8 * (lane & 1);
  };
  int wcol[C::WT ? C::MI : 1], xcol[C::XT ? C::MI : 1];
  if constexpr (C::WT) {
#pragma unroll
    for (int i = 0; i < C::MI; ++i) wcol[i] = column(wn * C::HALF + 32 * i);
  }
  if constexpr (C::XT) {
#pragma unroll
    for (int i = 0; i < C::MI; ++i) xcol[i] = column(wm * C::HALF + 32 * i);
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
    const uint8_t *part = base + (x ? C::TILE * 128 : 0);
    uint4 v;
    if constexpr (x ? C::XT : C::WT) {
      const uint8_t *src = part + (x ? xcol[C::XT ? i : 0] : wcol[C::WT ? i : 0]) + 8 * s * (2 * C::TILE);
      const uint2 lo = read_tr(src), hi = read_tr(src + 4 * (2 * C::TILE));
      v = make_uint4(lo.x, lo.y, hi.x, hi.y);
    } else {
      v = *reinterpret_cast<const uint4 *>(part + ((x ? wm : wn) * C::HALF + 32 * i + fr) * 128 + 16 * ((4 * half + s) ^ ((fr >> 1) & 7)));
    }
    if constexpr (x) f.b[i] = v;
    else f.a[i] = v;
  };

  f32x16 acc[C::MI][C::MI];  // [columns][rows]
  Frag f0, f1;
  const auto step = [&](auto sel, const Frag &f, Frag &g, const uint8_t *gbase, int gs, int ds, uint8_t *dbase) {
    constexpr int S = decltype(sel)::value, SLOTS = C::MI * C::MI;
    constexpr int DF = S == 3 ? 0 : C::LATE, DN = S == 3 ? C::LATE : S == 0 ? C::LOADS - C::LATE : 0;
    constexpr int READS = 2 * C::MI, RPS = (READS + SLOTS - 1) / SLOTS, DPS = (DN + SLOTS - 1) / SLOTS;
    each<SLOTS>([&](auto slot) {
      constexpr int n = decltype(slot)::value, i = n / C::MI, k = n % C::MI;
      acc[i][k] = mfma_f16(f.a[i], f.b[k], acc[i][k]);
      each<RPS>([&](auto q) {
        constexpr int r = n * RPS + decltype(q)::value;
        if constexpr (r < READS) read_item(g, gbase, gs, std::integral_constant<int, r>{});
      });
      each<DPS>([&](auto q) {
        constexpr int d = n * DPS + decltype(q)::value;
        if constexpr (d < DN) fetch_one(ds, dbase, std::integral_constant<int, DF + d>{});
      });
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  uint8_t *cur = lds;
  const auto stage = [&](int now, int ds, auto between) {
    uint8_t *nxt = lds + (cur == lds ? C::STAGE : 0);
    step(std::integral_constant<int, 0>{}, f0, f1, cur, 1, now, nxt);
    step(std::integral_constant<int, 1>{}, f1, f0, cur, 2, 0, cur);
    between();
    step(std::integral_constant<int, 2>{}, f0, f1, cur, 3, 0, cur);
    wait_lgkm0();  // step 3's fragments are in registers: this wave is done with the stage's LDS
    wait_vm<0>();  // and its part of the next stage has landed
    barrier_no_fence();
    step(std::integral_constant<int, 3>{}, f1, f0, nxt, 0, ds, cur);
    cur = nxt;
  };

  const int stages = max((p.chunks + 7) / 8, 2);  // at least both buffers: one of zeros for a short K
  aim(t);
  each<C::LOADS>([&](auto j) { fetch_one(0, lds, j); });
  each<C::LATE>([&](auto j) { fetch_one(1, lds + C::STAGE, j); });
  advance();
  wait_vm<C::LATE>();
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
    for (int s = 2; s < stages; ++s) {
      pin();
      stage(s - 1, s, [] {});
    }
    pin();
    // The last two stages bring the next tile's first two.
    stage(stages - 1, 0, [&] {
      limit = nt.e < 0 ? 0 : p.chunks;
      if (nt.e >= 0) aim(nt);
    });
    pin();
    stage(0, 1, [] {});
    pin();

    // ---- the tile's results, a block of 32 rows and 64 columns at a time
    uint8_t *turn = lds + C::TURN + wave * C::TURN_BYTES;
    const int fl = fresh_lane();
    const int32_t wm0 = t.m0 + wm * C::HALF, wn0 = t.n0 + wn * C::HALF;
    const int64_t mat = static_cast<int64_t>(t.e) * p.M * p.N, stride = 2 * static_cast<int64_t>(p.N);
    const bool mirror = SYM && t.m0 != t.n0;
    each<C::MI / 2>([&](auto kp) {
      constexpr int k0 = 2 * decltype(kp)::value;
      each<C::MI / 2>([&](auto ip) {
        constexpr int i0 = 2 * decltype(ip)::value;
        const int32_t n = wn0 + 32 * i0;
        each<2>([&](auto kk) {
          constexpr int k = k0 + decltype(kk)::value;
          const int32_t row = wm0 + 32 * k;
          const int rows = p.M - row, limit_bytes = 2 * (p.N - n);
          const int64_t first = mat + static_cast<int64_t>(row) * p.N + n;
          float v[2][16];
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            asm volatile("" : "+a"(acc[i0 + q][k]));  // not read before its turn
#pragma unroll
            for (int r = 0; r < 16; ++r) v[q][r] = p.alpha * acc[i0 + q][k][r];
          }
          if (rows > 0 && limit_bytes > 0) {
            if constexpr (EPI != kEpiGram) {
              TurnLoad<128> in, in2;
              in.load(reinterpret_cast<const uint8_t *>(p.in + first), fl, stride, rows, limit_bytes);
              if constexpr (EPI != kEpiPoly) in2.load(reinterpret_cast<const uint8_t *>(p.in2 + first), fl, stride, rows, limit_bytes);
              float w[2][16];
              in.put(turn, fl);
#pragma unroll
              for (int q = 0; q < 2; ++q) turn_get_f16(turn, fl, q, w[q]);
              if constexpr (EPI != kEpiPoly) {
                in2.put(turn, fl);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                  float lo[16];
                  turn_get_f16(turn, fl, q, lo);
#pragma unroll
                  for (int r = 0; r < 16; ++r) w[q][r] += lo[r];
                }
              }
#pragma unroll
              for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int r = 0; r < 16; ++r) v[q][r] = __builtin_fmaf(p.beta, w[q][r], v[q][r]);
            }
            if constexpr (EPI == kEpiLast) {
#pragma unroll
              for (int q = 0; q < 2; ++q) turn_put_bf16<128>(turn, fl, q, v[q]);
            } else {
#pragma unroll
              for (int q = 0; q < 2; ++q) turn_put_f16(turn, fl, q, v[q]);
            }
            turn_store<128>(turn, fl, reinterpret_cast<uint8_t *>(p.out + first), stride, rows, limit_bytes);
            if constexpr (EPI == kEpiNext) {
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                float lo[16];
                split_f16(v[q], lo);
                turn_put_f16(turn, fl, q, lo);
              }
              turn_store<128>(turn, fl, reinterpret_cast<uint8_t *>(p.out2 + first), stride, rows, limit_bytes);
            }
          }
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            if constexpr (SYM) {
#pragma unroll
              for (int r = 0; r < 16; ++r) acc[i0 + q][k][r] = v[q][r];
            } else {
              acc[i0 + q][k] = f32x16{};
            }
          }
          __builtin_amdgcn_sched_barrier(0);
        });
        if constexpr (SYM) {
          // Columns n + 32 q .. of the 64 rows are rows of the transposed tile.
          each<2>([&](auto qc) {
            constexpr int q = decltype(qc)::value;
            const int32_t row = wn0 + 32 * (i0 + q), col = wm0 + 32 * k0;
            if (mirror) {
              turn_put_f16_t(turn, fl, 0, acc[i0 + q][k0]);
              turn_put_f16_t(turn, fl, 1, acc[i0 + q][k0 + 1]);
              if (p.N > row && p.M > col)
                turn_store<128>(turn, fl, reinterpret_cast<uint8_t *>(p.out + mat + static_cast<int64_t>(row) * p.N + col), stride,
                                p.N - row, 2 * (p.M - col));
            }
            acc[i0 + q][k0] = f32x16{};
            acc[i0 + q][k0 + 1] = f32x16{};
            __builtin_amdgcn_sched_barrier(0);
          });
        }
      });
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
