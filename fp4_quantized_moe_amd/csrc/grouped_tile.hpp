// Shared pieces of the MXFP4 and gated grouped GEMM kernels: finding the
// (expert, rows) of a tile, operand chunks, and the epilogues.
//
// Every kernel computes 32 x 32 accumulator tiles with the WEIGHT rows n as
// MFMA's first operand and the routed rows m as its second, so a lane holds
// one routed row (m = lane % 32) and 16 of the tile's 32 output columns: its
// element r is column 8 (r / 4) + 4 (lane / 32) + r % 4.  Four consecutive
// columns of a row are then one vector store, and the two lanes l, l + 32
// hold a whole 32-column MX block of a row, which lets an epilogue
// requantize without LDS.
//
// Operands are rows of 16-byte chunks along the contraction (32 MXFP4
// elements = one scaling block, or 8 bf16).  One MFMA contracts two chunks:
// lanes 0-31 supply the first, lanes 32-63 the second.  Any chunk order is
// right as long as both operands use the same one.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp4_mfma.hpp"
#include "mx_launch.hpp"
#include "mx_device.hpp"
#include "quads_device.hpp"

namespace quads {

typedef int i32x8 __attribute__((ext_vector_type(8)));

struct GroupedParams {
  const uint8_t *x, *x_scales;  // routed-row operand (rows x_row bytes apart)
  const uint8_t *w, *w_scales;  // weights [E, N, K]
  const int32_t *row_token;     // or null: identity
  const int32_t *offsets;       // [E + 1]
  int E;
  int32_t N;          // weight rows per expert
  int32_t width;      // columns of a tile pass: N, or N / 2 for the SwiGLU epilogues
  int32_t chunks;     // 16-byte chunks of a row
  int64_t x_row, w_row;      // row strides in bytes
  int64_t w_expert;          // expert stride in bytes
  void *y;
  void *y2;           // kEpiSwiglu: pre-activations or null; kEpiSwigluMx: scales
  const uint16_t *gu;  // kEpiGatedBwd
};

enum GroupedOperands {
  kOpMx = 0,    // MXFP4 rows, weights [E, N, K]
  kOpBf16 = 1,  // bf16 rows, weights [E, N, K]
  kOpBf16T = 2  // bf16 rows, weights [E, K, N] (contraction along the weights' rows)
};

// Zeros that are read in the place of chunks and scales behind K (a scale byte
// 0 is 2^-127).  Choosing the address, not the data, keeps loads in flight.
__device__ __attribute__((aligned(16))) uint32_t g_zero_chunk[4];

struct TileAt {
  int e;          // expert, or -1: past the last tile
  int32_t r0;     // first routed row
  int32_t rows;   // rows of this tile (1 .. TM)
  int32_t total;  // row tiles of all experts
  int32_t before;  // row tiles of the experts before e
};

// Row tile `index` of the grouping: experts' rows are cut into tiles of TM.
// Every wave finds it alone: 64 experts at a time, one a lane, a wave scan of
// their tiles.  offsets is non-decreasing.
template <int TM>
__device__ __forceinline__ TileAt find_tile(const int32_t *offsets, int E, int index) {
  const int lane = threadIdx.x & 63;
  TileAt t{-1, 0, 0, 0, 0};
  for (int e0 = 0; e0 < E; e0 += 64) {
    const int e = e0 + lane;
    const int32_t lo = offsets[min(e, E)], hi = offsets[min(e + 1, E)];
    const int32_t n = (hi - lo + TM - 1) / TM;
    const int32_t end = t.total + static_cast<int32_t>(wave_scan<false>(static_cast<uint32_t>(n)));
    const uint64_t here = __ballot(index >= end - n && index < end);
    if (here) {
      const int owner = __builtin_ctzll(here);
      t.e = e0 + owner;
      t.before = __builtin_amdgcn_readlane(end - n, owner);
      t.r0 = __builtin_amdgcn_readlane(lo, owner) + (index - t.before) * TM;
      t.rows = min(__builtin_amdgcn_readlane(hi, owner) - t.r0, static_cast<int32_t>(TM));
    }
    t.total = __builtin_amdgcn_readlane(end, 63);
  }
  return t;
}

// All row tiles.
template <int TM>
__device__ __forceinline__ int32_t count_tiles(const int32_t *offsets, int E) {
  return find_tile<TM>(offsets, E, -1).total;
}

// Row tiles in increasing order, without scans: experts are walked by scalar loads.
struct Walker {
  typedef const __attribute__((address_space(4))) int32_t uniform_i32;
  uniform_i32 *offsets;
  int32_t e, before, first, last;  // expert, row tiles before it, its rows
  __device__ __forceinline__ Walker(const int32_t *o, const TileAt &t)
      : offsets((uniform_i32 *)reinterpret_cast<uintptr_t>(o)), e(t.e), before(t.before), first(offsets[t.e]), last(offsets[t.e + 1]) {}
  // Row tile `index`, which exists and is no earlier than the last one asked for.
  template <int TM>
  __device__ __forceinline__ void to(int32_t index, int32_t &r0, int32_t &rows) {
    int32_t n = (last - first + TM - 1) / TM;
    while (index >= before + n) {
      before += n;
      ++e;
      first = last;
      last = offsets[e + 1];
      n = (last - first + TM - 1) / TM;
    }
    r0 = first + (index - before) * TM;
    rows = min(last - r0, static_cast<int32_t>(TM));
  }
};

__device__ __forceinline__ int64_t source_row(const GroupedParams &p, int32_t row) {
  return p.row_token ? p.row_token[row] : row;
}

__device__ __forceinline__ f32x16 mfma_bf16(uint4 a, uint4 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Byte SEL of sa / sb scales the lane's chunk.
template <int SEL>
__device__ __forceinline__ f32x16 mfma_mx(uint4 a, uint4 b, f32x16 c, uint32_t sa, uint32_t sb) {
  i32x8 va = {}, vb = {};
  va[0] = a.x;
  va[1] = a.y;
  va[2] = a.z;
  va[3] = a.w;
  vb[0] = b.x;
  vb[1] = b.y;
  vb[2] = b.z;
  vb[3] = b.w;
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(va, vb, c, 4, 4, SEL, static_cast<int>(sa), SEL,
                                                         static_cast<int>(sb));
}

// The operand lanes 32 apart: {lower lanes' v in both, upper lanes' v in both}.
__device__ __forceinline__ uint2 both_halves(uint32_t v) {
  const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return make_uint2(r[0], r[1]);
}

// Requantizes one 32-column block of 32 rows held as h[16] per lane.  Codes
// go to `codes` + 16 bytes of the block, the scale byte to *scale.
__device__ __forceinline__ void store_mx_block(const float (&h)[16], int lane, bool row_ok, uint8_t *codes, uint8_t *scale) {
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) a = max(a, __float_as_uint(h[i]) & 0x7FFFFFFFu);
  const uint2 m = both_halves(a);
  const uint32_t s = mx_scale_byte(max(m.x, m.y), 0u);
  const float inv = mx_inv_scale(s);
  float t[8];
  uint32_t lo, hi;  // quads 0, 1 and quads 2, 3 of this lane's columns, 16 bits each
#pragma unroll
  for (int i = 0; i < 8; ++i) t[i] = h[i] * inv;
  lo = mx_pack8(t);
#pragma unroll
  for (int i = 0; i < 8; ++i) t[i] = h[8 + i] * inv;
  hi = mx_pack8(t);
  if (s == kMxNan) lo = hi = 0;
  // Byte 4 q + 2 half of the block holds quad q of that half.  Lower lanes
  // store dwords 0 and 1, upper lanes dwords 2 and 3.
  const auto r = __builtin_amdgcn_permlane32_swap(lo, hi, false, false);
  const uint32_t d0 = (r[0] & 0xFFFFu) | (r[1] << 16), d1 = (r[0] >> 16) | (r[1] & 0xFFFF0000u);
  if (row_ok) {
    const int half = lane >> 5;
    *reinterpret_cast<uint2 *>(codes + 8 * half) = make_uint2(d0, d1);
    if (half == 0) *scale = static_cast<uint8_t>(s);
  }
}

// 1 / (1 + e^-z) as in silu: off by (5 + 1.23 |z|) 2^-24 of it, of which 1.23 |z|
// is the argument of exp2 (its product and constant), and 0 below z = -87.3,
// where the reciprocal is subnormal.  The outputs are rounded to bf16 (2^-8) or
// MXFP4 next.
__device__ __forceinline__ float sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-z * 1.44269504088896341f));
}

// Gradients of h = silu(g) u from d = dh, in place of g and u: with
// s = sigmoid(g), d gate = d u s (1 + g (1 - s)) and d up = d g s.
__device__ __forceinline__ void gated_grad(float d, float &g, float &u) {
  const float s = sigmoid(g), z = g;
  g = d * u * (s * (1.0f + z * (1.0f - s)));
  u = d * (z * s);
}

// Stores one 32 (columns n0 ..) x 32 (rows) tile: `a` is the accumulator
// (the gate's with the SwiGLU epilogues, whose up projection is `b`).  `row`
// is the lane's routed row, row_ok whether the tile has it.  Columns are
// whole quads: width % 16 == 0.
template <int EPI>
__device__ __forceinline__ void store_tile(const GroupedParams &p, const f32x16 &a, const f32x16 &b, int64_t row,
                                           bool row_ok, int32_t n0) {
  const int half = (threadIdx.x & 63) >> 5;
  if constexpr (EPI == kEpiSwigluMx) {
    float h[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) h[i] = silu(a[i]) * b[i];
    if (n0 >= p.width) return;
    store_mx_block(h, threadIdx.x & 63, row_ok, static_cast<uint8_t *>(p.y) + row * (p.width >> 1) + (n0 >> 1),
                   static_cast<uint8_t *>(p.y2) + row * (p.width >> 5) + (n0 >> 5));
  } else {
    if (!row_ok) return;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int32_t n = n0 + 8 * q + 4 * half;
      if (n >= p.width) continue;
      if constexpr (EPI == kEpiF32) {
        *reinterpret_cast<float4 *>(static_cast<float *>(p.y) + row * p.width + n) =
            make_float4(a[4 * q], a[4 * q + 1], a[4 * q + 2], a[4 * q + 3]);
      } else if constexpr (EPI == kEpiBf16) {
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.y) + row * p.width + n) =
            make_uint2(pack_bf16(a[4 * q], a[4 * q + 1]), pack_bf16(a[4 * q + 2], a[4 * q + 3]));
      } else if constexpr (EPI == kEpiSwiglu) {
        float h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = silu(a[4 * q + i]) * b[4 * q + i];
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.y) + row * p.width + n) =
            make_uint2(pack_bf16(h[0], h[1]), pack_bf16(h[2], h[3]));
        if (p.y2) {
          uint16_t *pre = static_cast<uint16_t *>(p.y2) + row * 2 * p.width + n;
          *reinterpret_cast<uint2 *>(pre) =
              make_uint2(pack_bf16(a[4 * q], a[4 * q + 1]), pack_bf16(a[4 * q + 2], a[4 * q + 3]));
          *reinterpret_cast<uint2 *>(pre + p.width) =
              make_uint2(pack_bf16(b[4 * q], b[4 * q + 1]), pack_bf16(b[4 * q + 2], b[4 * q + 3]));
        }
      }
    }
  }
}

}  // namespace quads
