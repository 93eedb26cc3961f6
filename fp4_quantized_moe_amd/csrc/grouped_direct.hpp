// Grouped GEMM without LDS: every wave computes one 32 x 32 tile (two with a
// SwiGLU epilogue) and loads its MFMA fragments straight from memory.  Right
// for every size the entry points accept; used where the staged kernels do
// not apply.
#pragma once

#include "grouped_tile.hpp"

namespace quads {

enum GroupedOperands {
  kOpMx = 0,    // MXFP4 rows, weights [E, N, K]
  kOpBf16 = 1,  // bf16 rows, weights [E, N, K]
  kOpBf16T = 2  // bf16 rows, weights [E, K, N] (contraction along the weights' rows)
};

constexpr int kDirectWaves = 4;

template <int OP, int EPI>
__global__ __launch_bounds__(64 * kDirectWaves) void k_grouped_direct(GroupedParams p, int col_groups) {
  const TileAt t = find_tile<32>(p.offsets, p.E, static_cast<int>(blockIdx.x / col_groups));
  if (t.e < 0) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, half = lane >> 5;
  const int32_t n0 = (static_cast<int32_t>(blockIdx.x % col_groups) * kDirectWaves + wave) * 32;
  if (n0 >= p.width) return;
  constexpr bool PAIR = EPI == kEpiSwiglu || EPI == kEpiSwigluMx;
  const int32_t n = min(n0 + (lane & 31), p.width - 1);
  const int64_t row = t.r0 + min(lane & 31, t.rows - 1);
  const int64_t src = source_row(p, static_cast<int32_t>(row));
  const uint8_t *xr = p.x + src * p.x_row;
  const uint8_t *we = p.w + t.e * p.w_expert;
  const int64_t up = static_cast<int64_t>(p.width) * p.w_row;
  const uint8_t *wr = OP == kOpBf16T ? we + 2 * static_cast<int64_t>(n) : we + n * p.w_row;
  const uint8_t *xs = nullptr, *ws = nullptr;
  if constexpr (OP == kOpMx) {
    xs = p.x_scales + src * p.chunks;
    ws = p.w_scales + (static_cast<int64_t>(t.e) * p.N + n) * p.chunks;
  }
  f32x16 acc = {}, acc2 = {};
  const uint4 zero = make_uint4(0, 0, 0, 0);
  const int steps = (p.chunks + 1) / 2;
  for (int s = 0; s < steps; ++s) {
    const int c = 2 * s + half;
    const bool in = c < p.chunks;
    const int cc = in ? c : 0;
    uint4 b = *reinterpret_cast<const uint4 *>(xr + 16 * static_cast<int64_t>(cc)), a, a2 = zero;
    if constexpr (OP == kOpBf16T) {
      uint32_t h[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) h[j] = *reinterpret_cast<const uint16_t *>(wr + (8 * static_cast<int64_t>(cc) + j) * p.w_row);
      a = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
    } else {
      a = *reinterpret_cast<const uint4 *>(wr + 16 * static_cast<int64_t>(cc));
      if constexpr (PAIR) a2 = *reinterpret_cast<const uint4 *>(wr + up + 16 * static_cast<int64_t>(cc));
    }
    if (!in) a = a2 = b = zero;
    if constexpr (OP == kOpMx) {
      uint32_t sb = xs[cc], sa = ws[cc], sa2 = 0;
      if constexpr (PAIR) sa2 = ws[static_cast<int64_t>(p.width) * p.chunks + cc];
      if (!in) sa = sa2 = sb = 127;  // 2^0
      acc = mfma_mx<0>(a, b, acc, sa, sb);
      if constexpr (PAIR) acc2 = mfma_mx<0>(a2, b, acc2, sa2, sb);
    } else {
      acc = mfma_bf16(a, b, acc);
      if constexpr (PAIR) acc2 = mfma_bf16(a2, b, acc2);
    }
  }
  store_tile<EPI>(p, acc, acc2, t.r0 + (lane & 31), (lane & 31) < t.rows, n0);
}

// Most row tiles of TM rows that R rows in E groups can give.
inline int64_t max_row_tiles(int64_t R, int E, int TM) { return R / TM + (R < E ? R : E); }

template <int OP, int EPI>
hipError_t launch_direct(const GroupedParams &p, int64_t R, hipStream_t stream) {
  const int64_t groups = (p.width + 32 * kDirectWaves - 1) / (32 * kDirectWaves);
  const int64_t grid = max_row_tiles(R, p.E, 32) * groups;
  if (grid > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((k_grouped_direct<OP, EPI>), dim3(static_cast<unsigned>(grid)), dim3(64 * kDirectWaves), 0, stream,
                     p, static_cast<int>(groups));
  return hipGetLastError();
}

}  // namespace quads
