// Grouped MXFP4 GEMM for few rows per expert and many columns in all (decode
// batches): each wave streams weight rows on its own, through LDS by DMA.
// Bound: reading the weights once.
//
// An item is 32 routed rows of an expert times two 32-column tiles (the gate
// and up tile of the same columns with the SwiGLU epilogues) over the whole
// contraction.  A stage is 128 bytes of its 64 weight and 32 routed rows with
// their scales, read in whole lines (a fragment's lanes read 16 bytes from 32
// rows, which the vector memory path takes a row at a time: straight into
// fragments the same bytes arrived at 3.3 TB/s).  Each wave keeps a ring of
// three stages and issues the DMA of the next but two as soon as a stage's
// fragments are in registers, also across items: no barriers, and about
// 100 KB of weights in flight on every CU.
//
// An expert with one row tile has its weights read past the caches, since nobody
// comes back to them; with more tiles the later ones find them there.  With the
// weights of four layers in turn, as in a model, 128 experts of 2048 -> 2 x 1024
// and back, the two products took (past the caches for experts of one tile / for
// all experts / for none): 256 tokens x 8 evenly routed 89.5 / 89.2 / 97.4 us,
// by Zipf(1.1) 107.4 / 112.4 / 109.9; 512 tokens evenly 130.5 / 143.1 / 131.3,
// by Zipf 133.5 / 158.4 / 134.3.  A lone layer, warm: 89.2 / 89.3 / 96.4,
// 106.3 / 112.5 / 107.8, 124.7 / 143.2 / 127.7 and 129.0 / 158.1 / 131.4.
// Where the last-level cache would hold all of a lone layer's used experts, they
// lose a little (51 of them: 43.7 / 42.8 / 41.6).
#pragma once

#include <type_traits>

#include "grouped_dma.hpp"
#include "grouped_tile.hpp"

namespace quads {

constexpr int kStreamWaves = 4, kStreamDepth = 3;
constexpr int kStreamRows = 96;                          // 64 weight rows, 32 routed rows
constexpr int kStreamStage = kStreamRows * (128 + 8);    // bytes: chunks, then scales
constexpr int kStreamLoads = kStreamRows / 8 + kStreamRows / 32;  // DMA instructions of a stage

template <int EPI>
__global__ __launch_bounds__(64 * kStreamWaves, 1) void k_grouped_stream(GroupedParams p, int col_groups) {
  constexpr bool PAIR = EPI == kEpiSwiglu || EPI == kEpiSwigluMx;
  constexpr int COLS = PAIR ? 32 : 64;
  __shared__ __attribute__((aligned(128))) uint8_t lds[kStreamWaves * kStreamDepth * kStreamStage];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), half = lane >> 5;
  uint8_t *ring = lds + wave * kStreamDepth * kStreamStage;

  // This wave's items: at .. end - 1.  Workgroups are dealt to the 8 XCDs in
  // turn; neighbouring items share an XCD's L2.
  const uint32_t items = count_tiles<32>(p.offsets, p.E) * static_cast<uint32_t>(col_groups);
  const uint32_t waves = gridDim.x * kStreamWaves;
  const uint32_t index = ((blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3)) * kStreamWaves + wave;
  // items / waves each, and one more for the first of them
  const uint32_t low = items / waves, more = items % waves;
  uint32_t at = index * low + min(index, more);
  const uint32_t end = at + low + (index < more ? 1u : 0u);
  if (at >= end) return;
  uint32_t tile = at / col_groups, group = at % col_groups;
  const TileAt t0 = find_tile<32>(p.offsets, p.E, static_cast<int>(tile));
  Walker walk(p.offsets, t0);

  struct Item {
    int32_t r0, rows, n0;
  };
  Item load{t0.r0, t0.rows, 0};

  // Sources of the item that is being staged.  Lane 8 r + s of a staging
  // instruction brings the chunk of slot s of row r of its eight; row r of the
  // stage keeps chunk c in slot c ^ (r / 2 % 8).
  const uint8_t *zero = reinterpret_cast<const uint8_t *>(g_zero_chunk);
  const int lr = lane >> 3;
  const int chunk0 = (lane & 7) ^ (lr >> 1);  // of rows 16 k ..; rows 16 k + 8 ..: ^ 4
  const uint8_t *wsrc, *wscale, *xsrc[4], *xscale;
  int64_t second, second_scale;  // from the first 32 weight rows to the other 32
  const auto aim_rows = [&] {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t src = source_row(p, load.r0 + min(8 * j + lr, load.rows - 1));
      xsrc[j] = p.x + src * p.x_row + 16 * (chunk0 ^ (4 * (j & 1)));
    }
    xscale = p.x_scales + source_row(p, load.r0 + min(lane >> 1, load.rows - 1)) * p.chunks + 4 * (lane & 1);
  };
  const auto aim_columns = [&] {
    load.n0 = static_cast<int32_t>(group) * COLS;
    const int32_t other = PAIR ? p.width : load.n0 + 32 < p.width ? 32 : 0;
    const int64_t row = static_cast<int64_t>(walk.e) * p.N + load.n0;
    wsrc = p.w + (row + lr) * p.w_row + 16 * chunk0;
    wscale = p.w_scales + (row + (lane >> 1)) * p.chunks + 4 * (lane & 1);
    second = other * p.w_row;
    second_scale = static_cast<int64_t>(other) * p.chunks;
  };
  const auto fetch = [&](int s, uint8_t *base) {
    const int64_t off = 128 * static_cast<int64_t>(s);
    const bool in0 = 8 * s + chunk0 < p.chunks, in1 = 8 * s + (chunk0 ^ 4) < p.chunks;
    const bool sin = 8 * s + 4 * (lane & 1) < p.chunks;
    const auto weights = [&](auto once) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint8_t *src = wsrc + (j >= 4 ? second : 0) + 8 * (j & 3) * p.w_row + off;
        if (j & 1)  // the swizzle of rows 16 k + 8 ..
          src = in1 ? src + ((chunk0 ^ 4) - chunk0) * 16 : zero;
        else
          src = in0 ? src : zero;
        if constexpr (decltype(once)::value)
          dma_wave_once(src, base + 1024 * j);
        else
          dma_wave(src, base + 1024 * j, 16);
      }
    };
    if (walk.last - walk.first <= 32)  // the expert's only row tile
      weights(std::true_type{});
    else
      weights(std::false_type{});
#pragma unroll
    for (int j = 0; j < 4; ++j) dma_wave((j & 1 ? in1 : in0) ? xsrc[j] + off : zero, base + 1024 * (8 + j), 16);
    uint8_t *sc = base + kStreamRows * 128;
    dma_wave(sin ? wscale + 8 * s : zero, sc, 4);
    dma_wave(sin ? wscale + second_scale + 8 * s : zero, sc + 256, 4);
    dma_wave(sin ? xscale + 8 * s : zero, sc + 512, 4);
  };

  const int stages = (p.chunks + 7) / 8;
  int ls = 0;          // stage of the next fetch
  bool any = true;     // there is something left to fetch
  const auto next_fetch = [&](uint8_t *base) {
    // Behind the last item its first stage is fetched again: the count of
    // loads in flight stays the same.
    fetch(any ? ls : 0, base);
    if (!any || ++ls < stages) return;
    ls = 0;
    if (++at == end) {
      any = false;
      return;
    }
    if (++group == static_cast<uint32_t>(col_groups)) {
      group = 0;
      walk.to<32>(static_cast<int32_t>(++tile), load.r0, load.rows);
      aim_rows();
    }
    aim_columns();
  };

  const int fr = lane & 31;
  f32x16 acc = {}, acc2 = {};
  aim_rows();
  aim_columns();
  // What is being multiplied follows what is being fetched by its own walk.
  uint32_t mtile = tile, mgroup = group, left = end - at;
  Walker mwalk(p.offsets, t0);
  Item mul{t0.r0, t0.rows, load.n0};
#pragma unroll
  for (int d = 0; d < kStreamDepth; ++d) next_fetch(ring + d * kStreamStage);
  uint8_t *cur = ring;
  int s = 0;
  while (true) {
    wait_vm<(kStreamDepth - 1) * kStreamLoads>();
    asm volatile("" ::: "memory");
    uint4 a[4], a2[4], b[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int slot = 16 * ((4 * half + j) ^ ((fr >> 1) & 7));
      a[j] = *reinterpret_cast<const uint4 *>(cur + fr * 128 + slot);
      a2[j] = *reinterpret_cast<const uint4 *>(cur + (32 + fr) * 128 + slot);
      b[j] = *reinterpret_cast<const uint4 *>(cur + (64 + fr) * 128 + slot);
    }
    const uint8_t *sc = cur + kStreamRows * 128 + fr * 8 + 4 * half;
    const uint32_t sa = *reinterpret_cast<const uint32_t *>(sc), sa2 = *reinterpret_cast<const uint32_t *>(sc + 256),
                   sb = *reinterpret_cast<const uint32_t *>(sc + 512);
    wait_lgkm0();  // the stage is in registers: its LDS is free
    next_fetch(cur);
    acc = mfma_mx<0>(a[0], b[0], acc, sa, sb);
    acc2 = mfma_mx<0>(a2[0], b[0], acc2, sa2, sb);
    acc = mfma_mx<1>(a[1], b[1], acc, sa, sb);
    acc2 = mfma_mx<1>(a2[1], b[1], acc2, sa2, sb);
    acc = mfma_mx<2>(a[2], b[2], acc, sa, sb);
    acc2 = mfma_mx<2>(a2[2], b[2], acc2, sa2, sb);
    acc = mfma_mx<3>(a[3], b[3], acc, sa, sb);
    acc2 = mfma_mx<3>(a2[3], b[3], acc2, sa2, sb);
    cur = cur == ring + (kStreamDepth - 1) * kStreamStage ? ring : cur + kStreamStage;
    if (++s < stages) continue;
    const int64_t row = static_cast<int64_t>(mul.r0) + fr;
    store_tile<EPI>(p, acc, acc2, row, fr < mul.rows, mul.n0);
    if constexpr (!PAIR) store_tile<EPI>(p, acc2, acc, row, fr < mul.rows, mul.n0 + 32);
    if (--left == 0) break;
    s = 0;
    acc = f32x16{};
    acc2 = f32x16{};
    if (++mgroup == static_cast<uint32_t>(col_groups)) {
      mgroup = 0;
      mwalk.to<32>(static_cast<int32_t>(++mtile), mul.r0, mul.rows);
    }
    mul.n0 = static_cast<int32_t>(mgroup) * COLS;
  }
  wait_vm<0>();  // nothing of this wave writes LDS after its end
}

// At least this many items, or most of the CUs have too little in flight and
// the split contraction of k_grouped_direct is faster.
constexpr int64_t kStreamItems = 512;

template <int EPI>
int64_t stream_items(const GroupedParams &p, int64_t R) {
  constexpr int COLS = EPI == kEpiSwiglu || EPI == kEpiSwigluMx ? 32 : 64;
  return (R < p.E ? R : p.E) * ((p.width + COLS - 1) / COLS);
}

template <int EPI>
hipError_t launch_stream(const GroupedParams &p, int64_t R, hipStream_t stream) {
  constexpr int COLS = EPI == kEpiSwiglu || EPI == kEpiSwigluMx ? 32 : 64;
  const int groups = (p.width + COLS - 1) / COLS;
  const dim3 grid(256), threads(64 * kStreamWaves);
  hipLaunchKernelGGL((k_grouped_stream<EPI>), grid, threads, 0, stream, p, groups);
  return hipGetLastError();
}

}  // namespace quads
