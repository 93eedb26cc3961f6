// Grouped GEMM that streams its operands from memory into the MFMA fragments,
// for few rows per expert (decode) and for every size that the staged kernel
// does not take.  Bound: reading the weights once.
//
// An item is 32 routed rows of an expert times two 32-column tiles (the gate
// and up tile of the same columns with the SwiGLU epilogues).  A workgroup's
// four waves split its contraction: wave w takes the stages w, w + 4, ... of
// 128 bytes, so that together they read 512 contiguous bytes of every weight
// row.  In a stage lanes 0-31 take the first 64 bytes of their row and lanes
// 32-63 the second: every line is read whole by four consecutive loads.  The
// partial sums meet in LDS and are added in wave order, by another wave for
// each item in turn.
//
// Workgroups stay (two a CU) and take consecutive items, mostly the columns of
// one row tile.  Each wave has its next stage in flight while it multiplies
// one, across items and their barrier too: what keeps HBM busy.
#pragma once

#include "grouped_dma.hpp"
#include "grouped_tile.hpp"

namespace quads {

constexpr int kSplit = 4;  // waves of a workgroup

// A lane's operands of one stage: four 16-byte chunks of each row, and their
// scales as one dword.
struct DirectStage {
  uint4 a[4], a2[4], b[4];
  uint32_t sa, sa2, sb;
  int shift;  // brings the stage's first scale byte down (a row's last dword may begin before it)
};

// DWORDS: an MXFP4 scale row has at least a dword (K >= 128), read at any byte.
template <int OP, int EPI, bool DWORDS>
__global__ __launch_bounds__(64 * kSplit, 2) void k_grouped_direct(GroupedParams p, int col_groups) {
  constexpr bool PAIR = EPI == kEpiSwiglu || EPI == kEpiSwigluMx;
  constexpr int COLS = PAIR ? 32 : 64;
  __shared__ float partial[2][kSplit][32][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), half = lane >> 5;

  // This workgroup's items: at .. end - 1.  Workgroups are dealt to the 8 XCDs
  // in turn; neighbouring items share an XCD's L2.
  const uint32_t items = count_tiles<32>(p.offsets, p.E) * static_cast<uint32_t>(col_groups);
  const uint32_t per = (items + gridDim.x - 1) / gridDim.x;
  uint32_t at = ((blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3)) * per;
  const uint32_t end = min(items, at + per);
  if (at >= end) return;
  uint32_t tile = at / col_groups, group = at % col_groups;
  const TileAt t0 = find_tile<32>(p.offsets, p.E, static_cast<int>(tile));
  Walker walk(p.offsets, t0);
  int32_t r0 = t0.r0, rows = t0.rows;

  const int stages = (p.chunks + 7) / 8, rounds = (stages + kSplit - 1) / kSplit;

  // Sources of the item that is being loaded.
  const uint8_t *xr, *xs, *wr, *wr2, *ws, *ws2;
  const auto aim_rows = [&] {
    const int64_t src = source_row(p, r0 + min(lane & 31, rows - 1));
    xr = p.x + src * p.x_row;
    xs = p.x_scales + src * p.chunks;
  };
  const auto aim_columns = [&] {
    const int32_t n = static_cast<int32_t>(group) * COLS + (lane & 31);
    const int64_t a = min(n, p.width - 1), b = PAIR ? a + p.width : min(n + 32, p.width - 1);
    const uint8_t *we = p.w + walk.e * p.w_expert;
    wr = we + a * p.w_row;
    wr2 = we + b * p.w_row;
    ws = p.w_scales + (static_cast<int64_t>(walk.e) * p.N + a) * p.chunks;
    ws2 = p.w_scales + (static_cast<int64_t>(walk.e) * p.N + b) * p.chunks;
  };

  // Stage s of the item into r (chunks at and behind `limit`: zeros).
  int32_t limit = p.chunks;
  const uint8_t *zero = reinterpret_cast<const uint8_t *>(g_zero_chunk);
  const auto load = [&](DirectStage &r, int s) {
    const int c0 = 8 * s + 4 * half;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool in = c0 + j < limit;
      const int64_t c = c0 + j;
      r.b[j] = *reinterpret_cast<const uint4 *>(in ? xr + 16 * c : zero);
      r.a[j] = *reinterpret_cast<const uint4 *>(in ? wr + 16 * c : zero);
      r.a2[j] = *reinterpret_cast<const uint4 *>(in ? wr2 + 16 * c : zero);
    }
    if constexpr (OP == kOpMx) {
      if constexpr (DWORDS) {
        const int valid = min(limit - c0, 4);  // scale bytes of this half; behind K: 0 (2^-127)
        const int c = valid >= 4 ? c0 : limit - 4;
        r.shift = 8 * (4 - max(valid, 1));
        __builtin_memcpy(&r.sb, valid > 0 ? xs + c : zero, 4);
        __builtin_memcpy(&r.sa, valid > 0 ? ws + c : zero, 4);
        __builtin_memcpy(&r.sa2, valid > 0 ? ws2 + c : zero, 4);
      } else {
        r.sa = r.sb = r.sa2 = 0;
        r.shift = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bool in = c0 + j < limit;
          r.sb |= static_cast<uint32_t>(*(in ? xs + c0 + j : zero)) << (8 * j);
          r.sa |= static_cast<uint32_t>(*(in ? ws + c0 + j : zero)) << (8 * j);
          r.sa2 |= static_cast<uint32_t>(*(in ? ws2 + c0 + j : zero)) << (8 * j);
        }
      }
    }
  };
  f32x16 acc = {}, acc2 = {};
  const auto multiply = [&](const DirectStage &r) {
    if constexpr (OP == kOpMx) {
      const uint32_t sa = r.sa >> r.shift, sa2 = r.sa2 >> r.shift, sb = r.sb >> r.shift;
      acc = mfma_mx<0>(r.a[0], r.b[0], acc, sa, sb);
      acc2 = mfma_mx<0>(r.a2[0], r.b[0], acc2, sa2, sb);
      acc = mfma_mx<1>(r.a[1], r.b[1], acc, sa, sb);
      acc2 = mfma_mx<1>(r.a2[1], r.b[1], acc2, sa2, sb);
      acc = mfma_mx<2>(r.a[2], r.b[2], acc, sa, sb);
      acc2 = mfma_mx<2>(r.a2[2], r.b[2], acc2, sa2, sb);
      acc = mfma_mx<3>(r.a[3], r.b[3], acc, sa, sb);
      acc2 = mfma_mx<3>(r.a2[3], r.b[3], acc2, sa2, sb);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        acc = mfma_bf16(r.a[j], r.b[j], acc);
        acc2 = mfma_bf16(r.a2[j], r.b[j], acc2);
      }
    }
  };

  int round = 0, count = 0;
  // Multiplies `now`, the stage of this round, with the following one (the
  // next item's first behind the last round) on its way into `next`.  False
  // after the last item.
  const auto step = [&](const DirectStage &now, DirectStage &next) -> bool {
    const bool item_done = round + 1 == rounds;
    const int64_t out_row = static_cast<int64_t>(r0) + (lane & 31);
    const bool row_ok = (lane & 31) < rows;
    const int32_t n0 = static_cast<int32_t>(group) * COLS;
    const bool more = at + 1 < end;
    int s = wave + (round + 1) * kSplit;
    if (item_done) {
      s = wave;
      if (!more) {
        limit = 0;
      } else {
        if (++group == static_cast<uint32_t>(col_groups)) {
          group = 0;
          walk.to<32>(static_cast<int32_t>(++tile), r0, rows);
          aim_rows();
        }
        aim_columns();
      }
    }
    // No branch between these: where paths with different numbers of loads
    // meet, the compiler can only wait for all of them.
    load(next, s);
    __builtin_amdgcn_sched_barrier(0);  // all of it before the products
    multiply(now);
    ++round;
    if (!item_done) return true;
    // Two buffers: one barrier an item suffices, since whoever adds up an
    // item's sums joins the next item's barrier after that.
    float(*sum)[32][64] = partial[count & 1];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      sum[wave][i][lane] = acc[i];
      sum[wave][16 + i][lane] = acc2[i];
    }
    wait_lgkm0();
    barrier_no_fence();
    if (wave == (count & (kSplit - 1))) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        acc[i] = ((sum[0][i][lane] + sum[1][i][lane]) + sum[2][i][lane]) + sum[3][i][lane];
        acc2[i] = ((sum[0][16 + i][lane] + sum[1][16 + i][lane]) + sum[2][16 + i][lane]) + sum[3][16 + i][lane];
      }
      store_tile<EPI>(p, acc, acc2, out_row, row_ok, n0);
      if constexpr (!PAIR) store_tile<EPI>(p, acc2, acc, out_row, row_ok, n0 + 32);
    }
    acc = f32x16{};
    acc2 = f32x16{};
    round = 0;
    ++count;
    ++at;
    return more;
  };

  DirectStage s0, s1;
  aim_rows();
  aim_columns();
  load(s0, wave);
  while (step(s0, s1) && step(s1, s0)) {
  }
}

// Most row tiles of TM rows that R rows in E groups can give.
inline int64_t max_row_tiles(int64_t R, int E, int TM) { return R / TM + (R < E ? R : E); }

template <int OP, int EPI>
hipError_t launch_direct(const GroupedParams &p, int64_t R, hipStream_t stream) {
  constexpr int COLS = EPI == kEpiSwiglu || EPI == kEpiSwigluMx ? 32 : 64;
  const int64_t groups = (p.width + COLS - 1) / COLS;
  const int64_t items = (max_row_tiles(R, p.E, 32) * groups + 7) / 8 * 8;
  if (items > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
  const int64_t grid = items < 512 ? items : 512;  // two workgroups on each of the 256 CUs
  const dim3 blocks(static_cast<unsigned>(grid)), threads(64 * kSplit);
  if (OP == kOpMx && p.chunks < 4)
    hipLaunchKernelGGL((k_grouped_direct<OP, EPI, OP != kOpMx>), blocks, threads, 0, stream, p, static_cast<int>(groups));
  else
    hipLaunchKernelGGL((k_grouped_direct<OP, EPI, true>), blocks, threads, 0, stream, p, static_cast<int>(groups));
  return hipGetLastError();
}

}  // namespace quads
