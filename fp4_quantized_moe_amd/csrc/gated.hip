// The gated expert block of the trainer in bf16 on gfx950, with the gradient
// of its activation:
//   forward   [g | u] = W_gate_up x,  h = silu(g) u
//   backward  dh = W_down^T dy,  d u = dh g s,  d g = dh u s (1 + g (1 - s)),  s = sigmoid(g)
// The forward keeps [g | u] in bf16 (288 GB of HBM hold them; recomputing the
// projection would cost twice the backward's own product).  dh exists in the
// accumulators only: the backward's epilogue reads g and u and writes d g, d u.
#include "grouped_staged.hpp"
#include "mx_launch.hpp"

namespace quads {
namespace {

GroupedParams params(const GatedLaunch &a, bool backward) {
  GroupedParams p{};
  p.x = reinterpret_cast<const uint8_t *>(a.x);
  p.w = reinterpret_cast<const uint8_t *>(a.w);
  p.row_token = a.row_token;
  p.offsets = a.expert_offsets;
  p.E = a.E;
  p.width = static_cast<int32_t>(a.inter);
  p.N = backward ? p.width : 2 * p.width;
  p.chunks = static_cast<int32_t>(a.hidden / 8);
  p.x_row = 2 * a.hidden;
  p.w_row = 2 * (backward ? a.inter : a.hidden);
  p.w_expert = 2 * a.hidden * p.N;
  p.y = a.out;
  p.y2 = a.pre;
  p.gu = a.gu;
  return p;
}

}  // namespace

hipError_t launch_gated_forward(const GatedLaunch &a, hipStream_t stream) {
  if (a.R == 0) return hipSuccess;
  const GroupedParams p = params(a, false);
  // The streaming kernel reads an expert's weights once for every 32 rows:
  // it saves the 10 us that a staged tile takes from its first load to its
  // last store while that is little (3 MB once to seven times: 8 us against
  // 11; 67 MB once: 17 against 16).
  const int64_t readings = (a.R + 32 * static_cast<int64_t>(a.E) - 1) / (32 * static_cast<int64_t>(a.E));
  if (static_cast<int64_t>(a.E) * p.w_expert * readings <= (int64_t(16) << 20))
    return launch_direct<kOpBf16, kEpiSwiglu>(p, a.R, stream);
  return launch_staged_tiles<kOpBf16, kEpiSwiglu>(p, a.R, stream);
}

hipError_t launch_gated_backward(const GatedLaunch &a, hipStream_t stream) {
  if (a.R == 0) return hipSuccess;
  return launch_staged_tiles<kOpBf16T, kEpiGatedBwd>(params(a, true), a.R, stream);
}

}  // namespace quads
