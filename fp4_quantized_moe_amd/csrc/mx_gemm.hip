// MXFP4 grouped expert GEMM on the scaled matrix instruction of gfx950:
//   Y[i, n] = sum_k W[e(i), n, k] X[t(i), k],  W and X e2m1 * 2^E in blocks of 32.
// v_mfma_scale_f32_32x32x64_f8f6f4 multiplies the codes as stored, scales each
// 32-element block product by 2^(E_w + E_x) and accumulates in fp32.
#include "grouped_staged.hpp"
#include "grouped_stream.hpp"
#include "launch.hpp"

namespace quads {
namespace {

GroupedParams params(const MxGemmLaunch &a) {
  GroupedParams p{};
  p.x = a.x_codes;
  p.x_scales = a.x_scales;
  p.w = a.w_codes;
  p.w_scales = a.w_scales;
  p.row_token = a.row_token;
  p.offsets = a.expert_offsets;
  p.E = a.E;
  p.N = static_cast<int32_t>(a.N);
  p.width = static_cast<int32_t>(a.epi == kEpiF32 || a.epi == kEpiBf16 ? a.N : a.N / 2);
  p.chunks = static_cast<int32_t>(a.K / 32);
  p.x_row = p.w_row = a.K / 2;
  p.w_expert = a.N * (a.K / 2);
  p.y = a.y;
  p.y2 = a.y_scales;
  return p;
}

template <int EPI>
hipError_t run(const MxGemmLaunch &a, hipStream_t stream) {
  const GroupedParams p = params(a);
  // From 32 rows an expert on a weight row meets more than one 32-row tile:
  // staged through LDS.  Scale rows are whole dwords with K % 128 == 0.
  if (a.R > 32 * a.E) {
    if (a.K % 128 == 0) return launch_staged_tiles<kOpMx, EPI>(p, a.R, stream);
    if (a.K > 128) return launch_staged_tiles<kOpMx, EPI, true>(p, a.R, stream);
  }
  if (a.K % 128 == 0 && stream_items<EPI>(p, a.R) >= kStreamItems) return launch_stream<EPI>(p, stream);
  return launch_direct<kOpMx, EPI>(p, a.R, stream);
}

}  // namespace

hipError_t launch_mx_gemm(const MxGemmLaunch &a, hipStream_t stream) {
  if (a.R == 0) return hipSuccess;
  switch (a.epi) {
    case kEpiF32: return run<kEpiF32>(a, stream);
    case kEpiBf16: return run<kEpiBf16>(a, stream);
    case kEpiSwiglu: return run<kEpiSwiglu>(a, stream);
    default: return run<kEpiSwigluMx>(a, stream);
  }
}

}  // namespace quads
