// MXFP4 grouped expert GEMM on the scaled matrix instruction of gfx950:
//   Y[i, n] = sum_k W[e(i), n, k] X[t(i), k],  W and X e2m1 * 2^E in blocks of 32.
// v_mfma_scale_f32_32x32x64_f8f6f4 multiplies the codes as stored, scales each
// 32-element block product by 2^(E_w + E_x) and accumulates in fp32.
#include "grouped_staged.hpp"
#include "grouped_stream.hpp"
#include "mx_launch.hpp"

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
MxKernel choose(const MxGemmLaunch &a, const GroupedParams &p) {
  if (a.R == 0) return kMxNone;
  // The streaming kernels read an expert's weights once for every 32 rows.
  // One reading is what the call costs anyway (decode); two or three still
  // pay while they are short beside the 12 us that a staged tile takes from
  // its first load to its last store.  Measured, streamed against staged:
  // 17 MB twice 12.4 and 15.2 us, 34 MB twice 12.9 and 13.2, 17 MB four times
  // 16.5 and 12.8, 268 MB twice 95 and 65.  Rows that do not begin on a line
  // (K % 128 != 0) stream worse: 8 MB five times 21 and 13.
  // The readings are an average: the host does not know the experts' rows, and
  // a skewed routing reads a loud expert's weights more often.
  const int64_t readings = (a.R + 32 * static_cast<int64_t>(a.E) - 1) / (32 * static_cast<int64_t>(a.E));
  const int64_t bytes = static_cast<int64_t>(a.E) * a.N * (a.K / 2) * readings;
  if (readings > 1 && bytes > (int64_t(a.K % 128 ? 16 : 48) << 20) && a.K >= 128)
    return staged_large<EPI>(p, a.R) ? kMxStagedLarge : kMxStagedSmall;
  return a.K % 128 == 0 && stream_items<EPI>(p, a.R) >= kStreamItems ? kMxStream : kMxDirect;
}

template <int EPI>
hipError_t run(const MxGemmLaunch &a, hipStream_t stream) {
  const GroupedParams p = params(a);
  switch (choose<EPI>(a, p)) {
    case kMxNone: return hipSuccess;
    case kMxDirect: return launch_direct<kOpMx, EPI>(p, a.R, stream);
    case kMxStream: return launch_stream<EPI>(p, a.R, stream);
    default: break;
  }
  // Scale rows are whole dwords with K % 128 == 0.
  if (a.K % 128 == 0) return launch_staged_tiles<kOpMx, EPI>(p, a.R, stream);
  return launch_staged_tiles<kOpMx, EPI, true>(p, a.R, stream);
}

}  // namespace

hipError_t launch_mx_gemm(const MxGemmLaunch &a, hipStream_t stream) {
  switch (a.epi) {
    case kEpiF32: return run<kEpiF32>(a, stream);
    case kEpiBf16: return run<kEpiBf16>(a, stream);
    case kEpiSwiglu: return run<kEpiSwiglu>(a, stream);
    default: return run<kEpiSwigluMx>(a, stream);
  }
}

MxKernel mx_gemm_kernel(const MxGemmLaunch &a) {
  switch (a.epi) {
    case kEpiF32: return choose<kEpiF32>(a, params(a));
    case kEpiBf16: return choose<kEpiBf16>(a, params(a));
    case kEpiSwiglu: return choose<kEpiSwiglu>(a, params(a));
    default: return choose<kEpiSwigluMx>(a, params(a));
  }
}

}  // namespace quads
