// Host-side launchers of the MXFP4 and gated kernels, called by api.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace quads {

// ---- mx_quantize.hip ---------------------------------------------------------
struct MxQuantizeLaunch {
  const void *x;
  bool x_bf16, even;
  int64_t elems;      // a multiple of 32; blocks never straddle rows (cols % 32 == 0)
  uint8_t *codes;     // may be null with qdq_out
  uint8_t *scales;
  uint16_t *qdq_out;  // bf16 values, or null (bf16 x only)
};
hipError_t launch_mx_quantize(const MxQuantizeLaunch &a, hipStream_t stream);
hipError_t launch_mx_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t elems, void *out, bool out_bf16,
                                hipStream_t stream);

// Epilogues of the MXFP4 and gated grouped products (grouped_tile.hpp).
enum GroupedEpi {
  kEpiF32 = 0,       // y fp32 [R, N]
  kEpiBf16 = 1,      // y bf16 [R, N]
  kEpiSwiglu = 2,    // h bf16 [R, N/2], optionally the bf16 pre-activations [R, N] too
  kEpiSwigluMx = 3,  // h as MXFP4 codes [R, N/4] and scales [R, N/64]
  kEpiGatedBwd = 4,  // d gate, d up bf16 [R, 2 N] from the accumulated dh and the saved pre-activations
};

// ---- mx_gemm.hip -------------------------------------------------------------
struct MxGemmLaunch {
  int epi;  // kEpiF32 | kEpiBf16 | kEpiSwiglu | kEpiSwigluMx
  int E;
  int64_t R, N, K;
  const uint8_t *x_codes, *x_scales, *w_codes, *w_scales;
  const int32_t *row_token, *expert_offsets;
  void *y;
  void *y_scales;
};
hipError_t launch_mx_gemm(const MxGemmLaunch &a, hipStream_t stream);

// The kernel that launch_mx_gemm takes: the values of QUADS_MX_KERNEL_*.
enum MxKernel { kMxNone = 0, kMxDirect = 1, kMxStream = 2, kMxStagedSmall = 3, kMxStagedLarge = 4 };
MxKernel mx_gemm_kernel(const MxGemmLaunch &a);

// ---- gated.hip ---------------------------------------------------------------
struct GatedLaunch {
  int E;
  int64_t R, hidden, inter;
  const uint16_t *x;  // forward: x [act_rows, hidden]; backward: dy [R, hidden]
  const uint16_t *w;  // forward: [E, 2 inter, hidden]; backward: W_down [E, hidden, inter]
  const int32_t *row_token, *expert_offsets;
  uint16_t *out;       // forward: h [R, inter]; backward: d gate | d up [R, 2 inter]
  uint16_t *pre;       // forward: gate | up [R, 2 inter], or null
  const uint16_t *gu;  // backward: the saved gate | up
};
hipError_t launch_gated_forward(const GatedLaunch &a, hipStream_t stream);
hipError_t launch_gated_backward(const GatedLaunch &a, hipStream_t stream);

}  // namespace quads
