// Host-side launchers of the operators around the experts (norm, gradients of
// the router and of the combine, orthogonalised updates), called by api.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace quads {

constexpr int64_t kLaunchGroups = int64_t(1) << 23;  // of 256 lanes: a grid's lanes are counted in 32 bits

// ---- norm.hip ------------------------------------------------------------------
enum NormQuant { kNormQuantNone = 0, kNormQuantMx4 = 1, kNormQuantMx8 = 2 };

struct NormLaunch {
  int64_t rows;
  int32_t cols;            // a multiple of 16 (32 with a quantized output), at most kNormCols
  bool x_f32, residual_f32, weight_f32;
  NormQuant quant;
  bool even;               // scale rule of kNormQuantMx4
  float eps;
  const void *x, *residual, *weight;  // residual may be null
  void *sum;                          // of the residual's type; null without a residual
  uint16_t *y;                        // or null
  uint8_t *codes, *scales;            // quant only
  float *rstd;                        // or null
};
constexpr int32_t kNormCols = 16384;
hipError_t launch_rms_norm(const NormLaunch &a, hipStream_t stream);

struct NormGradLaunch {
  int64_t rows;
  int32_t cols;
  bool dy_f32, s_f32, weight_f32;
  const void *dy, *s, *weight, *dsum;  // dsum (of s's type) may be null
  const float *rstd;
  void *dx;                            // of s's type
  float *dweight;                      // or null
  float *ws;                           // partial sums, with dweight only
};
size_t norm_grad_ws_bytes(int64_t rows, int32_t cols);
hipError_t launch_rms_norm_grad(const NormGradLaunch &a, hipStream_t stream);

hipError_t launch_mx8_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t elems, void *out, bool out_bf16,
                                 hipStream_t stream);

// ---- route_grad.hip --------------------------------------------------------------
struct BalanceLaunch {
  const float *logits;
  const int32_t *ids;
  const uint8_t *mask;  // or null
  int64_t T;
  int32_t E, top;
  float coef;
  float *loss;      // [1]
  int32_t *counts;  // [E]
  float *slope;     // [E]
  void *ws;
};
size_t balance_ws_bytes(int64_t T, int32_t E);
hipError_t launch_balance(const BalanceLaunch &a, hipStream_t stream);

struct RouteGradLaunch {
  const float *logits;
  const int32_t *ids;
  const uint8_t *mask;  // or null
  const float *dw, *slope, *dloss;  // each or null
  int64_t T;
  int32_t E, top;
  float *dlogits;
};
hipError_t launch_route_grad(const RouteGradLaunch &a, hipStream_t stream);

struct CombineGradLaunch {
  const void *dout, *y;  // y may be null if dw is
  bool dout_bf16, y_bf16;
  const int32_t *inverse;
  const float *w;
  int64_t T, rows;
  int32_t top;
  int64_t N;
  uint16_t *dy;
  float *dw;  // or null
};
hipError_t launch_combine_grad(const CombineGradLaunch &a, hipStream_t stream);

}  // namespace quads
