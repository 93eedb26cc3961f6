// Host-side launcher of the orthogonalised updates, called by api.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace quads {

struct OrthogonalLaunch {
  const void *g;  // [batch, rows, cols]
  bool g_f32;
  int64_t batch, rows, cols;
  int32_t steps;
  float a, b, c, eps;
  uint16_t *out;  // bf16
  void *ws;
};
size_t orthogonalize_ws_bytes(int64_t batch, int64_t rows, int64_t cols);
hipError_t launch_orthogonalize(const OrthogonalLaunch &o, hipStream_t stream);

}  // namespace quads
