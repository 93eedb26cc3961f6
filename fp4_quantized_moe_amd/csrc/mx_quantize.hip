// MXFP4 quantize, dequantize and weight QDQ on gfx950.
//
// The scale of a block depends on that block alone, so one pass over the data
// does everything (the NVFP4 quantizer needs the tensor's amax first).  A lane
// holds 8 consecutive elements (one 16-byte bf16 load, two fp32 loads); the
// four lanes of an aligned quad hold one block, and its largest magnitude
// crosses the quad by two DPP quad permutations.  Bound: HBM.  Activations
// read 2 (4) and write 0.53 bytes an element, QDQ reads and writes 2.
#include "launch.hpp"
#include "mx_device.hpp"

namespace quads {
namespace {

constexpr int kThreads = 256;

// Maximum over the aligned quad of lanes (quad_perm [1,0,3,2] and [2,3,0,1]).
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0xB1, 0xF, 0xF, true)));
  return max(v, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0x4E, 0xF, 0xF, true)));
}

__device__ __forceinline__ void store_bf16x8(uint16_t *p, const float (&v)[8]) {
  *reinterpret_cast<uint4 *>(p) =
      make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}

// units = elements / 8; thread t of workgroup b takes units (b * U + j) * 256 + t.
template <bool BF16, bool CODES, bool QDQ, int U>
__global__ __launch_bounds__(kThreads) void k_mx_quantize(const void *x, int64_t units, uint32_t add, uint32_t *codes,
                                                          uint8_t *scales, uint16_t *qdq) {
  const int64_t u0 = static_cast<int64_t>(blockIdx.x) * (U * kThreads) + threadIdx.x;
  float v[U][8];
  uint4 raw[U][BF16 ? 1 : 2];
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const int64_t u = min(u0 + j * kThreads, units - 1);
    const uint4 *src = static_cast<const uint4 *>(x) + u * (BF16 ? 1 : 2);
#pragma unroll
    for (int q = 0; q < (BF16 ? 1 : 2); ++q) raw[j][q] = src[q];
  }
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const int64_t u = u0 + j * kThreads;
    uint32_t a = 0;
    if constexpr (BF16) {
      const uint32_t w[4] = {raw[j][0].x, raw[j][0].y, raw[j][0].z, raw[j][0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[j][2 * i] = __uint_as_float(w[i] << 16);
        v[j][2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    } else {
      const uint32_t w[8] = {raw[j][0].x, raw[j][0].y, raw[j][0].z, raw[j][0].w,
                             raw[j][1].x, raw[j][1].y, raw[j][1].z, raw[j][1].w};
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] = __uint_as_float(w[i]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) a = max(a, __float_as_uint(v[j][i]) & 0x7FFFFFFFu);
    const uint32_t s = mx_scale_byte(quad_max(a), add);
    const float inv = mx_inv_scale(s);
    float t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = v[j][i] * inv;
    uint32_t c = mx_pack8(t);
    if (s == kMxNan) c = 0;
    if (u < units) {
      if constexpr (CODES) {
        codes[u] = c;
        if ((u & 3) == 0) scales[u >> 2] = static_cast<uint8_t>(s);
      }
      if constexpr (QDQ) {
        const float m = mx_scale(s);
        mx_unpack8(c, t);
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] *= m;
        store_bf16x8(qdq + 8 * u, t);
      }
    }
  }
}

template <bool BF16, int U>
__global__ __launch_bounds__(kThreads) void k_mx_dequantize(const uint32_t *codes, const uint8_t *scales,
                                                            int64_t units, void *out) {
  const int64_t u0 = static_cast<int64_t>(blockIdx.x) * (U * kThreads) + threadIdx.x;
  uint32_t c[U], s[U];
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const int64_t u = min(u0 + j * kThreads, units - 1);
    c[j] = codes[u];
    s[j] = scales[u >> 2];
  }
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const int64_t u = u0 + j * kThreads;
    if (u >= units) return;
    float v[8];
    mx_unpack8(c[j], v);
    const float m = mx_scale(s[j]);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= m;
    if constexpr (BF16) {
      store_bf16x8(static_cast<uint16_t *>(out) + 8 * u, v);
    } else {
      float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(out) + 8 * u);
      o[0] = make_float4(v[0], v[1], v[2], v[3]);
      o[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
  }
}

unsigned grid_for(int64_t units, int u) {
  const int64_t per = static_cast<int64_t>(u) * kThreads;
  return static_cast<unsigned>((units + per - 1) / per);
}

template <bool BF16, bool CODES, bool QDQ>
void go(const MxQuantizeLaunch &a, int64_t units, hipStream_t stream) {
  const uint32_t add = a.even ? kMxEvenAdd : 0u;
  hipLaunchKernelGGL((k_mx_quantize<BF16, CODES, QDQ, 1>), dim3(grid_for(units, 1)), dim3(kThreads), 0, stream, a.x,
                     units, add, reinterpret_cast<uint32_t *>(a.codes), a.scales, a.qdq_out);
}

}  // namespace

hipError_t launch_mx_quantize(const MxQuantizeLaunch &a, hipStream_t stream) {
  const int64_t units = a.elems / 8;
  if (units == 0) return hipSuccess;
  if (a.qdq_out) {
    if (a.codes)
      go<true, true, true>(a, units, stream);
    else
      go<true, false, true>(a, units, stream);
  } else if (a.x_bf16) {
    go<true, true, false>(a, units, stream);
  } else {
    go<false, true, false>(a, units, stream);
  }
  return hipGetLastError();
}

hipError_t launch_mx_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t elems, void *out, bool out_bf16,
                                hipStream_t stream) {
  const int64_t units = elems / 8;
  if (units == 0) return hipSuccess;
  const dim3 grid(grid_for(units, 1));
  if (out_bf16)
    hipLaunchKernelGGL((k_mx_dequantize<true, 1>), grid, dim3(kThreads), 0, stream,
                       reinterpret_cast<const uint32_t *>(codes), scales, units, out);
  else
    hipLaunchKernelGGL((k_mx_dequantize<false, 1>), grid, dim3(kThreads), 0, stream,
                       reinterpret_cast<const uint32_t *>(codes), scales, units, out);
  return hipGetLastError();
}

}  // namespace quads
