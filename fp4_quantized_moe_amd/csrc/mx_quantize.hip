// MXFP4 quantize, dequantize and weight QDQ on gfx950.
//
// The scale of a block depends on that block alone, so one pass over the data
// does everything (the NVFP4 quantizer needs the tensor's amax first).  A lane
// holds 8 consecutive elements (one 16-byte bf16 load, two fp32 loads); the
// four lanes of an aligned quad hold one block, and its largest magnitude
// crosses the quad by two DPP quad permutations.  Bound: HBM.  Activations
// read 2 (4) and write 0.53 bytes an element, QDQ reads and writes 2.
#include <algorithm>

#include "mx_launch.hpp"
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

// One lane, one unit of 8 elements.  Lanes behind the last unit (a block ends
// with a quad of lanes) load it once more, to take part in the DPP moves.
template <bool BF16, bool CODES, bool QDQ>
__global__ __launch_bounds__(kThreads) void k_mx_quantize(const void *x, int64_t units, uint32_t add, uint32_t *codes,
                                                          uint8_t *scales, uint16_t *qdq) {
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const uint4 *src = static_cast<const uint4 *>(x) + min(unit, units - 1) * (BF16 ? 1 : 2);
  float v[8];
  if constexpr (BF16) {
    const uint4 r = src[0];
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
    const uint4 r0 = src[0], r1 = src[1];
    const uint32_t w[8] = {r0.x, r0.y, r0.z, r0.w, r1.x, r1.y, r1.z, r1.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
  }
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = max(a, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  const uint32_t s = mx_scale_byte(quad_max(a), add);
  const float inv = mx_inv_scale(s);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] *= inv;
  uint32_t c = mx_pack8(v);
  if (s == kMxNan) c = 0;
  if (unit >= units) return;
  if constexpr (CODES) {
    codes[unit] = c;
    if ((unit & 3) == 0) scales[unit >> 2] = static_cast<uint8_t>(s);
  }
  if constexpr (QDQ) {
    const float m = mx_scale(s);
    mx_unpack8(c, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= m;
    store_bf16x8(qdq + 8 * unit, v);
  }
}

template <bool BF16>
__global__ __launch_bounds__(kThreads) void k_mx_dequantize(const uint32_t *codes, const uint8_t *scales,
                                                            int64_t units, void *out) {
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (unit >= units) return;
  float v[8];
  mx_unpack8(codes[unit], v);
  const float m = mx_scale(scales[unit >> 2]);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] *= m;
  if constexpr (BF16) {
    store_bf16x8(static_cast<uint16_t *>(out) + 8 * unit, v);
  } else {
    float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(out) + 8 * unit);
    o[0] = make_float4(v[0], v[1], v[2], v[3]);
    o[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

// Units of one launch: a grid's lanes are counted in 32 bits.
constexpr int64_t kLaunchUnits = int64_t(1) << 31;

dim3 grid_for(int64_t units) { return dim3(static_cast<unsigned>((units + kThreads - 1) / kThreads)); }

template <bool BF16, bool CODES, bool QDQ>
hipError_t go(const MxQuantizeLaunch &a, hipStream_t stream) {
  const uint32_t add = a.even ? kMxEvenAdd : 0u;
  for (int64_t u = 0, units; u < a.elems / 8; u += units) {
    units = std::min(a.elems / 8 - u, kLaunchUnits);
    hipLaunchKernelGGL((k_mx_quantize<BF16, CODES, QDQ>), grid_for(units), dim3(kThreads), 0, stream,
                       static_cast<const uint8_t *>(a.x) + u * (BF16 ? 16 : 32), units, add,
                       CODES ? reinterpret_cast<uint32_t *>(a.codes) + u : nullptr, CODES ? a.scales + u / 4 : nullptr,
                       QDQ ? a.qdq_out + 8 * u : nullptr);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <bool BF16>
hipError_t go_back(const uint8_t *codes, const uint8_t *scales, int64_t elems, void *out, hipStream_t stream) {
  for (int64_t u = 0, units; u < elems / 8; u += units) {
    units = std::min(elems / 8 - u, kLaunchUnits);
    hipLaunchKernelGGL((k_mx_dequantize<BF16>), grid_for(units), dim3(kThreads), 0, stream,
                       reinterpret_cast<const uint32_t *>(codes) + u, scales + u / 4, units,
                       static_cast<uint8_t *>(out) + u * (BF16 ? 16 : 32));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_mx_quantize(const MxQuantizeLaunch &a, hipStream_t stream) {
  if (a.qdq_out) return a.codes ? go<true, true, true>(a, stream) : go<true, false, true>(a, stream);
  return a.x_bf16 ? go<true, true, false>(a, stream) : go<false, true, false>(a, stream);
}

hipError_t launch_mx_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t elems, void *out, bool out_bf16,
                                hipStream_t stream) {
  return out_bf16 ? go_back<true>(codes, scales, elems, out, stream)
                  : go_back<false>(codes, scales, elems, out, stream);
}

}  // namespace quads
