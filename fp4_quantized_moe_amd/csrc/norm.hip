// Root-mean-square norm with the residual's addition, and its gradient.
//
//   s = x + residual (rounded to the stream's type and kept),
//   r = (mean(s^2) + eps)^(-1/2),  y = s r w,
// y leaves as bf16, as MXFP4 or MXFP8 (each rounded once from the fp32 y), or
// as bf16 and one of them.  Gradient, with n = s r, d = dy w:
//   dx = r (d - n mean(d n)) + dsum,  dw = sum over rows of dy n.
//
// Bound: HBM.  A row stays in registers between its sum and its outputs, so
// every element is read and written once.  A lane holds units of 8 consecutive
// elements (16 bytes of bf16); the four lanes of an aligned quad hold a block
// of 32, whose largest magnitude crosses the quad by two DPP permutations.
// Measured: 16384 x 2048 (fp32 added to a bf16 stream, out in bf16 and MXFP8,
// 370 MB) 67 us, 5.5 TB/s; the gradient of 8192 x 2048 (168 MB) 26 us and 4 for
// the fold of dw; MXFP8 back to bf16 (102 MB) 16.5 us, 6.2 TB/s.  256 rows of
// 2048 take 3.6 us, a launch and two trips to memory.
#include <algorithm>

#include "layer_launch.hpp"
#include "mx_device.hpp"
#include "quads_device.hpp"

namespace quads {
namespace {

// Sum over the wave in a fixed order, in all lanes.
__device__ __forceinline__ float wave_sum(float v) {
  const auto step = [&](auto ctrl, auto mask) {
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), decltype(ctrl)::value, decltype(mask)::value, 0xf, false));
  };
  step(std::integral_constant<int, 0x111>{}, std::integral_constant<int, 0xf>{});
  step(std::integral_constant<int, 0x112>{}, std::integral_constant<int, 0xf>{});
  step(std::integral_constant<int, 0x114>{}, std::integral_constant<int, 0xf>{});
  step(std::integral_constant<int, 0x118>{}, std::integral_constant<int, 0xf>{});
  step(std::integral_constant<int, 0x142>{}, std::integral_constant<int, 0xa>{});
  step(std::integral_constant<int, 0x143>{}, std::integral_constant<int, 0xc>{});
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

// Sum over the TPR lanes of a row, in all of them: 16 (row rotations by 8, 4, 2
// and 1), a wave, or several of a workgroup's (`parts`: their meeting place; a
// barrier).
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float *parts) {
  if constexpr (TPR == 16) {
    const auto step = [&](auto ctrl) {
      v += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), decltype(ctrl)::value, 0xf, 0xf, true));
    };
    step(std::integral_constant<int, 0x128>{});
    step(std::integral_constant<int, 0x124>{});
    step(std::integral_constant<int, 0x122>{});
    step(std::integral_constant<int, 0x121>{});
    return v;
  }
  v = wave_sum(v);
  if constexpr (TPR <= 64) return v;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (lane == 0) parts[wave] = v;
  __syncthreads();
  const float4 *row = reinterpret_cast<const float4 *>(parts + (wave & ~(TPR / 64 - 1)));
  v = 0.0f;
#pragma unroll
  for (int i = 0; i < TPR / 256; ++i) {
    const float4 p = row[i];
    v = (((v + p.x) + p.y) + p.z) + p.w;
  }
  return v;
}

// A unit of 8 values as loaded: bf16 fills `lo` alone.
struct Raw {
  uint4 lo, hi;
};

__device__ __forceinline__ Raw load_unit(const void *p, int64_t unit, bool f32) {
  Raw r;
  if (f32) {
    const uint4 *q = static_cast<const uint4 *>(p) + 2 * unit;
    r.lo = q[0];
    r.hi = q[1];
  } else {
    r.lo = static_cast<const uint4 *>(p)[unit];
    r.hi = r.lo;
  }
  return r;
}

__device__ __forceinline__ void unpack(const Raw &r, bool f32, float (&v)[8]) {
  const uint32_t lo[4] = {r.lo.x, r.lo.y, r.lo.z, r.lo.w}, hi[4] = {r.hi.x, r.hi.y, r.hi.z, r.hi.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (f32) {
      v[i] = __uint_as_float(lo[i]);
      v[4 + i] = __uint_as_float(hi[i]);
    } else {
      v[2 * i] = __uint_as_float(lo[i] << 16);
      v[2 * i + 1] = __uint_as_float(lo[i] & 0xFFFF0000u);
    }
  }
}

__device__ __forceinline__ uint4 pack_unit(const float (&v)[8]) {
  return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}

__device__ __forceinline__ void store_unit(void *p, int64_t unit, bool f32, const float (&v)[8]) {
  if (f32) {
    float4 *q = static_cast<float4 *>(p) + 2 * unit;
    q[0] = make_float4(v[0], v[1], v[2], v[3]);
    q[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    static_cast<uint4 *>(p)[unit] = pack_unit(v);
  }
}

struct NormParams {
  int64_t rows, base;  // a launch has the rows from base on
  int32_t units;  // of 8 columns
  float cols, eps;
  uint32_t add;  // MXFP4's scale rule
  bool x_f32, residual_f32, weight_f32;
  const void *x, *residual, *weight;
  void *sum;
  uint16_t *y;
  uint8_t *codes, *scales;
  float *rstd;
};

// TPR lanes a row, V units a lane.
template <int TPR>
constexpr int kNormThreads = TPR < 256 ? 256 : TPR;
template <int QUANT, int TPR, int V>
__global__ __launch_bounds__(kNormThreads<TPR>) void k_rms_norm(NormParams p) {
  __shared__ __attribute__((aligned(16))) float parts[16];
  constexpr int ROWS = kNormThreads<TPR> / TPR;
  const int t = ROWS == 1 ? threadIdx.x : threadIdx.x % TPR;
  const int64_t row = p.base + static_cast<int64_t>(blockIdx.x) * ROWS + (ROWS == 1 ? 0 : threadIdx.x / TPR);  // uniform if one
  if (TPR < 256 && row >= p.rows) return;  // all lanes of a row, and no barrier
  const int64_t first = row * p.units;

  Raw x[V], res[V], w[V];
#pragma unroll
  for (int v = 0; v < V; ++v) x[v] = load_unit(p.x, first + min(t + v * TPR, p.units - 1), p.x_f32);
  if (p.residual) {
#pragma unroll
    for (int v = 0; v < V; ++v) res[v] = load_unit(p.residual, first + min(t + v * TPR, p.units - 1), p.residual_f32);
  }
#pragma unroll
  for (int v = 0; v < V; ++v) w[v] = load_unit(p.weight, min(t + v * TPR, p.units - 1), p.weight_f32);

  float s[V][8], ss = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int unit = t + v * TPR;
    unpack(x[v], p.x_f32, s[v]);
    if (p.residual) {
      float r[8];
      unpack(res[v], p.residual_f32, r);
#pragma unroll
      for (int i = 0; i < 8; ++i) s[v][i] = s[v][i] + r[i];
      if (!p.residual_f32) {  // what is normalised is the stream as it is kept
        const uint4 k = pack_unit(s[v]);
        if (unit < p.units) static_cast<uint4 *>(p.sum)[first + unit] = k;
        unpack(Raw{k, k}, false, s[v]);
      } else if (unit < p.units) {
        store_unit(p.sum, first + unit, true, s[v]);
      }
    }
    if (unit < p.units) {
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = __builtin_fmaf(s[v][i], s[v][i], ss);
    }
  }
  const float r = 1.0f / sqrtf(row_sum<TPR>(ss, parts) / p.cols + p.eps);
  if (p.rstd && t == 0) p.rstd[row] = r;

#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int unit = t + v * TPR;
    float y[8], g[8];
    unpack(w[v], p.weight_f32, g);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = s[v][i] * r * g[i];
    if (p.y && unit < p.units) static_cast<uint4 *>(static_cast<void *>(p.y))[first + unit] = pack_unit(y);
    if constexpr (QUANT != kNormQuantNone) {
      uint32_t a = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) a = max(a, __float_as_uint(y[i]) & 0x7FFFFFFFu);
      a = quad_max(a);  // quads lie inside the row or behind it: cols % 32 == 0
      const uint32_t b = QUANT == kNormQuantMx4 ? mx_scale_byte(a, p.add) : mx8_scale_byte(a);
      const float inv = mx_inv_scale(b);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] *= inv;
      if (unit < p.units) {
        if constexpr (QUANT == kNormQuantMx4) {
          const uint32_t c = mx_pack8(y);
          reinterpret_cast<uint32_t *>(p.codes)[first + unit] = b == kMxNan ? 0u : c;
        } else {
          const uint2 c = mx8_pack8(y);
          reinterpret_cast<uint2 *>(p.codes)[first + unit] = b == kMxNan ? make_uint2(0, 0) : c;
        }
        if ((t & 3) == 0) p.scales[(first + unit) >> 2] = static_cast<uint8_t>(b);
      }
    }
  }
}

template <int QUANT, int TPR, int V>
hipError_t run_norm(NormParams p, hipStream_t stream) {
  constexpr int64_t ROWS = kNormThreads<TPR> / TPR;  // of a workgroup
  constexpr int64_t GROUPS = kLaunchGroups * 256 / kNormThreads<TPR>;
  for (p.base = 0; p.base < p.rows; p.base += GROUPS * ROWS) {
    const int64_t groups = std::min((p.rows - p.base + ROWS - 1) / ROWS, GROUPS);
    hipLaunchKernelGGL((k_rms_norm<QUANT, TPR, V>), dim3(static_cast<unsigned>(groups)), dim3(kNormThreads<TPR>), 0, stream, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// Lanes of a row: the fewest that leave a lane at most two units, so that many
// rows are under way (8192 x 16384 to bf16 by 256 lanes of eight units 168 us,
// by 1024 of two 102; 8192 x 8192 52 and 44), and 16 for the shortest (65536 x
// 128 17 -> 7.7 us with them).  A wave a row only where there are rows to fill
// the card (a bf16 stream to bf16 and MXFP8: 2048 x 1024 5.3 us by a wave, 5.9 by
// 256 lanes, 4096 x 1024 8.2 and 9.5, but 1024 x 1024 4.4 and 4.15, 256 x 1024
// 3.8 and 3.0; up to 512 columns the wave is ahead with fewer rows too, 1024 x
// 512 3.0 and 3.8, 256 x 512 2.8 and 2.9, which the rule leaves), and not with
// four units a lane (16384 x 2048 to bf16 and MXFP8 80 us; four waves 67).
template <int QUANT>
hipError_t run_norm(const NormParams &p, hipStream_t stream) {
  if (p.units <= 16) return run_norm<QUANT, 16, 1>(p, stream);
  if (p.units <= 64 && p.rows >= 2048) return run_norm<QUANT, 64, 1>(p, stream);
  if (p.units <= 128 && p.rows >= 2048) return run_norm<QUANT, 64, 2>(p, stream);
  if (p.units <= 256) return run_norm<QUANT, 256, 1>(p, stream);
  if (p.units <= 512) return run_norm<QUANT, 256, 2>(p, stream);
  if (p.units <= 1024) return run_norm<QUANT, 512, 2>(p, stream);
  return run_norm<QUANT, 1024, 2>(p, stream);
}

// ---- gradient --------------------------------------------------------------------

struct NormGradParams {
  int64_t rows;
  int32_t units;
  float cols;
  bool weight_f32;
  const void *dy, *s, *weight, *dsum;
  const float *rstd;
  void *dx;
  float *partial;      // [row workgroups, cols] sums of dy n, or null
  float *dweight;      // with column workgroups
  int32_t col_groups;  // the first workgroups of the grid have columns of dweight, the others rows
};

constexpr int kGradThreads = 512, kColUnits = 4;

// 32 columns of dweight from all rows: 128 rows at once, four such loads under way.
template <bool DY32, bool S32>
__device__ __forceinline__ void weight_columns(const NormGradParams &p, int block) {
  constexpr int SLOTS = kGradThreads / kColUnits, AHEAD = 4;
  __shared__ float meet[kGradThreads / 64][kColUnits * 8];
  const int t = threadIdx.x, slot = t / kColUnits, unit = block * kColUnits + t % kColUnits, at = min(unit, p.units - 1);
  float acc[8] = {};
  for (int64_t base = slot; base < p.rows; base += AHEAD * SLOTS) {
    Raw s[AHEAD], dy[AHEAD];
    float r[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const int64_t row = min(base + k * SLOTS, p.rows - 1);
      s[k] = load_unit(p.s, row * p.units + at, S32);
      dy[k] = load_unit(p.dy, row * p.units + at, DY32);
      r[k] = p.rstd[row];
    }
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      float n[8], d[8];
      unpack(s[k], S32, n);
      unpack(dy[k], DY32, d);
      if (base + k * SLOTS < p.rows) {
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = __builtin_fmaf(d[i], n[i] * r[k], acc[i]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
#pragma unroll
    for (int off = kColUnits; off < 64; off *= 2) acc[i] += __shfl_xor(acc[i], off);
    if ((t & 63) < kColUnits) meet[t >> 6][t % kColUnits * 8 + i] = acc[i];
  }
  __syncthreads();
  if (t < kColUnits * 8 && block * kColUnits + t / 8 < p.units) {
    float sum = meet[0][t];
    for (int w = 1; w < kGradThreads / 64; ++w) sum += meet[w][t];
    p.dweight[block * kColUnits * 8 + t] = sum;
  }
}

// Workgroups behind those of dweight's columns.  512 / TPR rows of one at once; workgroups stay and take rows in turn,
// their columns' weights and sums of dy n in registers.  Few units a lane, so
// that two workgroups fit a CU: with a wave a row (8192 x 2048: four units a
// lane, 256 registers) the kernel took 45 us.
template <bool DY32, bool S32, int TPR, int V>
__global__ __launch_bounds__(kGradThreads) void k_rms_norm_grad(NormGradParams p) {
  constexpr int ROWS = kGradThreads / TPR;
  const int block = static_cast<int>(blockIdx.x) - p.col_groups, blocks = static_cast<int>(gridDim.x) - p.col_groups;
  if (block < 0) {
    weight_columns<DY32, S32>(p, blockIdx.x);
    return;
  }
  __shared__ __attribute__((aligned(16))) float parts[2][8];
  __shared__ __attribute__((aligned(16))) float meet[ROWS > 1 ? (ROWS - 1) * TPR * 8 : 1];
  const int t = threadIdx.x % TPR, slot = threadIdx.x / TPR;
  float acc[V][8] = {}, w[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v) unpack(load_unit(p.weight, min(t + v * TPR, p.units - 1), p.weight_f32), p.weight_f32, w[v]);
  int turn = 0;
  // Every wave makes the same number of rounds: the rows' sums contain a barrier.
  for (int64_t base = static_cast<int64_t>(block) * ROWS; base < p.rows; base += static_cast<int64_t>(blocks) * ROWS) {
    const bool live = base + slot < p.rows;
    const int64_t row = live ? base + slot : p.rows - 1, first = row * p.units;
    Raw s[V], dy[V], ds[V];
#pragma unroll
    for (int v = 0; v < V; ++v) s[v] = load_unit(p.s, first + min(t + v * TPR, p.units - 1), S32);
#pragma unroll
    for (int v = 0; v < V; ++v) dy[v] = load_unit(p.dy, first + min(t + v * TPR, p.units - 1), DY32);
    if (p.dsum) {
#pragma unroll
      for (int v = 0; v < V; ++v) ds[v] = load_unit(p.dsum, first + min(t + v * TPR, p.units - 1), S32);
    }
    const float r = p.rstd[row];
    float n[V][8], d[V][8], dot = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      unpack(s[v], S32, n[v]);
      unpack(dy[v], DY32, d[v]);
      const bool in = live && t + v * TPR < p.units;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        n[v][i] *= r;
        if (in) acc[v][i] = __builtin_fmaf(d[v][i], n[v][i], acc[v][i]);
        d[v][i] *= w[v][i];
        if (in) dot = __builtin_fmaf(d[v][i], n[v][i], dot);
      }
    }
    const float mean = row_sum<TPR>(dot, parts[turn]) / p.cols;
    turn ^= 1;  // a wave is at most one barrier ahead: the next row's sums go elsewhere
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (!live || t + v * TPR >= p.units) continue;
      float dx[8], e[8];
      if (p.dsum) unpack(ds[v], S32, e);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        dx[i] = r * (d[v][i] - n[v][i] * mean);
        if (p.dsum) dx[i] += e[i];
      }
      store_unit(p.dx, first + t + v * TPR, S32, dx);
    }
  }
  if (p.partial == nullptr) return;
  // The workgroup's rows meet unit by unit, in the slots' order.
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (v * TPR >= p.units) break;
    if constexpr (ROWS > 1) {
      __syncthreads();
      if (slot > 0) {
        float4 *m = reinterpret_cast<float4 *>(meet) + (slot - 1) * TPR * 2 + t;
        m[0] = make_float4(acc[v][0], acc[v][1], acc[v][2], acc[v][3]);
        m[TPR] = make_float4(acc[v][4], acc[v][5], acc[v][6], acc[v][7]);
      }
      __syncthreads();
    }
    if (slot == 0 && t + v * TPR < p.units) {
      for (int k = 0; k < ROWS - 1; ++k) {
        const float4 *m = reinterpret_cast<const float4 *>(meet) + k * TPR * 2 + t;
        const float4 a = m[0], b = m[TPR];
        acc[v][0] += a.x;
        acc[v][1] += a.y;
        acc[v][2] += a.z;
        acc[v][3] += a.w;
        acc[v][4] += b.x;
        acc[v][5] += b.y;
        acc[v][6] += b.z;
        acc[v][7] += b.w;
      }
      store_unit(p.partial, static_cast<int64_t>(block) * p.units + t + v * TPR, true, acc[v]);
    }
  }
}

// dweight = sum of the partial sums in order: 16 columns a workgroup, 64 parts.
constexpr int kFoldCols = 16;
__global__ __launch_bounds__(256) void k_fold_columns(const float *partial, int parts, int32_t cols, float *out) {
  __shared__ __attribute__((aligned(16))) float4 meet[64][4];
  const int c4 = threadIdx.x & 3, part = threadIdx.x >> 2;
  const int32_t col = blockIdx.x * kFoldCols + 4 * c4;  // cols % 16 == 0
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  const auto add = [&](const float4 &b) {
    a.x += b.x;
    a.y += b.y;
    a.z += b.z;
    a.w += b.w;
  };
#pragma unroll 8
  for (int k = part; k < parts; k += 64) add(*reinterpret_cast<const float4 *>(partial + static_cast<int64_t>(k) * cols + col));
  meet[part][c4] = a;
  __syncthreads();
  if (part == 0) {
    for (int k = 1; k < 64; ++k) add(meet[k][c4]);
    *reinterpret_cast<float4 *>(out + col) = a;
  }
}

// As the forward's lanes, but no 1024 (which spills; of 16384 columns 16 rows
// 8.4 us, so 9.6, 8192 rows 225 and 221).
int grad_lanes(int64_t rows, int32_t units) {
  return units <= 16 ? 16 : units <= 128 && rows >= 2048 ? 64 : units <= 512 ? 256 : 512;
}

int grad_groups(int64_t rows, int32_t units) {
  const int64_t per = kGradThreads / grad_lanes(rows, units);
  return static_cast<int>(std::min<int64_t>((rows + per - 1) / per, 512));
}

// dweight by workgroups of its own in the same launch, which read dy and s a
// second time: few rows (333 x 656 in a graph 6.9 -> 3.9 us, 1024 x 2048 10.8 ->
// 5.9, 1024 x 8192 28.8 -> 23.9; but 2047 x 2048 12.3 -> 15.0).
bool weight_by_columns(int64_t rows) { return rows <= 1024; }

template <bool DY32, bool S32>
void run_norm_grad(const NormGradParams &p, int groups, hipStream_t stream) {
  const int lanes = grad_lanes(p.rows, p.units), per = (p.units + lanes - 1) / lanes;
  const auto go = [&](auto tpr, auto v) {
    hipLaunchKernelGGL((k_rms_norm_grad<DY32, S32, decltype(tpr)::value, decltype(v)::value>), dim3(groups), dim3(kGradThreads),
                       0, stream, p);
  };
  const std::integral_constant<int, 1> one;
  const std::integral_constant<int, 2> two;
  if (lanes == 16) go(std::integral_constant<int, 16>{}, one);
  else if (lanes == 64 && per <= 1) go(std::integral_constant<int, 64>{}, one);
  else if (lanes == 64) go(std::integral_constant<int, 64>{}, two);
  else if (lanes == 256 && per <= 1) go(std::integral_constant<int, 256>{}, one);
  else if (lanes == 256) go(std::integral_constant<int, 256>{}, two);
  else if (per <= 2) go(std::integral_constant<int, 512>{}, two);
  else go(std::integral_constant<int, 512>{}, std::integral_constant<int, 4>{});
}

// ---- MXFP8 back to values ----------------------------------------------------------

template <bool BF16>
__global__ __launch_bounds__(256) void k_mx8_dequantize(const uint2 *codes, const uint8_t *scales, int64_t units, void *out) {
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (unit >= units) return;
  float v[8];
  mx8_unpack8(codes[unit], v);
  const float m = mx_scale(scales[unit >> 2]);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] *= m;
  store_unit(out, unit, !BF16, v);
}

}  // namespace

hipError_t launch_rms_norm(const NormLaunch &a, hipStream_t stream) {
  NormParams p{};
  p.rows = a.rows;
  p.units = a.cols / 8;
  p.cols = static_cast<float>(a.cols);
  p.eps = a.eps;
  p.add = a.even ? kMxEvenAdd : 0u;
  p.x_f32 = a.x_f32;
  p.residual_f32 = a.residual_f32;
  p.weight_f32 = a.weight_f32;
  p.x = a.x;
  p.residual = a.residual;
  p.weight = a.weight;
  p.sum = a.sum;
  p.y = a.y;
  p.codes = a.codes;
  p.scales = a.scales;
  p.rstd = a.rstd;
  switch (a.quant) {
    case kNormQuantNone: return run_norm<kNormQuantNone>(p, stream);
    case kNormQuantMx4: return run_norm<kNormQuantMx4>(p, stream);
    default: return run_norm<kNormQuantMx8>(p, stream);
  }
}

size_t norm_grad_ws_bytes(int64_t rows, int32_t cols) {
  if (weight_by_columns(rows)) return 0;
  return static_cast<size_t>(grad_groups(rows, cols / 8)) * cols * sizeof(float);
}

hipError_t launch_rms_norm_grad(const NormGradLaunch &a, hipStream_t stream) {
  NormGradParams p{};
  p.rows = a.rows;
  p.units = a.cols / 8;
  p.cols = static_cast<float>(a.cols);
  p.weight_f32 = a.weight_f32;
  p.dy = a.dy;
  p.s = a.s;
  p.weight = a.weight;
  p.dsum = a.dsum;
  p.rstd = a.rstd;
  p.dx = a.dx;
  const int groups = grad_groups(a.rows, p.units);
  const auto run = [&](int grid) {
    if (a.dy_f32 && a.s_f32) run_norm_grad<true, true>(p, grid, stream);
    else if (a.dy_f32) run_norm_grad<true, false>(p, grid, stream);
    else if (a.s_f32) run_norm_grad<false, true>(p, grid, stream);
    else run_norm_grad<false, false>(p, grid, stream);
    return hipGetLastError();
  };
  if (a.dweight && weight_by_columns(a.rows)) {
    p.dweight = a.dweight;
    p.col_groups = (p.units + kColUnits - 1) / kColUnits;
    if (a.dx != a.dy && a.dx != a.s) return run(p.col_groups + groups);
    const hipError_t e = run(p.col_groups);  // before dx takes the place of what they read
    if (e != hipSuccess || groups == 0) return e;
    p.col_groups = 0;
    return run(groups);
  }
  p.partial = a.dweight ? a.ws : nullptr;
  if (groups > 0) {
    const hipError_t e = run(groups);
    if (e != hipSuccess) return e;
  }
  if (a.dweight)
    hipLaunchKernelGGL(k_fold_columns, dim3(a.cols / kFoldCols), dim3(256), 0, stream, a.ws, groups, a.cols, a.dweight);
  return hipGetLastError();
}

hipError_t launch_mx8_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t elems, void *out, bool out_bf16,
                                 hipStream_t stream) {
  constexpr int64_t kLaunchUnits = int64_t(1) << 31;  // a grid's lanes are counted in 32 bits
  for (int64_t u = 0, units; u < elems / 8; u += units) {
    units = std::min(elems / 8 - u, kLaunchUnits);
    const dim3 grid(static_cast<unsigned>((units + 255) / 256));
    const uint2 *c = reinterpret_cast<const uint2 *>(codes) + u;
    uint8_t *o = static_cast<uint8_t *>(out) + u * (out_bf16 ? 16 : 32);
    if (out_bf16) hipLaunchKernelGGL((k_mx8_dequantize<true>), grid, dim3(256), 0, stream, c, scales + u / 4, units, o);
    else hipLaunchKernelGGL((k_mx8_dequantize<false>), grid, dim3(256), 0, stream, c, scales + u / 4, units, o);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace quads
