// What the router and the combine need for training.
//
//   k_balance       per-expert counts over the valid tokens and the balance loss
//                     L = coef E sum_e (c_e / (top n)) (1/n sum_t p_te),  p = softmax(logits)
//                   with its slope dL/dp_te = coef E c_e / (top n^2), the same
//                   for all valid tokens (the counts are constants)
//   k_route_grad    gradient of the logits from dp = dloss slope + the combine
//                   weights' gradient at the chosen experts:
//                     dl = p (dp - sum_e p dp)
//   k_combine_grad  dy[inverse[t, j]] = w_tj dout_t,  dw_tj = <dout_t, y[inverse[t, j]]>
//
// Bound: HBM where there are many tokens, launches and latency below.  A
// token's logits are held by LANES lanes (16 up to 128 experts, so that a wave
// has four tokens and their reductions are four DPP steps; else a wave), PER
// experts a lane: expert q LANES + lane.  Measured: 8192 tokens of 128 experts
// (4.5 MB read, as much written by the gradient) 4.9 us for k_balance, 4.0 for
// its fold, 5.9 for k_route_grad, a launch and memory's latency each; 8192 x 8
// rows of 2048 (873 MB) 173 us for k_combine_grad, 5.0 TB/s, the rate of a copy.
#include <algorithm>
#include <type_traits>

#include "layer_launch.hpp"
#include "mx_device.hpp"
#include "quads_device.hpp"

namespace quads {
namespace {

template <int CTRL>
__device__ __forceinline__ float dpp_move(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xf, 0xf, true));
}

// Reductions over the token's lanes, in all of them: row rotations by 8, 4, 2
// and 1 give every lane of 16 the same set of partners; the four rows of a
// wave by swaps.
template <int LANES, class F>
__device__ __forceinline__ float token_reduce(float v, F f) {
  v = f(v, dpp_move<0x128>(v));
  v = f(v, dpp_move<0x124>(v));
  v = f(v, dpp_move<0x122>(v));
  v = f(v, dpp_move<0x121>(v));
  if constexpr (LANES == 64) {
    v = f(v, __shfl_xor(v, 16));
    v = f(v, __shfl_xor(v, 32));
  }
  return v;
}

template <int LANES>
__device__ __forceinline__ float token_sum(float v) {
  return token_reduce<LANES>(v, [](float a, float b) { return a + b; });
}

// p = softmax(l) over E experts; 0 throughout where every logit is -inf, NaN
// throughout where one is NaN or +inf.
template <int LANES, int PER>
__device__ __forceinline__ void softmax(float (&l)[PER]) {
  float m = l[0];
#pragma unroll
  for (int q = 1; q < PER; ++q) m = fmaxf(m, l[q]);
  m = token_reduce<LANES>(m, [](float a, float b) { return fmaxf(a, b); });
  if (m == -INFINITY) m = 0.0f;
  float sum = 0.0f;
#pragma unroll
  for (int q = 0; q < PER; ++q) {
    l[q] = expf(l[q] - m);
    sum += l[q];
  }
  sum = token_sum<LANES>(sum);
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
  for (int q = 0; q < PER; ++q) l[q] *= inv;
}

template <int LANES, int PER>
__device__ __forceinline__ void load_logits(const float *row, int E, int lane, float (&l)[PER]) {
#pragma unroll
  for (int q = 0; q < PER; ++q) l[q] = q * LANES + lane < E ? row[q * LANES + lane] : -INFINITY;
}

// ---- balance loss ------------------------------------------------------------------

constexpr int kBalanceThreads = 1024, kBalanceWaves = kBalanceThreads / 64;

struct BalanceParams {
  const float *logits;
  const int32_t *ids;
  const uint8_t *mask;
  int64_t T;
  int32_t E, top;
  float coef;
  float *loss;
  int32_t *counts;
  float *slope;
  float *partial_p;    // [groups, E]
  int32_t *partial_c;  // [groups, E + 1]; behind the counts the valid tokens
};

// The loss from the sums of the whole call in LDS; all threads of the workgroup.
__device__ __forceinline__ void balance_finish(const BalanceParams &p, const float *sum_p, const int32_t *count, int32_t n,
                                               float *parts) {
  const int t = threadIdx.x;
  // In 64 bits: what fp32 rounds off here is off by the same for all experts, and adds up in the loss.
  const double tokens = n, scale = n > 0 ? static_cast<double>(p.coef) * p.E / (tokens * tokens * p.top) : 0.0;
  float l = 0.0f;
  if (t < p.E) {  // E <= 1024 threads
    const float slope = static_cast<float>(scale * count[t]);
    p.counts[t] = count[t];
    p.slope[t] = slope;
    l = slope * sum_p[t];
  }
  l = token_sum<64>(l);
  if ((t & 63) == 0) parts[t >> 6] = l;
  __syncthreads();
  if (t == 0) {
    for (int w = 1; w < kBalanceWaves; ++w) l += parts[w];
    p.loss[0] = l;
  }
}

// Sums over this workgroup's tokens; with one workgroup the loss too.  A
// token's probabilities are added up in its lanes' registers, the workgroup's
// groups of lanes meet in LDS in order; counts by integer LDS atomics.
template <int LANES, int PER>
__global__ __launch_bounds__(kBalanceThreads) void k_balance(BalanceParams p) {
  constexpr int GROUPS = kBalanceThreads / LANES;  // tokens at once
  constexpr int ROUND = LANES * PER > 256 ? 16 : GROUPS;  // groups that meet at once: at most 64 KB of LDS
  __shared__ float meet[ROUND][LANES * PER];
  __shared__ int32_t count[LANES * PER];
  __shared__ int32_t valid_tokens;
  __shared__ float parts[kBalanceWaves];
  const int t = threadIdx.x, lane = t % LANES, group = t / LANES;
  for (int e = t; e < LANES * PER; e += kBalanceThreads) count[e] = 0;
  if (t == 0) valid_tokens = 0;
  __syncthreads();

  float acc[PER] = {};
  int32_t n = 0;
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * GROUPS; base < p.T; base += static_cast<int64_t>(gridDim.x) * GROUPS) {
    const int64_t token = base + group;
    const bool live = token < p.T && (p.mask == nullptr || p.mask[token] != 0);
    const int64_t at = min(token, p.T - 1);
    float l[PER];
    load_logits<LANES, PER>(p.logits + at * p.E, p.E, lane, l);
    const int32_t id = lane < p.top ? p.ids[at * p.top + lane] : -1;  // top <= 16 <= LANES
    softmax<LANES, PER>(l);
#pragma unroll
    for (int q = 0; q < PER; ++q) acc[q] += live ? l[q] : 0.0f;
    if (live && id >= 0 && id < p.E) atomicAdd(&count[id], 1);
    n += live;
  }
  if (lane == 0 && n != 0) atomicAdd(&valid_tokens, n);

  // Groups [r ROUND, (r + 1) ROUND) put their sums down; thread e adds them in order.
  float sum = 0.0f;
  for (int r = 0; r < GROUPS / ROUND; ++r) {
    if (group / ROUND == r) {
#pragma unroll
      for (int q = 0; q < PER; ++q) meet[group % ROUND][q * LANES + lane] = acc[q];
    }
    __syncthreads();
    if (t < p.E)
      for (int g = 0; g < ROUND; ++g) sum += meet[g][t];
    __syncthreads();
  }
  if (gridDim.x > 1) {
    if (t < p.E) {
      p.partial_p[static_cast<int64_t>(blockIdx.x) * p.E + t] = sum;
      p.partial_c[static_cast<int64_t>(blockIdx.x) * (p.E + 1) + t] = count[t];
    }
    if (t == 0) p.partial_c[static_cast<int64_t>(blockIdx.x) * (p.E + 1) + p.E] = valid_tokens;
    return;
  }
  float *all = &meet[0][0];
  if (t < p.E) all[t] = sum;
  balance_finish(p, all, count, valid_tokens, parts);  // thread t reads its own sum
}

// The workgroups' sums in order: thread (s, e) adds every S-th of expert e's.
__global__ __launch_bounds__(kBalanceThreads) void k_balance_fold(BalanceParams p, int groups) {
  __shared__ float sum_p[kBalanceThreads];
  __shared__ int32_t sum_c[kBalanceThreads];
  __shared__ int32_t valid_tokens;
  __shared__ float parts[kBalanceWaves];
  const int t = threadIdx.x, S = kBalanceThreads / p.E, s = t / p.E, e = t % p.E;
  if (t < 64) {
    int32_t n = 0;
    for (int g = t; g < groups; g += 64) n += p.partial_c[static_cast<int64_t>(g) * (p.E + 1) + p.E];
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) n += __shfl_xor(n, off);
    if (t == 0) valid_tokens = n;
  }
  float a = 0.0f;
  int32_t c = 0;
  if (s < S) {
#pragma unroll 8
    for (int g = s; g < groups; g += S) {
      a += p.partial_p[static_cast<int64_t>(g) * p.E + e];
      c += p.partial_c[static_cast<int64_t>(g) * (p.E + 1) + e];
    }
  }
  sum_p[t] = a;
  sum_c[t] = c;
  __syncthreads();
  if (t < p.E) {
    for (int k = 1; k < S; ++k) {
      a += sum_p[k * p.E + t];
      c += sum_c[k * p.E + t];
    }
  }
  __syncthreads();
  if (t < p.E) {
    sum_p[t] = a;
    sum_c[t] = c;
  }
  balance_finish(p, sum_p, sum_c, valid_tokens, parts);  // thread t reads its own sums
}

// Workgroups by the rounds of tokens and the experts a lane.  One (and one
// launch) while its rounds cost less than a second launch (512 x 16 6.9 and 7.2
// us, 128 x 128 5.6 and 6.6; but 192 x 128 7.2 and 6.8, 512 x 128 14.3 and 6.8);
// then up to 128, and 256 where these would make more than four rounds each
// (65536 x 128 19.5 -> 15.9 us, 65536 x 256 44 -> 29.5; but 16384 x 128 9.6 ->
// 10.0, 8192 x 512 16.9 -> 20.7, the fold).
int balance_groups(int64_t T, int32_t E) {
  const int lanes = E <= 128 ? 16 : 64, per = (E + lanes - 1) / lanes;
  const int64_t at_once = kBalanceThreads / lanes, rounds = (T + at_once - 1) / at_once;
  if (rounds <= 1 || (rounds <= 8 && rounds * per <= 16)) return 1;
  return static_cast<int>(std::min<int64_t>(rounds, rounds > 4 * 128 ? 256 : 128));
}

// f(integral_constant<LANES>, integral_constant<PER>) for E experts.
template <class F>
void by_experts(int32_t E, F &&f) {
  const auto go = [&](auto lanes, auto per) { f(lanes, per); };
  using L16 = std::integral_constant<int, 16>;
  using L64 = std::integral_constant<int, 64>;
  if (E <= 16) go(L16{}, std::integral_constant<int, 1>{});
  else if (E <= 32) go(L16{}, std::integral_constant<int, 2>{});
  else if (E <= 64) go(L16{}, std::integral_constant<int, 4>{});
  else if (E <= 128) go(L16{}, std::integral_constant<int, 8>{});
  else if (E <= 256) go(L64{}, std::integral_constant<int, 4>{});
  else if (E <= 512) go(L64{}, std::integral_constant<int, 8>{});
  else go(L64{}, std::integral_constant<int, 16>{});
}

// ---- gradient of the logits ----------------------------------------------------------

struct RouteGradParams {
  const float *logits;
  const int32_t *ids;
  const uint8_t *mask;
  const float *dw, *slope, *dloss;
  int64_t T, base;  // a launch has the tokens from base on
  int32_t E, top;
  float *dlogits;
};

template <int LANES, int PER>
__global__ __launch_bounds__(256) void k_route_grad(RouteGradParams p) {
  const int lane = threadIdx.x % LANES;
  const int64_t token = p.base + static_cast<int64_t>(blockIdx.x) * (256 / LANES) + threadIdx.x / LANES;
  const int64_t at = min(token, p.T - 1);  // lanes behind the last token take part in the DPP moves
  const bool live = p.mask == nullptr || p.mask[at] != 0;
  float l[PER], dp[PER];
  load_logits<LANES, PER>(p.logits + at * p.E, p.E, lane, l);
  const float g = p.slope ? (p.dloss ? p.dloss[0] : 1.0f) : 0.0f;
#pragma unroll
  for (int q = 0; q < PER; ++q) dp[q] = p.slope && q * LANES + lane < p.E ? g * p.slope[q * LANES + lane] : 0.0f;
  if (p.dw) {
    const bool has = lane < p.top;
    int32_t id = has ? p.ids[at * p.top + lane] : -1;
    if (id >= p.E) id = -1;  // a lane may have a place of that number, where p = 0 times an infinite dw is NaN
    const float w = has ? p.dw[at * p.top + lane] : 0.0f;
    for (int j = 0; j < p.top; ++j) {
      const int32_t e = __shfl(id, j, LANES);
      const float d = __shfl(w, j, LANES);
#pragma unroll
      for (int q = 0; q < PER; ++q)
        if (e == q * LANES + lane) dp[q] += d;
    }
  }
  softmax<LANES, PER>(l);
  float dot = 0.0f;
#pragma unroll
  for (int q = 0; q < PER; ++q) dot = __builtin_fmaf(l[q], dp[q], dot);
  dot = token_sum<LANES>(dot);
  if (token >= p.T) return;
#pragma unroll
  for (int q = 0; q < PER; ++q)
    if (q * LANES + lane < p.E) p.dlogits[token * p.E + q * LANES + lane] = live ? l[q] * (dp[q] - dot) : 0.0f;
}

// ---- gradient of the combine -----------------------------------------------------------

struct CombineGradParams {
  const void *dout, *y;
  const int32_t *inverse;
  const float *w;
  int64_t T, base, rows, N;  // a launch has the tokens from base on
  int32_t top;
  uint16_t *dy;
  float *dw;
};

template <bool BF16>
__device__ __forceinline__ void load8(const void *p, int64_t unit, float (&v)[8]) {
  if constexpr (BF16) {
    const uint4 r = static_cast<const uint4 *>(p)[unit];
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
    const float4 *q = static_cast<const float4 *>(p) + 2 * unit;
    const float4 a = q[0], b = q[1];
    v[0] = a.x;
    v[1] = a.y;
    v[2] = a.z;
    v[3] = a.w;
    v[4] = b.x;
    v[5] = b.y;
    v[6] = b.z;
    v[7] = b.w;
  }
}

// WAVES waves share a token; its row of dout is read once for its SLOTS >= top
// slots.  A slot whose row number lies outside y has no row: nothing is
// written for it but dw = 0.  Tokens write in no order: a row that two of them
// name gets units of both.
template <int SLOTS, int WAVES, bool DOUT_BF16, bool Y_BF16>
__global__ __launch_bounds__(256) void k_combine_grad(CombineGradParams p) {
  __shared__ float parts[4][SLOTS];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, part = wave % WAVES;
  const int64_t token = p.base + static_cast<int64_t>(blockIdx.x) * (4 / WAVES) + wave / WAVES;
  if (WAVES == 1 && token >= p.T) return;  // whole waves; with WAVES == 4 every workgroup has a token
  const int64_t units = p.N / 8;
  int64_t row[SLOTS];
  float w[SLOTS], dot[SLOTS];
#pragma unroll
  for (int j = 0; j < SLOTS; ++j) {
    const int32_t r = j < p.top ? p.inverse[token * p.top + j] : -1;
    row[j] = r >= 0 && r < p.rows ? r : -1;
    w[j] = j < p.top ? p.w[token * p.top + j] : 0.0f;
    dot[j] = 0.0f;
  }
  const bool dots = p.dw != nullptr;
  for (int64_t u = part * 64 + lane; u < units; u += 64 * WAVES) {
    float d[8];
    load8<DOUT_BF16>(p.dout, token * units + u, d);
    if (dots) {
      constexpr int AT_ONCE = SLOTS < 8 ? SLOTS : 8;
#pragma unroll
      for (int first = 0; first < SLOTS; first += AT_ONCE) {
        float y[AT_ONCE][8];
#pragma unroll
        for (int j = 0; j < AT_ONCE; ++j) load8<Y_BF16>(p.y, max(row[first + j], int64_t(0)) * units + u, y[j]);
#pragma unroll
        for (int j = 0; j < AT_ONCE; ++j)
#pragma unroll
          for (int i = 0; i < 8; ++i) dot[first + j] = __builtin_fmaf(d[i], y[j][i], dot[first + j]);
        // The next eight go into the same registers: loaded ahead, 16 slots take 256
        // of them (4096 x 16 bf16 rows of 2048 242 us, so 120).
        if constexpr (SLOTS > AT_ONCE) __builtin_amdgcn_sched_barrier(0);
      }
    }
#pragma unroll
    for (int j = 0; j < SLOTS; ++j) {
      if (row[j] < 0) continue;
      reinterpret_cast<uint4 *>(p.dy)[row[j] * units + u] =
          make_uint4(pack_bf16(w[j] * d[0], w[j] * d[1]), pack_bf16(w[j] * d[2], w[j] * d[3]),
                     pack_bf16(w[j] * d[4], w[j] * d[5]), pack_bf16(w[j] * d[6], w[j] * d[7]));
    }
  }
  if (!dots) return;
#pragma unroll
  for (int j = 0; j < SLOTS; ++j) {
    dot[j] = token_sum<64>(dot[j]);
    if (row[j] < 0) dot[j] = 0.0f;
  }
  if constexpr (WAVES == 1) {
#pragma unroll
    for (int j = 0; j < SLOTS; ++j)
      if (lane == 0 && j < p.top) p.dw[token * p.top + j] = dot[j];
  } else {
#pragma unroll
    for (int j = 0; j < SLOTS; ++j)
      if (lane == 0) parts[wave][j] = dot[j];
    __syncthreads();
    const int j = threadIdx.x;
    if (j < p.top) p.dw[token * p.top + j] = ((parts[0][j] + parts[1][j]) + parts[2][j]) + parts[3][j];
  }
}

template <int SLOTS, int WAVES>
hipError_t run_combine_grad(const CombineGradLaunch &a, hipStream_t stream) {
  constexpr int64_t TOKENS = 4 / WAVES;  // of a workgroup
  CombineGradParams p{a.dout, a.y, a.inverse, a.w, a.T, 0, a.rows, a.N, a.top, a.dy, a.dw};
  for (; p.base < a.T; p.base += kLaunchGroups * TOKENS) {
    const int64_t groups = std::min((a.T - p.base + TOKENS - 1) / TOKENS, kLaunchGroups);
    const dim3 grid(static_cast<unsigned>(groups)), threads(256);
    if (a.dout_bf16 && a.y_bf16) hipLaunchKernelGGL((k_combine_grad<SLOTS, WAVES, true, true>), grid, threads, 0, stream, p);
    else if (a.dout_bf16) hipLaunchKernelGGL((k_combine_grad<SLOTS, WAVES, true, false>), grid, threads, 0, stream, p);
    else if (a.y_bf16) hipLaunchKernelGGL((k_combine_grad<SLOTS, WAVES, false, true>), grid, threads, 0, stream, p);
    else hipLaunchKernelGGL((k_combine_grad<SLOTS, WAVES, false, false>), grid, threads, 0, stream, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int WAVES>
hipError_t run_combine_grad(const CombineGradLaunch &a, hipStream_t stream) {
  if (a.top <= 2) return run_combine_grad<2, WAVES>(a, stream);
  if (a.top <= 4) return run_combine_grad<4, WAVES>(a, stream);
  if (a.top <= 8) return run_combine_grad<8, WAVES>(a, stream);
  return run_combine_grad<16, WAVES>(a, stream);
}

}  // namespace

size_t balance_ws_bytes(int64_t T, int32_t E) {
  const int groups = balance_groups(T, E);
  return groups > 1 ? static_cast<size_t>(groups) * (2 * E + 1) * 4 : 0;
}

hipError_t launch_balance(const BalanceLaunch &a, hipStream_t stream) {
  const int groups = balance_groups(a.T, a.E);
  BalanceParams p{a.logits, a.ids, a.mask, a.T, a.E, a.top, a.coef, a.loss, a.counts, a.slope, nullptr, nullptr};
  if (groups > 1) {
    p.partial_p = static_cast<float *>(a.ws);
    p.partial_c = reinterpret_cast<int32_t *>(p.partial_p + static_cast<int64_t>(groups) * a.E);
  }
  by_experts(a.E, [&](auto lanes, auto per) {
    hipLaunchKernelGGL((k_balance<decltype(lanes)::value, decltype(per)::value>), dim3(groups), dim3(kBalanceThreads), 0,
                       stream, p);
  });
  if (groups > 1) hipLaunchKernelGGL(k_balance_fold, dim3(1), dim3(kBalanceThreads), 0, stream, p, groups);
  return hipGetLastError();
}

hipError_t launch_route_grad(const RouteGradLaunch &a, hipStream_t stream) {
  RouteGradParams p{a.logits, a.ids, a.mask, a.dw, a.slope, a.dloss, a.T, 0, a.E, a.top, a.dlogits};
  hipError_t e = hipSuccess;
  by_experts(a.E, [&](auto lanes, auto per) {
    constexpr int64_t TOKENS = 256 / decltype(lanes)::value;
    for (; p.base < a.T && e == hipSuccess; p.base += kLaunchGroups * TOKENS) {
      const int64_t groups = std::min((a.T - p.base + TOKENS - 1) / TOKENS, kLaunchGroups);
      hipLaunchKernelGGL((k_route_grad<decltype(lanes)::value, decltype(per)::value>), dim3(static_cast<unsigned>(groups)),
                         dim3(256), 0, stream, p);
      e = hipGetLastError();
    }
  });
  return e;
}

hipError_t launch_combine_grad(const CombineGradLaunch &a, hipStream_t stream) {
  // Four waves a token where one each would leave the card idle, or where all
  // four have whole lines to read (8192 x 8 rows of 2048 198 -> 174 us, 4096 x 16
  // of 2048 205 -> 177; but 16384 x 8 of 512 92 -> 102, of 1024 in bf16 129 -> 137).
  // Around 1024 tokens, all in bf16, one wave and four: 512 x 8 of 1024 5.7 and
  // 5.0, 64 x 8 of 1536 5.8 and 3.7, 768 x 8 of 512 4.55 and 4.57, 1024 x 8 of 512
  // 4.9 and 6.6, of 1024 7.5 and 8.9, of 1536 10.9 and 11.3.  With two slots the
  // sides meet elsewhere: four waves are ahead up to 1500 tokens of 1024 (1024 x
  // 2 3.6 and 3.4), and nowhere at 512 (768 x 2 2.8 and 3.0), which the rule leaves.
  return a.T < 1024 || a.N >= 2048 ? run_combine_grad<4>(a, stream) : run_combine_grad<1>(a, stream);
}

}  // namespace quads
