// All Newton-Schulz steps of one small matrix by one workgroup, in LDS; and a
// step of a long one by a workgroup for each slab of its columns (further down).
//
// X (m x n, m <= n: a tall G is taken transposed) lies in LDS as hi and lo in
// fp16, rows of n + 8, and one m x m array holds A and then B.  Scales and
// roundings are those of the products over tiles, except that lo is kept up to
// the last step: here it costs no traffic.  Rows and columns behind the matrix,
// up to multiples of 32, are zeros and stay zeros.
//
// A wave makes 32 x 32 tiles.  A = X X^T and A^2 read rows of both operands.
// B X reads X's columns by transposing reads as the first operand and B's rows
// as the second, so a lane holds four neighbours of a row of X, and a wave takes
// whole blocks of 32 columns: what it overwrites no other wave reads.
//
// Bound: latency (LDS reads, and four barriers a step).  Waves wait for 48 to 64%
// of their cycles; of 2000 of 128 x 128 the matrix cores are busy for 20% and the
// LDS for 41% of the time and 12% more with bank conflicts, of 256 of 64 x 128 for
// 9, 28 and 10%.  Five steps of one 32 x 32 take 8 us, of 256 of 64 x 128 18, of
// one 128 x 224 38, of 2000 of 128 x 128 293 (0.29 PFLOP/s); by products over
// tiles 87, 118, 89 and 724.
#pragma once

#include "batched_tile.hpp"

namespace quads {

constexpr float kXScale = 2048.0f, kAScale = 1024.0f;

// Unit `unit` of 8 values of fp32 or bf16.
__device__ __forceinline__ void load_values(const void *g, bool f32, int64_t unit, float (&v)[8]) {
  if (f32) {
    const float4 *q = static_cast<const float4 *>(g) + 2 * unit;
    const float4 a = q[0], b = q[1];
    const float w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = w[i];
  } else {
    const uint4 r = static_cast<const uint4 *>(g)[unit];
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off);
  return v;
}

struct SmallOrthogonalParams {
  const void *g;
  uint16_t *out;
  bool f32, tall;
  int32_t rows, cols, np;  // np: the longer side, up to a multiple of 32
  int32_t steps;
  float a, b, c;
  double eps;
};

// LDS of a matrix with sides 32 mr and np.
constexpr int64_t small_orthogonal_lds(int64_t mr, int64_t np) { return 32 * mr * (4 * (np + 8) + 2 * (32 * mr + 8)); }

__device__ __forceinline__ uint2 read_lds8(uint32_t at) {
  typedef __attribute__((address_space(3))) const u32x2 lds_u32x2;
  const u32x2 v = *reinterpret_cast<lds_u32x2 *>(static_cast<uintptr_t>(at));
  return make_uint2(v[0], v[1]);
}
__device__ __forceinline__ void write_lds8(uint32_t at, uint32_t lo, uint32_t hi) {
  typedef __attribute__((address_space(3))) u32x2 lds_u32x2;
  *reinterpret_cast<lds_u32x2 *>(static_cast<uintptr_t>(at)) = u32x2{lo, hi};
}
__device__ __forceinline__ void write_lds16(uint32_t at, uint4 v) {
  typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
  *reinterpret_cast<lds_u32x4 *>(static_cast<uintptr_t>(at)) = u32x4{v.x, v.y, v.z, v.w};
}
__device__ __forceinline__ void write_lds2(uint32_t at, uint32_t v) {
  typedef __attribute__((address_space(3))) uint16_t lds_u16;
  *reinterpret_cast<lds_u16 *>(static_cast<uintptr_t>(at)) = static_cast<uint16_t>(v);
}

// Element i of 4 fp16 values.
__device__ __forceinline__ float half_of(uint2 v, int i) {
  const f16x2 p = __builtin_bit_cast(f16x2, i < 2 ? v.x : v.y);
  return static_cast<float>(p[i & 1]);
}

// X of 32 MR rows and np columns as hi and lo, and one array for A and B.
template <int MR, int WAVES>
struct SmallMatrix {
  static constexpr int MP = 32 * MR, TILES = MR * MR, OWN = (TILES + WAVES - 1) / WAVES, THREADS = 64 * WAVES;
  static constexpr uint32_t AROW = 2 * (MP + 8);
  int np, wave, lane, half, fr;
  uint32_t x0, xrow, lo, a0;  // lo: from hi to lo

  __device__ __forceinline__ SmallMatrix(uint32_t at, int columns)
      : np(columns), wave(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6)), lane(threadIdx.x & 63), half(lane >> 5),
        fr(lane & 31), x0(at), xrow(2 * (columns + 8)), lo(MP * xrow), a0(at + 2 * lo) {}

  __device__ __forceinline__ void clear() const {
    for (uint32_t at = 16 * threadIdx.x; at < 2 * lo; at += 16 * THREADS) write_lds16(x0 + at, make_uint4(0, 0, 0, 0));
  }

  // Eight neighbours of G's row, times scale, into row `row` of X from `col` on, or (tall) into rows `col` .. of column `row`.
  __device__ __forceinline__ void put(float (&v)[8], double scale, uint32_t row, uint32_t col, bool tall) const {
    float rest[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = static_cast<float>(v[i] * scale);
    split_f16(v, rest);
    if (!tall) {
      const uint32_t at = x0 + row * xrow + 2 * col;
      write_lds16(at, make_uint4(pack_f16(v[0], v[1]), pack_f16(v[2], v[3]), pack_f16(v[4], v[5]), pack_f16(v[6], v[7])));
      write_lds16(at + lo, make_uint4(pack_f16(rest[0], rest[1]), pack_f16(rest[2], rest[3]), pack_f16(rest[4], rest[5]),
                                      pack_f16(rest[6], rest[7])));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t at = x0 + (col + i) * xrow + 2 * row;
        write_lds2(at, pack_f16(v[i], v[i]));
        write_lds2(at + lo, pack_f16(rest[i], rest[i]));
      }
    }
  }

  // Tile (i, j) of the products of rows: a lane has element (row 32 j + fr of the
  // second, 8 q + 4 half + r of the first's 32 rows) in register 4 q + r.
  __device__ __forceinline__ f32x16 rows_product(uint32_t at, uint32_t stride, int i, int j, int k_end) const {
    f32x16 acc = {};
    const uint32_t x = at + (32 * i + fr) * stride + 16 * half, y = at + (32 * j + fr) * stride + 16 * half;
    uint4 f[4] = {read_lds16(x), read_lds16(y), read_lds16(x + 32), read_lds16(y + 32)};
    for (int k = 0; k < k_end; k += 32) {  // the next reads under way
      const uint32_t next = k + 32 < k_end ? 2 * (k + 32) : 0;
      const uint4 n[4] = {read_lds16(x + next), read_lds16(y + next), read_lds16(x + next + 32), read_lds16(y + next + 32)};
      acc = mfma_f16(f[0], f[1], acc);
      acc = mfma_f16(f[2], f[3], acc);
#pragma unroll
      for (int e = 0; e < 4; ++e) f[e] = n[e];
    }
    return acc;
  }
  __device__ __forceinline__ f32x16 gram(int i, int j) const { return rows_product(x0, xrow, i, j, np); }

  // Byte of a lane's first four results in a row of A; the next four are 16 on.
  __device__ __forceinline__ uint32_t a_at(int i, int j) const { return a0 + (32 * j + fr) * AROW + 2 * (32 * i + 4 * half); }

  __device__ __forceinline__ void put_a(int i, int j, int q, float v0, float v1, float v2, float v3) const {
    constexpr float alpha = kAScale / (kXScale * kXScale);
    write_lds8(a_at(i, j) + 16 * q, pack_f16(alpha * v0, alpha * v1), pack_f16(alpha * v2, alpha * v3));
  }

  // A -> b A + c A^2 in its place, when all have read it; barriers before (A is there) and behind.
  __device__ __forceinline__ void poly(float pb, float pc) const {
    __syncthreads();
    uint2 b[OWN][4];
    const float alpha = pc / (kAScale * kAScale), beta = pb / kAScale;
#pragma unroll
    for (int o = 0; o < OWN; ++o) {
      const int tile = wave + WAVES * o, i = tile / MR, j = tile % MR;
      if (tile >= TILES) continue;
      const f32x16 s = rows_product(a0, AROW, i, j, MP);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint2 in = read_lds8(a_at(i, j) + 16 * q);
        float v[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = __builtin_fmaf(half_of(in, r), beta, alpha * s[4 * q + r]);
        b[o][q] = make_uint2(pack_f16(v[0], v[1]), pack_f16(v[2], v[3]));
      }
    }
    __syncthreads();
#pragma unroll
    for (int o = 0; o < OWN; ++o) {
      const int tile = wave + WAVES * o, i = tile / MR, j = tile % MR;
      if (tile >= TILES) continue;
#pragma unroll
      for (int q = 0; q < 4; ++q) write_lds8(a_at(i, j) + 16 * q, b[o][q].x, b[o][q].y);
    }
    __syncthreads();
  }

  // X <- a X + B X; of the last step emit(row, column, the two dwords of four bf16 results) instead.
  template <class Emit>
  __device__ __forceinline__ void update(float a, bool last, Emit emit) const {
    for (int block = wave; block < np / 32; block += WAVES) {
      f32x16 acc[MR];
#pragma unroll
      for (int r = 0; r < MR; ++r) acc[r] = f32x16{};
      // Lane 16 g + 4 j + b of a transposing read addresses row j and columns 4 (4 (g % 2) + b) .. of the block, in half g / 2.
      const uint32_t x = x0 + (8 * half + ((lane >> 2) & 3)) * xrow + 2 * (32 * block + 4 * (4 * ((lane >> 4) & 1) + (lane & 3)));
#pragma unroll
      for (int k = 0; k < MP; k += 16) {
        const uint2 u = read_tr_at(x + k * xrow), v = read_tr_at(x + (k + 4) * xrow);
#pragma unroll
        for (int r = 0; r < MR; ++r)
          acc[r] = mfma_f16(make_uint4(u.x, u.y, v.x, v.y), read_lds16(a0 + (32 * r + fr) * AROW + 2 * k + 16 * half), acc[r]);
      }
#pragma unroll
      for (int r = 0; r < MR; ++r) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int row = 32 * r + fr, col = 32 * block + 8 * q + 4 * half;
          const uint32_t at = x0 + row * xrow + 2 * col;
          const uint2 h = read_lds8(at), l = read_lds8(at + lo);
          float v[4], rest[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            v[e] = __builtin_fmaf(half_of(l, e), a, __builtin_fmaf(half_of(h, e), a, acc[r][4 * q + e]));
          if (!last) {
            split_f16(v, rest);
            write_lds8(at, pack_f16(v[0], v[1]), pack_f16(v[2], v[3]));
            write_lds8(at + lo, pack_f16(rest[0], rest[1]), pack_f16(rest[2], rest[3]));
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] *= 1.0f / kXScale;
            emit(row, col, pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
          }
        }
      }
    }
  }
};

// Four results of X's row `row` from column `col` on, at their place in out.
__device__ __forceinline__ void emit_small(const SmallOrthogonalParams &p, uint16_t *out, int row, int col, uint32_t w0, uint32_t w1) {
  if (!p.tall) {
    if (row < p.rows && col < p.cols) *reinterpret_cast<u32x2 *>(out + static_cast<int64_t>(row) * p.cols + col) = u32x2{w0, w1};
  } else if (row < p.cols && col < p.rows) {
    uint16_t *to = out + static_cast<int64_t>(col) * p.cols + row;
    to[0] = static_cast<uint16_t>(w0);
    to[p.cols] = static_cast<uint16_t>(w0 >> 16);
    to[2 * p.cols] = static_cast<uint16_t>(w1);
    to[3 * p.cols] = static_cast<uint16_t>(w1 >> 16);
  }
}

template <int MR, int BYTES, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_orthogonal_small(SmallOrthogonalParams p) {
  using M = SmallMatrix<MR, WAVES>;
  __shared__ __attribute__((aligned(128))) uint8_t lds[BYTES];
  __shared__ double parts[WAVES];
  const M x(lds_address(lds), p.np);
  x.clear();
  const uint32_t row_units = p.cols / 8, units = p.rows * row_units;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * units;
  double ss = 0.0;
  for (uint32_t u = threadIdx.x; u < units; u += M::THREADS) {
    float v[8];
    load_values(p.g, p.f32, first + u, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) ss += static_cast<double>(v[i]) * static_cast<double>(v[i]);
  }
  ss = wave_sum(ss);
  if (x.lane == 0) parts[x.wave] = ss;
  __syncthreads();
  ss = parts[0];
  for (int w = 1; w < WAVES; ++w) ss += parts[w];
  const double scale = static_cast<double>(kXScale) / (sqrt(ss) + p.eps);
  for (uint32_t u = threadIdx.x; u < units; u += M::THREADS) {
    float v[8];
    load_values(p.g, p.f32, first + u, v);
    x.put(v, scale, u / row_units, 8 * (u % row_units), p.tall);
  }
  __syncthreads();

  for (int step = 0; step < p.steps; ++step) {
    for (int tile = x.wave; tile < M::TILES; tile += WAVES) {
      const f32x16 s = x.gram(tile / MR, tile % MR);
#pragma unroll
      for (int q = 0; q < 4; ++q) x.put_a(tile / MR, tile % MR, q, s[4 * q], s[4 * q + 1], s[4 * q + 2], s[4 * q + 3]);
    }
    x.poly(p.b, p.c);
    x.update(p.a, step + 1 == p.steps,
             [&](int row, int col, uint32_t w0, uint32_t w1) { emit_small(p, p.out + 8 * first, row, col, w0, w1); });
    __syncthreads();
  }
}

// ---- a long matrix in slabs of its columns ------------------------------------------
// A launch a step: a workgroup has np columns of X.  It adds the slabs' parts of
// A in their order, makes B (every slab's workgroup the same), its columns of the
// new X, and their part of the next A.
//
// Bound: with few matrices a launch and memory's latency a step (one 32 x 2048
// 40 us, five steps; one 128 x 2048 110), with many X's traffic and the slabs'
// parts of A, which every slab reads (256 of 32 x 2048 240 us, of 64 x 2048 796:
// 671 MB read and 201 written a step, where X in and out is 134 each).

struct SlabParams {
  SmallOrthogonalParams m;
  int32_t slabs, phase;       // phase 0: X from g, and its part of A; then the steps
  int32_t parts;
  const double *partial;      // [batch, parts] sums of squares
  uint4 *x;                   // [batch, slabs, 2, MP, np] fp16: hi, lo
  const float4 *gram;         // [batch, slabs, MP * MP] of the phase before, and
  float4 *next_gram;          // of this one
};

template <int MR, int BYTES, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_orthogonal_slab(SlabParams p) {
  using M = SmallMatrix<MR, WAVES>;
  __shared__ __attribute__((aligned(128))) uint8_t lds[BYTES];
  const M x(lds_address(lds), p.m.np);
  const int matrix = blockIdx.x / p.slabs, slab = blockIdx.x % p.slabs, np = p.m.np;
  const int64_t elems = static_cast<int64_t>(p.m.rows) * p.m.cols;
  const uint32_t row16 = np / 8, plane = M::MP * row16;  // units of 8 halves
  uint4 *mine = p.x + static_cast<int64_t>(blockIdx.x) * 2 * plane;
  if (p.phase == 0) {
    double ss = 0.0;
    for (int i = x.lane; i < p.parts; i += 64) ss += p.partial[static_cast<int64_t>(matrix) * p.parts + i];
    ss = wave_sum(ss);
    const double scale = static_cast<double>(kXScale) / (sqrt(ss) + p.m.eps);
    x.clear();
    __syncthreads();
    const uint32_t lines = p.m.tall ? np : p.m.rows, line_units = p.m.tall ? p.m.cols / 8 : row16;
    for (uint32_t u = threadIdx.x; u < lines * line_units; u += M::THREADS) {
      const uint32_t line = u / line_units, unit = u % line_units;
      const int64_t row = p.m.tall ? static_cast<int64_t>(slab) * np + line : line;
      const int64_t col = p.m.tall ? 8 * unit : static_cast<int64_t>(slab) * np + 8 * unit;
      if (row >= p.m.rows || col >= p.m.cols) continue;
      float v[8];
      load_values(p.m.g, p.m.f32, (matrix * elems + row * p.m.cols + col) / 8, v);
      x.put(v, scale, line, 8 * unit, p.m.tall);
    }
    __syncthreads();
  } else {
    for (uint32_t u = threadIdx.x; u < 2 * plane; u += M::THREADS) {
      const uint32_t row = u / row16;  // lo's rows follow hi's
      write_lds16(x.x0 + row * x.xrow + 16 * (u % row16), mine[u]);
    }
    const float4 *parts = p.gram + static_cast<int64_t>(matrix) * p.slabs * (M::MP * M::MP / 4);
    for (int tile = x.wave; tile < M::TILES; tile += WAVES) {
      float4 sum[4] = {};
      for (int k = 0; k < p.slabs; ++k)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float4 v = parts[k * (M::MP * M::MP / 4) + (tile * 4 + q) * 64 + x.lane];
          sum[q].x += v.x;
          sum[q].y += v.y;
          sum[q].z += v.z;
          sum[q].w += v.w;
        }
#pragma unroll
      for (int q = 0; q < 4; ++q) x.put_a(tile / MR, tile % MR, q, sum[q].x, sum[q].y, sum[q].z, sum[q].w);
    }
    x.poly(p.m.b, p.m.c);
    const bool last = p.phase == p.m.steps;
    x.update(p.m.a, last, [&](int row, int col, uint32_t w0, uint32_t w1) {
      emit_small(p.m, p.m.out + matrix * elems, row, slab * np + col, w0, w1);
    });
    if (last) return;
    __syncthreads();
  }
  for (uint32_t u = threadIdx.x; u < 2 * plane; u += M::THREADS)
    mine[u] = read_lds16(x.x0 + u / row16 * x.xrow + 16 * (u % row16));
  float4 *part = p.next_gram + static_cast<int64_t>(blockIdx.x) * (M::MP * M::MP / 4);
  for (int tile = x.wave; tile < M::TILES; tile += WAVES) {
    const f32x16 s = x.gram(tile / MR, tile % MR);
#pragma unroll
    for (int q = 0; q < 4; ++q)
      part[(tile * 4 + q) * 64 + x.lane] = make_float4(s[4 * q], s[4 * q + 1], s[4 * q + 2], s[4 * q + 3]);
  }
}

}  // namespace quads
