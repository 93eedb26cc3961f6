// Orthogonalised updates by Newton-Schulz products on gfx950: for each matrix
//   X = G / (|G|_F + eps),   then `steps` times   A = X X^T,  B = b A + c A^2,
//   X <- a X + B X   (X <- a X + X B with A = X^T X where G has more rows than
// columns), which moves every singular value s by s (a + b s^2 + c s^4) and
// leaves the singular vectors.
//
// Precision.  Products take fp16 operands (11 significant bits, the matrix
// cores' rate is bf16's) and add in fp32.  X itself is kept as a sum hi + lo of
// two fp16 values (22 bits): hi enters the products, hi + lo the term a X.  A
// rounding of X is noise in all directions, also in those that G lacks (an
// expert that saw few tokens has a gradient of low rank), where each further
// step multiplies it by a: 3.4445^5 = 485 times for X's first rounding.  Without
// lo an update of rank 16 in 256 is off by 4%, with it by 0.06%; noise in A and B
// only enters multiplied by X.  Power-of-two scales keep X and A in fp16's
// normal range: X times 2^11, A times 2^10.  B's entries below 2^-14 are rounded
// by up to 2^-25 where B's norm is of the order of 1, or B X does not matter.
//
// Bound: the matrix cores, 3 m^2 n + m^3 operations a step for the short side m
// and the long side n: A and A^2 are symmetric, and only tiles on and below the
// diagonal are computed; each is stored a second time transposed.
//
// Measured, 128 matrices of 1024 x 2048 in fp32, five steps, 7.0 ms: k_square_sums
// 204 us (1.07 GB, 5.3 TB/s), k_split 398 (2.15 GB, 5.4 TB/s); a step's A 333 us
// (1.03 PFLOP/s with the tiles on the diagonal in full), B 208 (0.83), X 785 in
// hi and lo (0.70; 3.0 GB at 3.8 TB/s), 671 in hi alone, 632 as the result.
// The X products' epilogue moves its planes after a tile's products; with it
// left out 596 us.  256 matrices of 1024 x 2048 13.9 to 14.3 ms, 128 of 2048 x
// 1024 in bf16 6.8 to 7.0.
#include <algorithm>

#include "batched_tile.hpp"
#include "orthogonal_launch.hpp"
#include "orthogonal_small.hpp"

namespace quads {
namespace {

// ---- normalisation -------------------------------------------------------------

constexpr int kNormThreads = 256;

struct SplitParams {
  const void *g;
  bool f32;
  int32_t rows, row_units;          // of a matrix; units of 8 elements
  int32_t pad_rows, pad_row_units;  // of hi and lo, which hold zeros outside it
  double eps;
  double *partial;  // [batch, parts]
  uint16_t *hi, *lo;
};

// Part blockIdx.x of matrix blockIdx.y's sum of squares, in 64 bits: squares of
// fp32 neither overflow nor vanish.
__global__ __launch_bounds__(kNormThreads) void k_square_sums(SplitParams p) {
  __shared__ double parts[kNormThreads / 64];
  const int64_t units = static_cast<int64_t>(p.rows) * p.row_units, base = blockIdx.y * units;
  const int64_t per = (units + gridDim.x - 1) / gridDim.x, end = min(units, (blockIdx.x + 1) * per);
  double s = 0.0;
  for (int64_t u = blockIdx.x * per + threadIdx.x; u < end; u += kNormThreads) {
    float v[8];
    load_values(p.g, p.f32, base + u, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) s += static_cast<double>(v[i]) * static_cast<double>(v[i]);
  }
  s = wave_sum(s);
  if ((threadIdx.x & 63) == 0) parts[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0)
    p.partial[static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x] = ((parts[0] + parts[1]) + parts[2]) + parts[3];
}

// The matrix divided by its norm, as hi + lo.  A workgroup has rows of its own.
__global__ __launch_bounds__(kNormThreads) void k_split(SplitParams p) {
  const int parts = static_cast<int>(gridDim.x);
  double ss = 0.0;
  for (int i = threadIdx.x & 63; i < parts; i += 64) ss += p.partial[static_cast<int64_t>(blockIdx.y) * parts + i];
  ss = wave_sum(ss);
  const double scale = static_cast<double>(kXScale) / (sqrt(ss) + p.eps);
  const int32_t per = (p.pad_rows + parts - 1) / parts, first = blockIdx.x * per, last = min(p.pad_rows, first + per);
  if (first >= last) return;
  const uint32_t units = static_cast<uint32_t>(last - first) * p.pad_row_units;  // at most 2^20 / 64 rows of 2^17
  for (uint32_t u = threadIdx.x; u < units; u += kNormThreads) {
    const int32_t row = first + static_cast<int32_t>(u / p.pad_row_units), col = static_cast<int32_t>(u % p.pad_row_units);
    float v[8] = {}, lo[8];
    if (row < p.rows && col < p.row_units) {
      load_values(p.g, p.f32, (static_cast<int64_t>(blockIdx.y) * p.rows + row) * p.row_units + col, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = static_cast<float>(v[i] * scale);
    }
    split_f16(v, lo);
    const int64_t at = (static_cast<int64_t>(blockIdx.y) * p.pad_rows + row) * p.pad_row_units + col;
    reinterpret_cast<uint4 *>(p.hi)[at] = make_uint4(pack_f16(v[0], v[1]), pack_f16(v[2], v[3]), pack_f16(v[4], v[5]), pack_f16(v[6], v[7]));
    reinterpret_cast<uint4 *>(p.lo)[at] = make_uint4(pack_f16(lo[0], lo[1]), pack_f16(lo[2], lo[3]), pack_f16(lo[4], lo[5]), pack_f16(lo[6], lo[7]));
  }
}

template <bool WT>
hipError_t launch_next(int epi, const BatchedParams &p, hipStream_t stream) {
  switch (epi) {
    case kEpiNext: return launch_batched<false, WT, kEpiNext>(p, stream);
    case kEpiRound: return launch_batched<false, WT, kEpiRound>(p, stream);
    case kEpiLast: return launch_batched<false, WT, kEpiLast>(p, stream);
    default: return launch_batched<false, WT, kEpiOnly>(p, stream);
  }
}

// Workgroups of a matrix: at least 64 for a large one, more where there are few
// matrices (one of 1536 x 2048 with 64: 10 and 14 us for the two kernels).
int parts_of(int64_t batch, int64_t units) {
  return static_cast<int>(std::min<int64_t>((units + 1023) / 1024, std::max<int64_t>(64, 512 / batch)));
}

int64_t up256(int64_t v) { return (v + 255) / 256 * 256; }

// A side of the workspace's matrices: contractions are whole stages, and no
// fewer than the products have under way.  The rows and columns behind the
// matrix are zeros, and zeros they stay.
int64_t padded(int64_t side) { return std::max<int64_t>(128, (side + 31) / 32 * 32); }

// The workspace: for every matrix of a pass hi twice (a step reads one and
// writes the other), lo, A and B; partial sums.
struct Layout {
  int64_t rows, cols, m;  // padded
  int64_t hi[2], lo, a, b, partial, bytes;
};

Layout layout(int64_t batch, int64_t rows, int64_t cols) {
  Layout l{};
  l.rows = padded(rows);
  l.cols = padded(cols);
  l.m = std::min(l.rows, l.cols);
  const int64_t x = up256(2 * batch * l.rows * l.cols), s = up256(2 * batch * l.m * l.m);
  l.hi[0] = 0;
  l.hi[1] = x;
  l.lo = 2 * x;
  l.a = 3 * x;
  l.b = l.a + s;
  l.partial = l.b + s;
  l.bytes = l.partial + up256(8 * batch * parts_of(batch, rows * cols / 8));
  return l;
}

hipError_t launch_pass(const OrthogonalLaunch &o, hipStream_t stream) {
  const int64_t rows = o.rows, cols = o.cols;
  const bool tall = rows > cols;
  const Layout l = layout(o.batch, rows, cols);
  uint8_t *ws = static_cast<uint8_t *>(o.ws);
  const auto at = [&](int64_t offset) { return reinterpret_cast<uint16_t *>(ws + offset); };

  const SplitParams s{o.g, o.g_f32, static_cast<int32_t>(rows), static_cast<int32_t>(cols / 8), static_cast<int32_t>(l.rows),
                      static_cast<int32_t>(l.cols / 8), o.eps, reinterpret_cast<double *>(ws + l.partial), at(l.hi[0]), at(l.lo)};
  const dim3 parts(parts_of(o.batch, rows * cols / 8), static_cast<unsigned>(o.batch));
  hipLaunchKernelGGL(k_square_sums, parts, dim3(kNormThreads), 0, stream, s);
  hipLaunchKernelGGL(k_split, parts, dim3(kNormThreads), 0, stream, s);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;

  const int64_t xrow = 2 * l.cols, xmat = l.rows * xrow, arow = 2 * l.m, amat = l.m * arow;
  BatchedParams gram{};  // A = X X^T or X^T X
  gram.batch = static_cast<int32_t>(o.batch);
  gram.M = gram.N = static_cast<int32_t>(l.m);
  gram.K = static_cast<int32_t>(std::max(l.rows, l.cols));
  gram.x_row = gram.w_row = xrow;
  gram.x_mat = gram.w_mat = xmat;
  gram.out = at(l.a);
  gram.out_row = arow;
  gram.out_mat = amat;
  gram.alpha = kAScale / (kXScale * kXScale);

  BatchedParams poly = gram;  // B = b A + c A A
  poly.K = static_cast<int32_t>(l.m);
  poly.x = poly.w = ws + l.a;
  poly.x_row = poly.w_row = poly.in_row = arow;
  poly.x_mat = poly.w_mat = poly.in_mat = amat;
  poly.in = at(l.a);
  poly.out = at(l.b);
  poly.alpha = o.c / (kAScale * kAScale);
  poly.beta = o.b / kAScale;

  BatchedParams next = poly;  // X <- a X + B X or a X + X B
  next.M = static_cast<int32_t>(l.rows);
  next.N = static_cast<int32_t>(l.cols);
  next.in_row = next.out_row = xrow;
  next.in_mat = next.out_mat = xmat;
  next.in2 = next.out2 = at(l.lo);
  next.alpha = 1.0f / kXScale;
  next.beta = o.a;

  for (int step = 0; step < o.steps; ++step) {
    const uint8_t *x = ws + l.hi[step & 1];
    gram.x = gram.w = x;
    e = tall ? launch_batched<true, true, kEpiGram>(gram, stream) : launch_batched<false, false, kEpiGram>(gram, stream);
    if (e != hipSuccess) return e;
    e = launch_batched<false, false, kEpiPoly>(poly, stream);
    if (e != hipSuccess) return e;
    next.in = reinterpret_cast<const uint16_t *>(x);
    next.out = at(l.hi[(step + 1) & 1]);
    if (step + 1 == o.steps) {
      next.M = static_cast<int32_t>(rows);
      next.N = static_cast<int32_t>(cols);
      next.out = o.out;
      next.out_row = 2 * cols;
      next.out_mat = 2 * rows * cols;
    }
    // tall: rows of X against rows of B, which is symmetric; else rows of B against columns of X
    const uint8_t *b = ws + l.b;
    next.x = tall ? x : b;
    next.x_row = tall ? xrow : arow;
    next.x_mat = tall ? xmat : amat;
    next.w = tall ? b : x;
    next.w_row = tall ? arow : xrow;
    next.w_mat = tall ? amat : xmat;
    // The last step's X is hi alone: what its rounding adds is multiplied by a
    // once (0.05%), and neither written nor read lo is 2 of a call's 19 passes
    // over a matrix of X's size.
    const int epi = o.steps == 1 ? kEpiOnly : step + 1 == o.steps ? kEpiLast : step + 2 == o.steps ? kEpiRound : kEpiNext;
    e = tall ? launch_next<false>(epi, next, stream) : launch_next<true>(epi, next, stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// Whether a matrix fits one workgroup's LDS, and in which kernel.
constexpr int kSmallLds[] = {32640, 81792, 163712};  // five, two or one workgroup a CU, with the partial sums

bool small(int64_t rows, int64_t cols) {
  const int64_t mr = (std::min(rows, cols) + 31) / 32, np = (std::max(rows, cols) + 31) / 32 * 32;
  return mr <= 4 && small_orthogonal_lds(mr, np) <= kSmallLds[2];
}

template <int MR, int CLASS>
hipError_t launch_small(const SmallOrthogonalParams &p, int64_t batch, hipStream_t stream) {
  if constexpr (small_orthogonal_lds(MR, 32 * MR) <= kSmallLds[CLASS]) {
    // Eight waves where a CU has one matrix (one of 128 x 224 60 us with four, so 37;
    // one of 32 x 224 16 and 12; sixteen 67 and 12), four where it has several (2000
    // of 96 x 128 192 with eight, so 149).
    constexpr int MANY = CLASS == 2 ? 8 : 4, FEW = 8;
    const dim3 grid(static_cast<unsigned>(batch));
    if (batch <= 256) hipLaunchKernelGGL((k_orthogonal_small<MR, kSmallLds[CLASS], FEW>), grid, dim3(64 * FEW), 0, stream, p);
    else hipLaunchKernelGGL((k_orthogonal_small<MR, kSmallLds[CLASS], MANY>), grid, dim3(64 * MANY), 0, stream, p);
    return hipGetLastError();
  }
  return hipErrorInvalidConfiguration;  // no such size
}

template <int MR>
hipError_t launch_small(const SmallOrthogonalParams &p, int64_t batch, hipStream_t stream) {
  const int64_t need = small_orthogonal_lds(MR, p.np);
  if (need <= kSmallLds[0]) return launch_small<MR, 0>(p, batch, stream);
  if (need <= kSmallLds[1]) return launch_small<MR, 1>(p, batch, stream);
  return launch_small<MR, 2>(p, batch, stream);
}

SmallOrthogonalParams small_params(const OrthogonalLaunch &o, int64_t np) {
  SmallOrthogonalParams p{};
  p.g = o.g;
  p.out = o.out;
  p.f32 = o.g_f32;
  p.tall = o.rows > o.cols;
  p.rows = static_cast<int32_t>(o.rows);
  p.cols = static_cast<int32_t>(o.cols);
  p.np = static_cast<int32_t>(np);
  p.steps = o.steps;
  p.a = o.a;
  p.b = o.b;
  p.c = o.c;
  p.eps = o.eps;
  return p;
}

hipError_t launch_small(const OrthogonalLaunch &o, hipStream_t stream) {
  const SmallOrthogonalParams p = small_params(o, (std::max(o.rows, o.cols) + 31) / 32 * 32);
  switch ((std::min(o.rows, o.cols) + 31) / 32) {
    case 1: return launch_small<1>(p, o.batch, stream);
    case 2: return launch_small<2>(p, o.batch, stream);
    case 3: return launch_small<3>(p, o.batch, stream);
    default: return launch_small<4>(p, o.batch, stream);
  }
}

// Slabs of a matrix with a short side of up to 128 rows that is no small one.
struct Slabs {
  int64_t mr, np, slabs;
  int64_t x, gram[2], partial, bytes;  // workspace
};

// Columns of a slab, by 32 mr rows: two workgroups a CU, from 96 rows on one.
// For few matrices, half and (what LDS holds) twice as many beside them: one 32 x
// 2048 39 us, 45 and 44; one 64 x 1024 45, 53 and 46; one 96 x 1024 67, 84 and 67;
// one 128 x 512 68, 74 and 73 (192).  With many matrices twice as many are better,
// since every slab reads the parts of all: 256 of 32 x 2048 238, 376 and 184, of
// 64 x 2048 790, 2000 and 525; and so they are for long ones (one 32 x 8192 71,
// 109 and 61).  One width stands for all of them.
constexpr int64_t kSlabColumns[] = {0, 256, 128, 128, 128};

Slabs slabs_of(int64_t batch, int64_t rows, int64_t cols) {
  Slabs l{};
  l.mr = (std::min(rows, cols) + 31) / 32;
  l.np = kSlabColumns[l.mr];
  l.slabs = (std::max(rows, cols) + l.np - 1) / l.np;
  const int64_t gram = up256(4 * batch * l.slabs * 32 * l.mr * 32 * l.mr);
  l.gram[0] = up256(4 * batch * l.slabs * 32 * l.mr * l.np);
  l.gram[1] = l.gram[0] + gram;
  l.partial = l.gram[1] + gram;
  l.bytes = l.partial + up256(8 * batch * parts_of(batch, rows * cols / 8));
  return l;
}

// By tiles a short side is padded to 128, and a step takes three launches; in
// slabs every one of them makes B anew.  Five steps of one 32 x 2048 127 us by
// tiles, 40 in slabs; of 256 903 and 240; of one 64 x 2048 125 and 58, of 256
// 925 and 796; of one 128 x 512 95 and 68, of 16 96 and 83, but of 64 114 and 124.
bool in_slabs(int64_t batch, int64_t rows, int64_t cols) {
  const int64_t mr = (std::min(rows, cols) + 31) / 32;
  if (mr > 4 || small(rows, cols)) return false;
  const int64_t slabs = slabs_of(1, rows, cols).slabs;
  return mr <= 2 ? slabs <= 32 : batch * slabs <= 128 && slabs <= 16;
}

// Matrices of a pass: in as few even passes as keep the workspace at 2.7 GB.
// (256 matrices of 1024 x 2048 take as long in two passes as in one.)
int64_t pass_of(int64_t batch, int64_t rows, int64_t cols) {
  const int64_t most = std::max<int64_t>(1, (int64_t(5) << 29) / (in_slabs(batch, rows, cols) ? slabs_of(1, rows, cols).bytes : layout(1, rows, cols).bytes));
  const int64_t passes = (batch + most - 1) / most;
  return (batch + passes - 1) / passes;
}

template <int MR>
hipError_t launch_slabs(const OrthogonalLaunch &o, hipStream_t stream) {
  constexpr int CLASS = MR <= 2 ? 1 : 2;
  static_assert(small_orthogonal_lds(MR, kSlabColumns[MR]) <= kSmallLds[CLASS], "a slab has to fit");
  const Slabs l = slabs_of(o.batch, o.rows, o.cols);
  uint8_t *ws = static_cast<uint8_t *>(o.ws);
  SplitParams s{};
  s.g = o.g;
  s.f32 = o.g_f32;
  s.rows = static_cast<int32_t>(o.rows);
  s.row_units = static_cast<int32_t>(o.cols / 8);
  s.partial = reinterpret_cast<double *>(ws + l.partial);
  const int parts = parts_of(o.batch, o.rows * o.cols / 8);
  hipLaunchKernelGGL(k_square_sums, dim3(parts, static_cast<unsigned>(o.batch)), dim3(kNormThreads), 0, stream, s);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  SlabParams p{};
  p.m = small_params(o, l.np);
  p.slabs = static_cast<int32_t>(l.slabs);
  p.parts = parts;
  p.partial = s.partial;
  p.x = reinterpret_cast<uint4 *>(ws);
  for (p.phase = 0; p.phase <= o.steps; ++p.phase) {
    p.gram = reinterpret_cast<const float4 *>(ws + l.gram[(p.phase + 1) & 1]);
    p.next_gram = reinterpret_cast<float4 *>(ws + l.gram[p.phase & 1]);
    hipLaunchKernelGGL((k_orthogonal_slab<MR, kSmallLds[CLASS], 8>), dim3(static_cast<unsigned>(o.batch * l.slabs)), dim3(512), 0,
                       stream, p);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_slabs(const OrthogonalLaunch &o, hipStream_t stream) {
  switch ((std::min(o.rows, o.cols) + 31) / 32) {
    case 1: return launch_slabs<1>(o, stream);
    case 2: return launch_slabs<2>(o, stream);
    case 3: return launch_slabs<3>(o, stream);
    default: return launch_slabs<4>(o, stream);
  }
}

}  // namespace

size_t orthogonalize_ws_bytes(int64_t batch, int64_t rows, int64_t cols) {
  if (small(rows, cols)) return 0;
  if (in_slabs(batch, rows, cols)) return static_cast<size_t>(slabs_of(pass_of(batch, rows, cols), rows, cols).bytes);
  return static_cast<size_t>(layout(pass_of(batch, rows, cols), rows, cols).bytes);
}

hipError_t launch_orthogonalize(const OrthogonalLaunch &o, hipStream_t stream) {
  if (small(o.rows, o.cols)) return launch_small(o, stream);
  const int64_t pass = pass_of(o.batch, o.rows, o.cols), elems = o.rows * o.cols;
  for (int64_t first = 0; first < o.batch; first += pass) {
    OrthogonalLaunch part = o;
    part.batch = std::min(pass, o.batch - first);
    part.g = static_cast<const uint8_t *>(o.g) + first * elems * (o.g_f32 ? 4 : 2);
    part.out = o.out + first * elems;
    const hipError_t e = in_slabs(o.batch, o.rows, o.cols) ? launch_slabs(part, stream) : launch_pass(part, stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace quads
