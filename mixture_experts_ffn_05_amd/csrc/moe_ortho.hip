// Update of a weight by the orthogonalised momentum of its gradient.
//
// With G the gradient (or the momentum's step) of a matrix, X0 = G / (|G|_F +
// eps), transposed if it has more rows than columns, and per step (a, b, c)
//
//   A = X X^T,   B = b A + c A A,   X <- a X + B X
//
// which applies a x + b x^3 + c x^5 to X's singular values and leaves its singular
// vectors: after a few steps all singular values are near 1 (Newton-Schulz
// iteration with a quintic).  out = keep out + scale X.
//
// The products are fp16 MFMAs on dense tiles (moe_dense.h) with power-of-two
// factors that keep every operand in fp16's range: X's singular values are at most
// 1 at the start, and the host bounds them, A and B from step to step.  fp16 and not
// bf16: the rate is the same and the rounding an eighth.
//
// What the roundings cost.  Small singular values grow by a^steps, and noise that is
// added to X at the scale of its strong directions grows with them: X in one fp16
// gives an error of 0.02 on a matrix of 8 strong directions over noise 0.05 (m = 512,
// n = 704), as gradients are.  But only the term a X carries that noise: a rounded
// factor of X X^T, of A A and of B X changes the polynomial a little and adds nothing
// outside the directions that it acts on.  So X is kept as the sum of two fp16 planes,
// of which the products take the first and a X takes both: 0.0003 there, 0.0010 over
// noise of a tenth, 0.0015 on a random matrix, where the store of a bf16 result alone
// is off by 0.0017 (in quadrature: 0.0020 to 0.0024).  The products cost what one
// fp16 costs; taking both planes in them (three products for one of X X^T, two of B X)
// would bring 0.0010 to 0.0008.  The last step adds no noise that grows: one plane.
// A bf16 gradient is exact in one plane.  A float32 result takes both planes of X, A
// and B in every product, and so do many steps (ortho_deep).  Sums are fp32, the norm fp64.  Matrices of up to 128 rows go
// another way (moe_ortho_narrow.hip), where the errors would not average out either.
#include "moe_ortho.h"

#include <math.h>

namespace moe {
namespace {

constexpr int kOrthoChunks = 1024;   // partial sums of squares of all matrices, or of each if there are more

// The momentum's step and partial sums of the update's squares.  blockIdx.y: the
// matrix; a workgroup takes a run of its rows.
template <typename T, bool VEC>
__global__ __launch_bounds__(256) void ortho_norm(OrthoIn in, int rows_per, double* __restrict__ part) {
  __shared__ double s_sum[4];
  const int mat = blockIdx.y, b = mat / in.parts, j = mat % in.parts;
  const int r0 = blockIdx.x * rows_per, rows = min(rows_per, in.M - r0);
  const int oct = (in.N + 7) / 8;
  double sum = 0.0;
  for (int64_t i = threadIdx.x; i < (int64_t)rows * oct; i += 256) {
    const int r = (int)(i / oct), c = 8 * (int)(i % oct);
    float u[8];
    ortho_update8<T, VEC, true>(in, ((int64_t)b * in.M + r0 + r) * in.parts * in.N + (int64_t)j * in.N + c, in.N - c,
                                u);
    float sq = 0.f;   // eight squares in fp32, their sums in fp64
#pragma unroll
    for (int q = 0; q < 8; ++q) sq = fmaf(u[q], u[q], sq);
    sum += (double)sq;
  }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) sum += __shfl_xor(sum, d, kWave);
  if ((threadIdx.x & 63) == 0) s_sum[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0) part[(int64_t)mat * gridDim.x + blockIdx.x] = s_sum[0] + s_sum[1] + s_sum[2] + s_sum[3];
}

// The update of every matrix as fp16 planes hi (and lo) [m, n], m <= n, zero in
// the padding, times 2^e so that its Frobenius norm lies in [2^14, 2^15); rho =
// 1 / ((norm + eps) 2^e) makes it X0.  64 x 64 tiles, through LDS where it is
// transposed.
template <typename T, bool VEC>
__global__ __launch_bounds__(256) void ortho_planes(OrthoIn in, const double* __restrict__ part, int chunks, float eps,
                                                    _Float16* __restrict__ hi, _Float16* __restrict__ lo, int mp,
                                                    int np, int64_t stride, float* __restrict__ rho) {
  __shared__ float s_t[64][65];
  __shared__ double s_norm;
  const int mat = blockIdx.y, b = mat / in.parts, j = mat % in.parts, tid = threadIdx.x;
  const bool flip = in.M > in.N;
  if (tid < 64) {
    double v = 0.0;
    for (int c = tid; c < chunks; c += kWave) v += part[(int64_t)mat * chunks + c];
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, kWave);
    if (tid == 0) s_norm = sqrt(v);
  }
  // rows and columns of the gradient that this tile covers, padding included
  const int tc = ((flip ? mp : np) + 63) / 64;
  const int r0 = (blockIdx.x / tc) * 64, c0 = (blockIdx.x % tc) * 64;
  __syncthreads();
  const double norm = s_norm;
  const bool good = norm > 0.0 && norm < 1.0e18;
  int e = good ? 14 - ilogb(norm) : 0;
  e = min(e, 120);
  const float up = ldexpf(1.0f, e);
  if (blockIdx.x == 0 && tid == 0)
    rho[mat] = norm < 1.0e18 ? (float)(1.0 / ldexp(norm + (double)eps, e)) : nanf("");   // eps >= 1e-12: rho^2 fits
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = (tid >> 3) + 32 * i, c = 8 * (tid & 7);
    float u[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (r0 + r < in.M && c0 + c < in.N)
      ortho_update8<T, VEC, false>(
          in, ((int64_t)b * in.M + r0 + r) * in.parts * in.N + (int64_t)j * in.N + c0 + c, in.N - c0 - c, u);
#pragma unroll
    for (int q = 0; q < 8; ++q) s_t[r][c + q] = u[q] * up;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = (tid >> 3) + 32 * i, c = 8 * (tid & 7);
    const int row = (flip ? c0 : r0) + r, col = (flip ? r0 : c0) + c;
    if (row >= mp || col >= np) continue;
    f16x8 h, l;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const float v = flip ? s_t[c + q][r] : s_t[r][c + q];
      h[q] = (_Float16)v;
      l[q] = (_Float16)(v - (float)h[q]);
    }
    const int64_t at = mat * stride + (int64_t)row * np + col;
    *(f16x8*)(hi + at) = h;
    if (lo) *(f16x8*)(lo + at) = l;
  }
}

// One product of every matrix.
struct OrthoProduct {
  const _Float16 *a, *b;
  int64_t a_stride, b_stride;   // between matrices
  int M, N, K, lda, ldb;
  int m_tiles, n_tiles, tiles, mats;
  bool symmetric;
  DensePlanes planes;
  // epilogue, pointers of matrix 0
  _Float16 *hi, *lo;
  const _Float16 *add_hi, *add_lo;
  int64_t out_stride, add_stride;
  float f_acc, f_add;
  float f_diag;
  bool exact;            // symmetric to the bit
  // a second set of products with the same b (matrices from `first` on), or first = mats
  int first;
  const _Float16* a2;
  _Float16 *hi2, *lo2;
  float f_acc2;
  int splits, k_split;   // reduction ranges, and their partial sums [splits, mats, M, N] in fp32
  float* partial;
  const float* rho;   // factor of X0, or null
  int rho_acc;        // its power in the sum's factor (f_add's is 1)
  void* out;
  int64_t ldo;
  int rows, cols, parts;   // of the result, and matrices side by side in out
  float keep;
  bool transposed, out_aligned;
};

// Tile `id` of a matrix: symmetric products' tiles on and below the diagonal row
// by row, others in bands of up to 8 row tiles.
__device__ __forceinline__ DenseUnit ortho_unit(const OrthoProduct& q, int id) {
  DenseUnit t;
  t.split = 0;
  if (q.symmetric) {
    int r = (int)((sqrtf(8.0f * id + 1.0f) - 1.0f) * 0.5f);
    while (r * (r + 1) / 2 > id) --r;
    while ((r + 1) * (r + 2) / 2 <= id) ++r;
    t.mt = r;
    t.nt = id - r * (r + 1) / 2;
  } else {
    const int band = id / (8 * q.n_tiles), in = id % (8 * q.n_tiles);
    const int rows = min(8, q.m_tiles - 8 * band);
    t.mt = 8 * band + in % rows;
    t.nt = in / rows;
  }
  return t;
}

template <class C, bool BCOL, int EPI>
__global__ __launch_bounds__(C::NT, dense_min_waves<C>()) void ortho_product(OrthoProduct q) {
  extern __shared__ __attribute__((aligned(1024))) unsigned char smem[];
  // the XCDs take contiguous runs of tiles, so that one L2 holds a matrix's operands
  const int64_t n = (int64_t)q.tiles * q.mats * q.splits;
  const int64_t per = n / kDXcds, rest = n % kDXcds, x = blockIdx.x % kDXcds;
  const int64_t id = x * per + min(x, rest) + blockIdx.x / kDXcds;
  int mat = (int)(id / q.tiles);
  DenseUnit t = ortho_unit(q, (int)(id % q.tiles));
  DenseProblem p{};
  const bool second = q.splits == 1 && mat >= q.first;
  if (second) mat -= q.first;
  if (q.splits > 1) {
    t.split = mat / q.mats;
    mat %= q.mats;
  }
  p.a = (second ? q.a2 : q.a) + mat * q.a_stride;
  p.b = q.b + mat * q.b_stride;
  p.M = q.M;
  p.N = q.N;
  p.K = q.K;
  p.lda = q.lda;
  p.ldb = q.ldb;
  p.splits = q.splits;
  p.k_split = q.k_split;
  p.partial = q.partial ? q.partial + ((int64_t)t.split * q.mats + mat) * q.M * q.N : nullptr;
  PlanesEpi e{};
  const float rho = q.rho ? q.rho[mat] : 1.0f;
  e.f_acc = (second ? q.f_acc2 : q.f_acc) * (q.rho_acc >= 1 ? rho : 1.0f) * (q.rho_acc >= 2 ? rho : 1.0f);
  e.f_add = q.f_add * rho;
  e.f_diag = q.f_diag;
  e.add_hi = q.add_hi ? q.add_hi + mat * q.add_stride : nullptr;
  e.add_lo = q.add_lo ? q.add_lo + mat * q.add_stride : nullptr;
  if constexpr (EPI == kEPlanes || EPI == kESymmetric) {
    _Float16 *hi = second ? q.hi2 : q.hi, *lo = second ? q.lo2 : q.lo;
    e.hi = hi + mat * q.out_stride;
    e.lo = lo ? lo + mat * q.out_stride : nullptr;
    e.ld = q.N;
    e.exact = q.exact;
  } else {
    e.ld = q.N;
    const int b = mat / q.parts, j = mat % q.parts;
    const int64_t rows = q.transposed ? q.cols : q.rows, cols = q.transposed ? q.rows : q.cols;
    const int64_t at = b * rows * q.ldo + j * cols;
    e.out = (char*)q.out + at * (EPI == kEFinalF32 ? 4 : 2);
    e.ldo = q.ldo;
    e.out_rows = q.rows;
    e.out_cols = q.cols;
    e.keep = q.keep;
    e.transposed = q.transposed;
    e.out_aligned = q.out_aligned;
  }
  dense_tile_at<C, false, BCOL, EPI>(p, t, smem, q.planes, e);
}

// A = factor * the sum of a split X X^T's partial sums, added in order, in planes: one
// 64 x 64 block on or below the diagonal per workgroup, stored at both places.
__global__ __launch_bounds__(256) void ortho_gram_sum(const float* __restrict__ part, int splits, int mats, int mp,
                                                      float f_acc, const float* __restrict__ rho,
                                                      _Float16* __restrict__ hi, _Float16* __restrict__ lo) {
  __shared__ float s_t[64][65];
  const int mat = blockIdx.y, tid = threadIdx.x;
  int br = (int)((sqrtf(8.0f * blockIdx.x + 1.0f) - 1.0f) * 0.5f);
  while (br * (br + 1) / 2 > (int)blockIdx.x) --br;
  while ((br + 1) * (br + 2) / 2 <= (int)blockIdx.x) ++br;
  const int bc = blockIdx.x - br * (br + 1) / 2;
  const float f = rho ? f_acc * rho[mat] * rho[mat] : f_acc;
  const int64_t ps = (int64_t)mats * mp * mp, base = (int64_t)mat * mp * mp;
  auto store = [&](int r, int c, const float (&v)[8]) {
    f16x8 h, l;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      h[q] = (_Float16)v[q];
      l[q] = (_Float16)(v[q] - (float)h[q]);
    }
    *(f16x8*)(hi + base + (int64_t)r * mp + c) = h;
    if (lo) *(f16x8*)(lo + base + (int64_t)r * mp + c) = l;
  };
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = (tid >> 3) + 32 * i, c = 8 * (tid & 7);
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0}, x[8];
    if (64 * br + r < mp && 64 * bc + c < mp) {
#pragma unroll 4
      for (int z = 0; z < splits; ++z) {
        load8(part + z * ps + base + (int64_t)(64 * br + r) * mp + 64 * bc + c, x);
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] += x[q];
      }
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] *= f;
      if (br != bc) store(64 * br + r, 64 * bc + c, v);
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) s_t[r][c + q] = v[q];
  }
  __syncthreads();   // a block on the diagonal is stored from its lower half alone: symmetric to the bit
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int c = (tid >> 3) + 32 * i, r = 8 * (tid & 7);
    float v[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = br == bc ? s_t[max(r + q, c)][min(r + q, c)] : s_t[r + q][c];
    if (64 * bc + c < mp && 64 * br + r < mp) store(64 * bc + c, 64 * br + r, v);
  }
}

// OrthoL's symmetric epilogue spills 97 registers beside its 256 accumulators.
typedef DenseCfg<256, 256, 2, 2, 1, true, true> OrthoL;   // 4 waves of 128 x 128, one workgroup per CU
typedef DenseCfg<128, 128, 2, 2, 1, true, true> OrthoM;   // 4 waves of 64 x 64, two per CU
typedef DenseCfg<64, 64, 2, 1, 4, true, true> OrthoS;     // four groups of 2 waves of 32 x 64, one per CU

// Microseconds per 64-deep slice with one workgroup on a CU and with every slot
// taken, and per tile besides its slices (the store of a tile's results most of
// all).  Measured on symmetric products of 128 matrices of 1408 rows and on single
// ones of 256 to 1024 rows.
struct OrthoShape {
  int side, slots;
  double alone, full, fixed;
};
constexpr OrthoShape kOrthoShapes[3] = {{256, 1, 1.25, 1.25, 24.0}, {128, 2, 0.69, 0.89, 10.0}, {64, 1, 0.18, 0.20, 7.0}};

// The shape with the least time for the tiles of all matrices, in whole rounds.
int ortho_shape(int64_t mats, int M, int N, bool symmetric, int slices, int cu_count) {
  int best = 0;
  double best_us = 1e30;
  for (int i = 0; i < 3; ++i) {
    const OrthoShape& c = kOrthoShapes[i];
    const int64_t mt = (M + c.side - 1) / c.side, nt = (N + c.side - 1) / c.side;
    const int64_t tiles = mats * (symmetric ? mt * (mt + 1) / 2 : mt * nt), slots = (int64_t)c.slots * cu_count;
    const int64_t rounds = (tiles + slots - 1) / slots;
    const double us = rounds * (slices * (tiles <= cu_count ? c.alone : c.full) + c.fixed);
    if (us < best_us) {
      best_us = us;
      best = i;
    }
  }
  return best;
}

template <class C, bool BCOL, int EPI>
hipError_t launch_product(OrthoProduct q, hipStream_t s) {
  static std::atomic<uint64_t> lds_done{0};
  const hipError_t err = allow_lds(reinterpret_cast<const void*>(&ortho_product<C, BCOL, EPI>), C::kLds, lds_done);
  if (err != hipSuccess) return err;
  q.m_tiles = (q.M + C::BM - 1) / C::BM;
  q.n_tiles = (q.N + C::BN - 1) / C::BN;
  q.tiles = q.symmetric ? q.m_tiles * (q.m_tiles + 1) / 2 : q.m_tiles * q.n_tiles;
  hipLaunchKernelGGL((ortho_product<C, BCOL, EPI>), dim3((unsigned)((int64_t)q.tiles * q.mats * q.splits)), dim3(C::NT), C::kLds,
                     s, q);
  return hipGetLastError();
}

template <bool BCOL, int EPI>
hipError_t product(OrthoProduct q, int cu_count, hipStream_t s) {
  if (q.splits <= 1) {
    q.splits = 1;
    q.k_split = (q.K + kDBK - 1) / kDBK * kDBK;
    q.partial = nullptr;
    if (!q.first) q.first = q.mats;
  }
  const int slices = q.planes.count * (q.k_split / kDBK);
  const int shape = ortho_shape((int64_t)q.mats * q.splits, q.M, q.N, q.symmetric, slices, cu_count);
  return shape == 0   ? launch_product<OrthoL, BCOL, EPI>(q, s)
         : shape == 1 ? launch_product<OrthoM, BCOL, EPI>(q, s)
                      : launch_product<OrthoS, BCOL, EPI>(q, s);
}

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

struct OrthoWs {
  int m, n, mp, np, mats;
  bool narrow;           // the other path
  bool gram;             // steps on X0 X0^T
  bool exact_x0, wide;   // X0 in one plane; A and B in two, and every product of both
  int splits, k_split;   // of X0 X0^T (gram)
  int chunks;            // partial sums of squares per matrix
  size_t part, rho, x0, x1, a, b, more, partial, bytes;
  size_t x_plane, a_plane;   // elements of one plane of all matrices
};
// Steps on A alone take (5 steps) 25.5 m^3 products of pairs of planes and 2.5 m^2 n,
// steps on X 7.5 m^2 n and 2.5 m^3: long rows take the former.  They are also the
// more exact for long rows, whose steps on X are off by up to 0.002 below 300 rows.
bool ortho_by_gram(int m, int n) { return n >= 5 * (int64_t)m; }

// Whether the steps may raise the smallest singular values more than 1024 times (five
// steps of a = 3.4: 490, six: 1700).  Steps on A know a singular value s from A's s^2,
// which two planes hold to 2^-22: noise on a zero of A grows by a^2 per step (after
// eight to more than 1, and with the other sign without end), and Q's largest
// elements, up to a^steps, take the digits of the others.  Such steps work on X, whose
// noise grows by a, with both planes in every product.
bool ortho_deep(int steps, const float* coef, const double* sigma) {
  double most = 1.0;
  for (int k = 0; k < steps; ++k) most *= poly_bound(coef + 3 * k, sigma[k]);
  return most > 1024.0;
}

// Partial sums of squares per matrix: enough workgroups to fill the chip, of at least
// 4096 elements each, in whole rows.
int ortho_chunks(int mats, int M, int N) {
  int64_t c = (kOrthoChunks + mats - 1) / mats;
  const int64_t most = ((int64_t)M * N + 4095) / 4096;
  if (c > most) c = most;
  const int rows = (int)((M + c - 1) / c);
  return (M + rows - 1) / rows;
}

OrthoWs ortho_ws(int dt, int out_dt, int batch, int M, int N, int parts, bool momentum, bool deep, int cu_count) {
  OrthoWs w;
  w.m = M < N ? M : N;
  w.n = M < N ? N : M;
  w.mp = (w.m + 7) / 8 * 8;
  w.np = (w.n + 7) / 8 * 8;
  w.mats = batch * parts;
  w.exact_x0 = dt == 1 && !momentum;
  w.wide = out_dt == 0 || deep;
  w.narrow = !w.wide && w.m <= kOrthoNarrow;
  w.gram = !w.wide && !w.narrow && ortho_by_gram(w.m, w.n);
  if (w.narrow) {
    w.bytes = ortho_narrow_workspace_bytes(w.mats, w.m, w.n);
    return w;
  }
  w.x_plane = align256((size_t)w.mats * w.mp * w.np);
  w.a_plane = align256((size_t)w.mats * w.mp * w.mp);
  size_t at = 0;
  w.chunks = ortho_chunks(w.mats, M, N);
  w.part = at;
  at += align256((size_t)w.mats * w.chunks * sizeof(double));
  w.rho = at;
  at += align256((size_t)w.mats * sizeof(float));
  w.x0 = at;
  at += 2 * 2 * w.x_plane;
  w.x1 = at;
  at += w.gram ? 0 : 2 * 2 * w.x_plane;
  const int planes = w.wide || w.gram ? 2 : 1;
  w.a = at;
  at += 2 * planes * w.a_plane;
  w.b = at;
  at += 2 * planes * w.a_plane;
  w.more = at;   // gram: T, and Q twice
  at += w.gram ? 3 * 2 * 2 * w.a_plane : 0;
  // X0 X0^T of few long matrices has few tiles: ranges of at least 8 slices
  const int tiles = (w.mp + 63) / 64, slices = (w.np + kDBK - 1) / kDBK;
  int splits = w.gram ? (int)((int64_t)cu_count / ((int64_t)tiles * (tiles + 1) / 2 * w.mats)) : 1;
  if (splits > slices / 8) splits = slices / 8;
  if (splits > 32) splits = 32;
  if (splits < 1) splits = 1;
  const int per = (slices + splits - 1) / splits;
  w.splits = (slices + per - 1) / per;
  w.k_split = per * kDBK;
  w.partial = at;
  at += w.splits > 1 ? align256((size_t)w.splits * w.mats * w.mp * w.mp * 4) : 0;
  w.bytes = at;
  return w;
}

template <typename T>
hipError_t ortho_prepare(const OrthoIn& in, const OrthoWs& w, char* base, float eps, hipStream_t s) {
  const bool vec = in.N % 8 == 0 && (uintptr_t)in.grad % 16 == 0 && (uintptr_t)in.momentum % 16 == 0;
  double* part = (double*)(base + w.part);
  _Float16* hi = (_Float16*)(base + w.x0);
  _Float16* lo = w.exact_x0 ? nullptr : hi + w.x_plane;
  const int chunks = w.chunks, rows_per = (in.M + chunks - 1) / chunks;
  const int rp = in.M > in.N ? w.np : w.mp, cp = in.M > in.N ? w.mp : w.np;
  const dim3 g1(chunks, w.mats), g2(((rp + 63) / 64) * ((cp + 63) / 64), w.mats);
  float* rho = (float*)(base + w.rho);
  if (vec) {
    hipLaunchKernelGGL((ortho_norm<T, true>), g1, dim3(256), 0, s, in, rows_per, part);
    hipLaunchKernelGGL((ortho_planes<T, true>), g2, dim3(256), 0, s, in, part, chunks, eps, hi, lo, w.mp, w.np,
                       (int64_t)w.mp * w.np, rho);
  } else {
    hipLaunchKernelGGL((ortho_norm<T, false>), g1, dim3(256), 0, s, in, rows_per, part);
    hipLaunchKernelGGL((ortho_planes<T, false>), g2, dim3(256), 0, s, in, part, chunks, eps, hi, lo, w.mp, w.np,
                       (int64_t)w.mp * w.np, rho);
  }
  return hipGetLastError();
}

}  // namespace
}  // namespace moe

namespace moe_launch {

size_t orthogonal_update_workspace_bytes(int dt, int out_dt, int batch, int M, int N, int parts, bool momentum,
                                         int cu_count) {
  const size_t few = moe::ortho_ws(dt, out_dt, batch, M, N, parts, momentum, false, cu_count).bytes;
  const size_t many = moe::ortho_ws(dt, out_dt, batch, M, N, parts, momentum, true, cu_count).bytes;
  return few > many ? few : many;
}

bool orthogonal_bounds(int steps, const float* coef, double* sigma, double* beta) {
  sigma[0] = 1.001;   // the rounded X0
  for (int k = 0; k < steps; ++k) {
    sigma[k + 1] = moe::step_bound(coef + 3 * k, sigma[k]);
    beta[k] = moe::poly_bound(0.0, coef[3 * k + 1], coef[3 * k + 2], sigma[k]);
    if (!(sigma[k + 1] <= 64.0) || !(beta[k] <= 4096.0) || !(fabsf(coef[3 * k]) <= 4096.0f)) return false;
  }
  return true;
}

hipError_t orthogonal_update(int dt, int out_dt, const void* grad, float* momentum, float mu, int nesterov, int batch,
                             int M, int N, int parts, int steps, const float* coef, float eps, float scale, float keep,
                             void* out, void* workspace, int cu_count, hipStream_t s) {
  using namespace moe;
  double sigma[kOrthoMaxSteps + 1], beta[kOrthoMaxSteps];
  if (!orthogonal_bounds(steps, coef, sigma, beta)) return hipErrorInvalidValue;
  const OrthoWs w = ortho_ws(dt, out_dt, batch, M, N, parts, momentum != nullptr, ortho_deep(steps, coef, sigma),
                             cu_count);
  if (w.narrow)
    return ortho_narrow(dt, grad, momentum, mu, nesterov, batch, M, N, parts, steps, coef, sigma, eps, scale, keep, out,
                        workspace, s);
  char* base = (char*)workspace;
  const OrthoIn in{grad, momentum, mu, nesterov, M, N, parts};
  hipError_t err = dt == 1 ? ortho_prepare<bf16_t>(in, w, base, eps, s) : ortho_prepare<float>(in, w, base, eps, s);
  if (err != hipSuccess) return err;
  _Float16* xs[2] = {(_Float16*)(base + w.x0), (_Float16*)(base + w.x1)};
  _Float16 *am = (_Float16*)(base + w.a), *bm = (_Float16*)(base + w.b);
  const float* rho0 = (const float*)(base + w.rho);
  const int64_t xst = (int64_t)w.mp * w.np, ast = (int64_t)w.mp * w.mp;
  const int64_t xp = (int64_t)w.x_plane, ap = (int64_t)w.a_plane;
  OrthoProduct last_product{};   // what every last product shares
  last_product.mats = w.mats;
  last_product.parts = parts;
  last_product.out = out;
  last_product.ldo = (int64_t)parts * N;
  last_product.rows = w.m;
  last_product.cols = w.n;
  last_product.keep = keep;
  last_product.transposed = M > N;
  last_product.out_aligned = N % 8 == 0 && (uintptr_t)out % 16 == 0;
  if (w.gram) {
    _Float16* more = (_Float16*)(base + w.more);
    _Float16 *tm = more, *qm[2] = {more + 2 * ap, more + 4 * ap};
    OrthoProduct q{};
    q.mats = w.mats;
    q.parts = parts;
    q.M = q.N = w.mp;
    q.symmetric = true;
    q.out_stride = q.add_stride = ast;
    // A0 = X0 X0^T
    const float sa0 = f16_scale(sigma[0] * sigma[0]);
    q.a = q.b = xs[0];
    q.a_stride = q.b_stride = xst;
    q.K = q.lda = q.ldb = w.np;
    if (!w.exact_x0) {
      q.planes.count = 3;
      q.planes.b[1] = q.planes.a[2] = xp;
    }
    q.hi = am;
    q.lo = am + ap;
    q.f_acc = sa0;
    q.rho = rho0;
    q.rho_acc = 2;
    q.exact = true;   // or every step feeds the difference back, ten times larger
    if (w.splits > 1) {
      q.splits = w.splits;
      q.k_split = w.k_split;
      q.partial = (float*)(base + w.partial);
    }
    err = product<false, kESymmetric>(q, cu_count, s);
    if (err != hipSuccess) return err;
    if (w.splits > 1) {
      const int blocks = (w.mp + 63) / 64;
      hipLaunchKernelGGL(ortho_gram_sum, dim3(blocks * (blocks + 1) / 2, w.mats), dim3(256), 0, s, q.partial, w.splits,
                         w.mats, w.mp, sa0, rho0, am, am + ap);
      err = hipGetLastError();
      if (err != hipSuccess) return err;
    }
    // the m x m products: both operands in two planes
    q.a_stride = q.b_stride = ast;
    q.K = q.lda = q.ldb = w.mp;
    q.planes.count = 3;
    q.planes.a[0] = q.planes.a[1] = q.planes.b[0] = q.planes.b[2] = 0;
    q.planes.b[1] = q.planes.a[2] = ap;
    q.splits = 0;
    q.partial = nullptr;
    q.rho = nullptr;
    double bound = 1.0;   // of Q
    float sq = 1.0f;
    for (int k = 0; k < steps; ++k) {
      const double poly = poly_bound(coef + 3 * k, sigma[k]);
      bound *= poly;
      const float sa = f16_scale(sigma[k] * sigma[k]), sp = f16_scale(poly), sqn = f16_scale(bound);
      const float st = f16_scale(fmax(poly, sigma[k] * sigma[k + 1]));
      // P = a I + b A + c A A; the first one is Q
      _Float16* pm = k == 0 ? qm[0] : bm;
      OrthoProduct u = q;
      u.a = u.b = am;
      u.add_hi = am;
      u.add_lo = am + ap;
      u.hi = pm;
      u.lo = pm + ap;
      u.f_acc = coef[3 * k + 2] * sp / (sa * sa);
      u.f_add = coef[3 * k + 1] * sp / sa;
      u.f_diag = coef[3 * k] * sp;
      u.exact = false;
      err = product<false, kESymmetric>(u, cu_count, s);
      if (err != hipSuccess) return err;
      // T = A P and Q <- Q P in one launch
      u = q;
      u.b = pm;
      const bool t_wanted = k + 1 < steps, q_wanted = k > 0;
      _Float16 *q_now = qm[(k + 1) & 1], *q_next = qm[k & 1];
      u.a = t_wanted ? am : q_now;
      u.hi = t_wanted ? tm : q_next;
      u.lo = u.hi + ap;
      u.f_acc = t_wanted ? st / (sa * sp) : sqn / (sq * sp);
      u.first = w.mats;
      u.exact = false;
      if (t_wanted && q_wanted) {
        u.mats = 2 * w.mats;
        u.a2 = q_now;
        u.hi2 = q_next;
        u.lo2 = q_next + ap;
        u.f_acc2 = sqn / (sq * sp);
      }
      if (t_wanted || q_wanted) err = product<false, kESymmetric>(u, cu_count, s);
      if (err != hipSuccess) return err;
      sq = k == 0 ? sp : sqn;
      if (!t_wanted) break;
      // A <- T P
      u = q;
      u.a = tm;
      u.b = pm;
      u.hi = am;
      u.lo = am + ap;
      u.f_acc = f16_scale(sigma[k + 1] * sigma[k + 1]) / (st * sp);
      err = product<false, kESymmetric>(u, cu_count, s);
      if (err != hipSuccess) return err;
    }
    // out = keep out + scale Q X0
    OrthoProduct f = last_product;
    f.a = qm[(steps - 1) & 1];
    f.a_stride = ast;
    f.b = xs[0];
    f.b_stride = xst;
    f.M = f.K = f.lda = w.mp;
    f.N = f.ldb = w.np;
    f.planes.count = w.exact_x0 ? 2 : 3;
    f.planes.a[1] = ap;
    if (!w.exact_x0) f.planes.b[2] = xp;
    f.f_acc = scale / sq;
    f.rho = rho0;
    f.rho_acc = 1;
    return product<true, kEFinal>(f, cu_count, s);
  }
  for (int k = 0; k < steps; ++k) {
    const float a = coef[3 * k], b = coef[3 * k + 1], c = coef[3 * k + 2];
    const bool first = k == 0, last = k == steps - 1;
    const bool two = first ? !w.exact_x0 : w.wide || !last;   // X's planes
    const float* rho = first ? rho0 : nullptr;
    // X is stored times sx (X0: rho makes it X), A times sa, B times sb
    const float sx = first ? 1.0f : f16_scale(sigma[k]), sa = f16_scale(sigma[k] * sigma[k]), sb = f16_scale(beta[k]);
    const float sn = last ? scale : f16_scale(sigma[k + 1]);
    _Float16 *x = xs[k & 1], *xn = xs[~k & 1];
    OrthoProduct q{};
    q.mats = w.mats;
    q.parts = parts;
    // A = X X^T
    q.a = q.b = x;
    q.a_stride = q.b_stride = xst;
    q.M = q.N = w.mp;
    q.K = q.lda = q.ldb = w.np;
    q.symmetric = true;
    if (w.wide && two) {
      q.planes.count = 3;
      q.planes.b[1] = q.planes.a[2] = xp;
    }
    q.hi = am;
    q.lo = w.wide ? am + ap : nullptr;
    q.out_stride = ast;
    q.f_acc = sa / (sx * sx);
    q.rho = rho;
    q.rho_acc = 2;
    err = product<false, kESymmetric>(q, cu_count, s);
    if (err != hipSuccess) return err;
    // B = b A + c A A
    q.a = q.b = am;
    q.a_stride = q.b_stride = ast;
    q.K = q.lda = q.ldb = w.mp;
    q.planes = DensePlanes{};
    if (w.wide) {
      q.planes.count = 3;
      q.planes.b[1] = q.planes.a[2] = ap;
    }
    q.add_hi = am;
    q.add_lo = w.wide ? am + ap : nullptr;
    q.add_stride = ast;
    q.hi = bm;
    q.lo = w.wide ? bm + ap : nullptr;
    q.rho = nullptr;
    q.f_acc = c * sb / (sa * sa);
    q.f_add = b * sb / sa;
    err = product<false, kESymmetric>(q, cu_count, s);
    if (err != hipSuccess) return err;
    // X <- a X + B X
    q.a = bm;
    q.b = x;
    q.b_stride = xst;
    q.N = q.ldb = w.np;
    q.symmetric = false;
    q.planes = DensePlanes{};
    if (w.wide) {
      q.planes.count = two ? 3 : 2;
      q.planes.a[two ? 2 : 1] = ap;
      if (two) q.planes.b[1] = xp;
    }
    q.add_hi = x;
    q.add_lo = two ? x + xp : nullptr;
    q.add_stride = xst;
    q.rho = rho;
    q.rho_acc = 1;
    q.f_acc = sn / (sb * sx);
    q.f_add = a * sn / sx;
    if (!last) {
      q.hi = xn;
      q.lo = w.wide || k + 2 < steps ? xn + xp : nullptr;
      q.out_stride = xst;
      err = product<true, kEPlanes>(q, cu_count, s);
    } else {
      q.out = last_product.out;
      q.ldo = last_product.ldo;
      q.rows = last_product.rows;
      q.cols = last_product.cols;
      q.keep = last_product.keep;
      q.transposed = last_product.transposed;
      q.out_aligned = last_product.out_aligned;
      err = out_dt == 0 ? product<true, kEFinalF32>(q, cu_count, s) : product<true, kEFinal>(q, cu_count, s);
    }
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

}  // namespace moe_launch
