// Orthogonalised update of matrices with at most 128 rows (or columns): a router
// weight, a narrow projection.
//
// Every step's polynomial is one of A0 = X0 X0^T, and all of them commute, so with
// P = a I + b A + c A A
//
//   A <- P A P,   Q <- Q P      (A0 and I before the first step)
//   X after all steps = Q X0
//
// and the long dimension is read twice: once for A0, once for Q X0.  The steps in
// between are products of m x m matrices (m rounded up to 32, 64 or 128), which one
// workgroup keeps in LDS and registers: four launches instead of seventeen, and no
// chain of 2048-long reductions per step.  (A 2048 x 60 matrix: 41 us, 354 by the
// general path.)  For bf16 results of steps that are not too many (ortho_deep).
//
//  * A0 is squared singular values: rounding it to 11 bits would lose all below a
//    64th of the largest.  It is taken by fp32 MFMAs (v_mfma_f32_16x16x4_f32) of the
//    update itself; its trace is the Frobenius norm's square, so the norm needs no
//    pass of its own.
//  * The m x m products are fp16 MFMAs of operands in two planes (22 bits), three
//    products each; fp32 MFMAs would take five times as long.  What rounds A in the
//    first steps is added to the small squared singular values and grows twelvefold
//    per step: where one direction stands over the others by a factor of 100 and more,
//    the result of 33 rows and more is off by up to 8e-4 (random matrices: 2e-6); a
//    bf16 result's own rounding is 1.7e-3.
//  * Fewer rows leave that noise fewer elements to average over (2 rows: 5.6e-3).  Up
//    to 32 rows A0 and the steps are fp64 MFMAs (v_mfma_f64_16x16x4_f64), which need
//    no planes and no scales: below 3e-4 for any of them, at 5 us more (2048 x 8: 26
//    us, 21 in planes).
//  * Every matrix is symmetric, so a product's second operand is read by rows, like
//    its first; the first one is a wave's own 16 rows and never leaves its registers.
//    A product is then X Y^T, and an A that is not symmetric to the bit would feed its
//    roundings' difference back, ten times larger in every step (an error of 0.02
//    after five): A is made symmetric before each step.
#include "moe_ortho.h"

namespace moe {
namespace {

constexpr int kTile = 64;         // of the long dimension
constexpr int kGramChunks = 32;   // partial sums of A0, at most
// A wave has 16 rows of a 64 or 128 row matrix (four waves at least).
template <int MT>
constexpr int narrow_threads() { return MT <= 64 ? 256 : 4 * MT; }
constexpr float kNormMost = 1e18f;
// A0's type: see the head of the file.
template <int MT>
using GramSum = std::conditional_t<MT <= 32, double, float>;
typedef double f64x4 __attribute__((ext_vector_type(4)));

struct NarrowSizes {
  int m, n;    // short and long side
  int tiles;   // of the long side
  int chunks, per;
};

// The update's octet `i` of tile `l0`: eight elements that lie together in memory,
// at index `at` of the gradient, and where they go in LDS: [long][short].
struct Octet {
  int64_t at;
  int valid;        // elements that exist (0: none)
  int lds, step;    // first LDS element, distance between elements
};
template <int MT>
__device__ __forceinline__ Octet octet(const OrthoIn& in, int mat, int l0, int i) {
  const int b = mat / in.parts, j = mat % in.parts;
  const int64_t base = (int64_t)b * in.M * in.parts * in.N + (int64_t)j * in.N;
  Octet o;
  if (in.M > in.N) {   // rows are the long side
    const int r = i / (MT / 8), c = 8 * (i % (MT / 8));
    o.at = base + (int64_t)(l0 + r) * in.parts * in.N + c;
    o.valid = l0 + r < in.M ? in.N - c : 0;
    o.lds = r * (MT + 1) + c;
    o.step = 1;
  } else {
    const int r = i / (kTile / 8), c = 8 * (i % (kTile / 8));
    o.at = base + (int64_t)r * in.parts * in.N + l0 + c;
    o.valid = r < in.M ? in.N - (l0 + c) : 0;
    o.lds = c * (MT + 1) + r;
    o.step = MT + 1;
  }
  return o;
}

template <typename T, bool VEC, int MT, bool FIRST>
__device__ __forceinline__ void load_tile(const OrthoIn& in, int mat, int l0, float* s_u) {
#pragma unroll
  for (int i = 0; i < MT * kTile / 8 / narrow_threads<MT>(); ++i) {
    const Octet o = octet<MT>(in, mat, l0, threadIdx.x + narrow_threads<MT>() * i);
    float u[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (o.valid > 0) ortho_update8<T, VEC, FIRST>(in, o.at, o.valid, u);
#pragma unroll
    for (int q = 0; q < 8; ++q) s_u[o.lds + q * o.step] = u[q];
  }
}

// Partial sums of A0: blockIdx.x a run of tiles, blockIdx.y the matrix; a wave takes
// 16 rows of the sums.  The momentum takes its step here.
template <typename T, bool VEC, int MT>
__global__ __launch_bounds__(narrow_threads<MT>()) void narrow_gram(OrthoIn in, NarrowSizes z,
                                                                   GramSum<MT>* __restrict__ part) {
  __shared__ float s_u[kTile * (MT + 1)];
  constexpr int NB = MT / 16;
  constexpr bool F64 = sizeof(GramSum<MT>) == 8;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, s16 = lane & 15, g = lane >> 4;
  std::conditional_t<F64, f64x4, f32x4> acc[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[b][i] = 0;
  const int t0 = blockIdx.x * z.per, t1 = min(t0 + z.per, z.tiles);
  for (int t = t0; t < t1; ++t) {
    __syncthreads();
    load_tile<T, VEC, MT, true>(in, blockIdx.y, t * kTile, s_u);
    __syncthreads();
    if (wave < NB) {
#pragma unroll
      for (int k = 0; k < kTile; k += 4) {
        const float* row = s_u + (k + g) * (MT + 1) + s16;
        const float a = row[16 * wave];
#pragma unroll
        for (int b = 0; b < NB; ++b)
          if constexpr (F64)
            acc[b] = __builtin_amdgcn_mfma_f64_16x16x4f64((double)row[16 * b], (double)a, acc[b], 0, 0, 0);
          else
            acc[b] = __builtin_amdgcn_mfma_f32_16x16x4f32(row[16 * b], a, acc[b], 0, 0, 0);
      }
    }
  }
  if (wave >= NB) return;
  GramSum<MT>* out = part + ((int64_t)blockIdx.y * z.chunks + blockIdx.x) * MT * MT + (16 * wave + s16) * MT;
#pragma unroll
  for (int b = 0; b < NB; ++b)
    if constexpr (F64) {   // a lane's columns: 4 i + g
#pragma unroll
      for (int i = 0; i < 4; ++i) out[16 * b + 4 * i + g] = acc[b][i];
    } else {
      *(f32x4*)(out + 16 * b + 4 * g) = acc[b];
    }
}

struct NarrowSteps {
  int steps;
  float coef[3 * kOrthoMaxSteps];
  float sa[kOrthoMaxSteps], sp[kOrthoMaxSteps], sq[kOrthoMaxSteps];   // factors of A, P (and P A), Q as stored
};

// A wave's 16 rows of a matrix as the first operand of a product: two planes; lane
// group g holds columns 32 kp + 16 (g % 2) + 8 (g / 2) + [0, 8) of its row.
template <int MT>
struct Strip {
  f16x8 hi[MT / 32], lo[MT / 32];
};
template <int MT>
__device__ __forceinline__ void to_strip(const f32x4 (&v)[MT / 16], float scale, Strip<MT>& s) {
#pragma unroll
  for (int kp = 0; kp < MT / 32; ++kp) {
    float x[8];
    merge_blocks(v[2 * kp], v[2 * kp + 1], x);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] *= scale;
      s.hi[kp][i] = (_Float16)x[i];
      s.lo[kp][i] = (_Float16)(x[i] - (float)s.hi[kp][i]);
    }
  }
}
// The strips of all waves make the matrix in LDS: rows of MT fp16, 16-byte chunks
// XORed by the row; the low plane behind the high one.
template <int MT>
__device__ __forceinline__ int chunk_at(int row, int kp, int g) {
  return row * MT * 2 + (((4 * kp + 2 * (g & 1) + (g >> 1)) ^ (row & (MT / 8 - 1))) * 16);
}
template <int MT>
__device__ __forceinline__ void put_strip(const Strip<MT>& s, int row, int g, unsigned char* buf) {
#pragma unroll
  for (int kp = 0; kp < MT / 32; ++kp) {
    *(f16x8*)(buf + chunk_at<MT>(row, kp, g)) = s.hi[kp];
    *(f16x8*)(buf + MT * MT * 2 + chunk_at<MT>(row, kp, g)) = s.lo[kp];
  }
}
// An element of the matrix in LDS.
template <int MT>
__device__ __forceinline__ float stored_at(const unsigned char* buf, int row, int col) {
  const unsigned char* p = buf + row * MT * 2 + (((col >> 3) ^ (row & (MT / 8 - 1))) * 16) + (col & 7) * 2;
  return (float)*(const _Float16*)p + (float)*(const _Float16*)(p + MT * MT * 2);
}
// A wave's 16 rows of x times the (symmetric) matrix in LDS: lane: row lane % 16,
// columns 16 b + 4 (lane / 16) + [0, 4).
template <int MT>
__device__ __forceinline__ void strip_product(const Strip<MT>& x, const unsigned char* buf, int lane, float scale,
                                              f32x4 (&acc)[MT / 16]) {
  const int s16 = lane & 15, g = lane >> 4;
#pragma unroll
  for (int b = 0; b < MT / 16; ++b) {
    f32x4 c{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int kp = 0; kp < MT / 32; ++kp) {
      const f16x8 h = *(const f16x8*)(buf + chunk_at<MT>(16 * b + s16, kp, g));
      const f16x8 l = *(const f16x8*)(buf + MT * MT * 2 + chunk_at<MT>(16 * b + s16, kp, g));
      c = __builtin_amdgcn_mfma_f32_16x16x32_f16(h, x.hi[kp], c, 0, 0, 0);
      c = __builtin_amdgcn_mfma_f32_16x16x32_f16(h, x.lo[kp], c, 0, 0, 0);
      c = __builtin_amdgcn_mfma_f32_16x16x32_f16(l, x.hi[kp], c, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[b][i] = c[i] * scale;
    // or every block's reads are hoisted, and 221 registers spilt in place of 48
    if (MT > 64 && b % 2) __builtin_amdgcn_sched_barrier(0);
  }
}

// A0 from its partial sums, added in order into the first, an element per thread.  (In
// the workgroup of the steps, 32 sums of a 64 row matrix took 14 us of 32; here 4.)
template <int MT>
__global__ __launch_bounds__(256) void narrow_sum(GramSum<MT>* __restrict__ part, int chunks) {
  GramSum<MT>* p = part + (int64_t)blockIdx.y * chunks * MT * MT + blockIdx.x * 256 + threadIdx.x;
  GramSum<MT> v = 0;
#pragma unroll 16
  for (int c = 0; c < chunks; ++c) v += p[(int64_t)c * MT * MT];
  *p = v;
}

// All steps of one matrix: A0 in, Q / (norm + eps) out.
template <int MT>
__global__ __launch_bounds__(MT * 4) void narrow_steps(const float* __restrict__ part, int chunks, float eps,
                                                       NarrowSteps st, float* __restrict__ q_out) {
  constexpr int NB = MT / 16;
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  unsigned char *s_a = smem, *s_p = smem + MT * MT * 4;   // A and P, two planes each
  __shared__ float s_trace[NB];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, s16 = lane & 15, g = lane >> 4;
  const int row = 16 * wave + s16;
  f32x4 av[NB], qv[NB], acc[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b)
    av[b] = *(const f32x4*)(part + (int64_t)blockIdx.x * chunks * MT * MT + row * MT + 4 * g + 16 * b);
  float diag = 0.f;   // of this lane's row, if it holds it
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (16 * b + 4 * g + i == row) diag = av[b][i];
  diag = wave_sum(diag);
  if (lane == 0) s_trace[wave] = diag;
  __syncthreads();
  float trace = 0.f;
#pragma unroll
  for (int w = 0; w < NB; ++w) trace += s_trace[w];
  const float norm = sqrtf(trace);
  const float inv = norm < kNormMost ? 1.0f / (norm + eps) : nanf("");
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int i = 0; i < 4; ++i) av[b][i] = av[b][i] * inv * inv;
  Strip<MT> as, qs, ts;
  for (int k = 0; k < st.steps; ++k) {
    const float a = st.coef[3 * k], b1 = st.coef[3 * k + 1], c1 = st.coef[3 * k + 2];
    const float sa = st.sa[k], sp = st.sp[k];
    // A as stored, what is above the diagonal from below it: see the head of the file
    to_strip<MT>(av, sa, as);
    put_strip<MT>(as, row, g, s_a);
    __syncthreads();
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int col = 16 * b + 4 * g + i;
        av[b][i] = stored_at<MT>(s_a, max(row, col), min(row, col)) * (1.0f / sa);
      }
    to_strip<MT>(av, sa, as);
    __syncthreads();
    put_strip<MT>(as, row, g, s_a);
    __syncthreads();
    strip_product<MT>(as, s_a, lane, 1.0f / (sa * sa), acc);   // A A
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        acc[b][i] = fmaf(c1, acc[b][i], fmaf(b1, av[b][i], 16 * b + 4 * g + i == row ? a : 0.f));   // P
    to_strip<MT>(acc, sp, ts);
    put_strip<MT>(ts, row, g, s_p);
    if (k == 0) {
#pragma unroll
      for (int b = 0; b < NB; ++b) qv[b] = acc[b];
    }
    __syncthreads();
    if (k > 0) strip_product<MT>(qs, s_p, lane, 1.0f / (st.sq[k - 1] * sp), qv);
    to_strip<MT>(qv, st.sq[k], qs);
    if (k + 1 == st.steps) break;
    // A is at most its own bound and P A, P A P are bounded by the next one's
    strip_product<MT>(as, s_p, lane, 1.0f / (sa * sp), acc);    // A P
    to_strip<MT>(acc, st.sp[k], ts);
    strip_product<MT>(ts, s_p, lane, 1.0f / (sp * sp), av);     // A P P
  }
  float* out = q_out + (int64_t)blockIdx.x * MT * MT + row * MT + 4 * g;
#pragma unroll
  for (int b = 0; b < NB; ++b) {
#pragma unroll
    for (int i = 0; i < 4; ++i) qv[b][i] *= inv;
    *(f32x4*)(out + 16 * b) = qv[b];
  }
}

// The same in fp64 for up to 32 rows.  A wave has 16 rows of every matrix in LDS; a
// product's second operand is read by rows of all waves (A and P are symmetric, to
// fp64's roundings: they stay far below what is looked at).
__global__ __launch_bounds__(128) void narrow_steps_f64(const double* __restrict__ part, int chunks, float eps,
                                                        NarrowSteps st, float* __restrict__ q_out) {
  constexpr int MT = 32, NB = MT / 16, LD = MT + 2;
  __shared__ double s_a[MT * LD], s_p[MT * LD], s_q[MT * LD], s_t[MT * LD];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, s16 = lane & 15, g = lane >> 4;
  const int row = 16 * wave + s16;
  const double* a0 = part + (int64_t)blockIdx.x * chunks * MT * MT;
  double trace = 0.0;
  for (int i = 0; i < MT; ++i) trace += a0[i * MT + i];   // in order, the same in every lane
  const double norm = sqrt(trace);
  const double inv = norm < (double)kNormMost ? 1.0 / (norm + (double)eps) : (double)nanf("");
  auto product = [&](const double* x, const double* y, f64x4 (&acc)[NB]) {
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[b] = f64x4{0.0, 0.0, 0.0, 0.0};
#pragma unroll
    for (int k = 0; k < MT; k += 4) {
      const double own = x[row * LD + k + g];
#pragma unroll
      for (int b = 0; b < NB; ++b)
        acc[b] = __builtin_amdgcn_mfma_f64_16x16x4f64(y[(16 * b + s16) * LD + k + g], own, acc[b], 0, 0, 0);
    }
  };
  auto at = [&](int b, int i) { return row * LD + 16 * b + 4 * i + g; };   // a lane's elements of a product
  auto put = [&](double* x, const f64x4 (&v)[NB]) {
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) x[at(b, i)] = v[b][i];
  };
  f64x4 v[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int i = 0; i < 4; ++i) v[b][i] = a0[row * MT + 16 * b + 4 * i + g] * inv * inv;
  put(s_a, v);
  for (int k = 0; k < st.steps; ++k) {
    const double a = st.coef[3 * k], b1 = st.coef[3 * k + 1], c1 = st.coef[3 * k + 2];
    __syncthreads();   // A is whole, and no wave reads the last P any more
    product(s_a, s_a, v);
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[b][i] = fma(c1, v[b][i], fma(b1, s_a[at(b, i)], 16 * b + 4 * i + g == row ? a : 0.0));
    put(s_p, v);
    if (k == 0) put(s_q, v);
    __syncthreads();
    // from here on a wave reads P's rows, and its own rows of the others alone
    if (k > 0) {
      product(s_q, s_p, v);
      wave_lds_fence();
      put(s_q, v);
    }
    if (k + 1 == st.steps) break;
    product(s_a, s_p, v);
    put(s_t, v);
    wave_lds_fence();
    product(s_t, s_p, v);
    put(s_a, v);
  }
  wave_lds_fence();
  float* out = q_out + (int64_t)blockIdx.x * MT * MT + row * MT;
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int i = 0; i < 4; ++i) out[16 * b + 4 * i + g] = (float)(s_q[at(b, i)] * inv);
}

// out = keep out + scale Q U for one tile of the long side; a wave takes 16 of its 64.
template <typename T, bool VEC, int MT>
__global__ __launch_bounds__(narrow_threads<MT>()) void narrow_apply(OrthoIn in, const float* __restrict__ q, float scale, float keep,
                                                    bf16_t* __restrict__ out) {
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  float *s_u = (float*)smem, *s_q = s_u + kTile * (MT + 1);
  constexpr int NB = MT / 16, NT = narrow_threads<MT>();
  // a wave's 16 of the tile's 64, and with eight waves half of the short side
  constexpr int kHalves = NT / 256, NH = NB / kHalves;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, s16 = lane & 15, g = lane >> 4;
  const int l0 = blockIdx.x * kTile, mat = blockIdx.y, strip = wave % 4, b0 = wave / 4 * NH;
  const float* qm = q + (int64_t)mat * MT * MT;
  for (int i = threadIdx.x; i < MT * MT; i += NT) s_q[i / MT * (MT + 1) + i % MT] = qm[i];
  load_tile<T, VEC, MT, false>(in, mat, l0, s_u);
  __syncthreads();
  f32x4 acc[NH];
#pragma unroll
  for (int b = 0; b < NH; ++b) acc[b] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int k = 0; k < MT; k += 4) {
    const float u = s_u[(16 * strip + s16) * (MT + 1) + k + g];
#pragma unroll
    for (int b = 0; b < NH; ++b)   // Q is symmetric
      acc[b] = __builtin_amdgcn_mfma_f32_16x16x4f32(s_q[(k + g) * (MT + 1) + 16 * (b0 + b) + s16], u, acc[b], 0, 0, 0);
  }
  __syncthreads();
#pragma unroll
  for (int b = 0; b < NH; ++b)
#pragma unroll
    for (int i = 0; i < 4; ++i) s_u[(16 * strip + s16) * (MT + 1) + 16 * (b0 + b) + 4 * g + i] = scale * acc[b][i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < MT * kTile / 8 / NT; ++i) {
    const Octet o = octet<MT>(in, mat, l0, threadIdx.x + NT * i);
    if (o.valid <= 0) continue;
    float v[8], p[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = s_u[o.lds + e * o.step];
    bf16_t* d = out + o.at;
    if (VEC && o.valid >= 8) {
      if (keep != 0.f) {
        load8(d, p);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = fmaf(keep, p[e], v[e]);
      }
      store8(d, v);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < o.valid) store_from_f32(d, e, keep != 0.f ? fmaf(keep, load_as_f32(d, e), v[e]) : v[e]);
    }
  }
}

// Rows of the padded Gram matrix.
int narrow_side(int m) { return m <= 32 ? 32 : m <= 64 ? 64 : 128; }

NarrowSizes narrow_sizes(int mats, int m, int n) {
  NarrowSizes z;
  z.m = m;
  z.n = n;
  z.tiles = (n + kTile - 1) / kTile;
  // enough workgroups to fill the chip
  int chunks = (512 + mats - 1) / mats;
  if (chunks > kGramChunks) chunks = kGramChunks;
  if (chunks > z.tiles) chunks = z.tiles;
  z.per = (z.tiles + chunks - 1) / chunks;
  z.chunks = (z.tiles + z.per - 1) / z.per;
  return z;
}

template <typename T, bool VEC, int MT>
hipError_t narrow_t(const OrthoIn& in, const NarrowSizes& z, int mats, const NarrowSteps& st, float eps, float scale,
                    float keep, void* out, void* workspace, hipStream_t s) {
  constexpr int steps_lds = 2 * MT * MT * 4, apply_lds = (kTile + MT) * (MT + 1) * 4;
  static std::atomic<uint64_t> steps_done{0}, apply_done{0};
  hipError_t err = hipSuccess;
  if constexpr (MT > 32) err = allow_lds(reinterpret_cast<const void*>(&narrow_steps<MT>), steps_lds, steps_done);
  if (err == hipSuccess)
    err = allow_lds(reinterpret_cast<const void*>(&narrow_apply<T, VEC, MT>), apply_lds, apply_done);
  if (err != hipSuccess) return err;
  GramSum<MT>* part = (GramSum<MT>*)workspace;
  float* q = (float*)(part + (size_t)mats * z.chunks * MT * MT);
  const dim3 threads(narrow_threads<MT>());
  hipLaunchKernelGGL((narrow_gram<T, VEC, MT>), dim3(z.chunks, mats), threads, 0, s, in, z, part);
  if (z.chunks > 1)
    hipLaunchKernelGGL((narrow_sum<MT>), dim3(MT * MT / 256, mats), dim3(256), 0, s, part, z.chunks);
  if constexpr (MT > 32)
    hipLaunchKernelGGL((narrow_steps<MT>), dim3(mats), dim3(MT * 4), steps_lds, s, part, z.chunks, eps, st, q);
  else
    hipLaunchKernelGGL(narrow_steps_f64, dim3(mats), dim3(MT * 4), 0, s, part, z.chunks, eps, st, q);
  hipLaunchKernelGGL((narrow_apply<T, VEC, MT>), dim3(z.tiles, mats), threads, apply_lds, s, in, q, scale, keep,
                     (bf16_t*)out);
  return hipGetLastError();
}

}  // namespace

size_t ortho_narrow_workspace_bytes(int mats, int m, int n) {
  const NarrowSizes z = narrow_sizes(mats, m, n);
  const size_t mt = narrow_side(m), sum = mt <= 32 ? sizeof(GramSum<32>) : sizeof(GramSum<64>);
  return (size_t)mats * mt * mt * (z.chunks * sum + sizeof(float));
}

hipError_t ortho_narrow(int dt, const void* grad, float* momentum, float mu, int nesterov, int batch, int M, int N,
                        int parts, int steps, const float* coef, const double* sigma, float eps, float scale,
                        float keep, void* out, void* workspace, hipStream_t s) {
  const int mats = batch * parts, m = M < N ? M : N, n = M < N ? N : M, mt = narrow_side(m);
  const NarrowSizes z = narrow_sizes(mats, m, n);
  const OrthoIn in{grad, momentum, mu, nesterov, M, N, parts};
  NarrowSteps st{};
  st.steps = steps;
  double q = 1.0;
  for (int k = 0; k < steps; ++k) {
    for (int i = 0; i < 3; ++i) st.coef[3 * k + i] = coef[3 * k + i];
    const double poly = poly_bound(coef + 3 * k, sigma[k]);
    q *= poly;
    // A <= sigma^2, A P <= sigma times the next sigma
    const double ap = fmax(poly, sigma[k] * sigma[k + 1]);
    st.sa[k] = f16_scale(sigma[k] * sigma[k]);
    st.sp[k] = f16_scale(ap);
    st.sq[k] = f16_scale(q);
  }
  const bool vec = N % 8 == 0 && (uintptr_t)grad % 16 == 0 && (uintptr_t)momentum % 16 == 0 && (uintptr_t)out % 16 == 0;
#define MOE_NARROW(T, V)                                                                                 \
  (mt == 32   ? narrow_t<T, V, 32>(in, z, mats, st, eps, scale, keep, out, workspace, s)                  \
   : mt == 64 ? narrow_t<T, V, 64>(in, z, mats, st, eps, scale, keep, out, workspace, s)                  \
              : narrow_t<T, V, 128>(in, z, mats, st, eps, scale, keep, out, workspace, s))
  if (dt == 1) return vec ? MOE_NARROW(bf16_t, true) : MOE_NARROW(bf16_t, false);
  return vec ? MOE_NARROW(float, true) : MOE_NARROW(float, false);
#undef MOE_NARROW
}

}  // namespace moe
