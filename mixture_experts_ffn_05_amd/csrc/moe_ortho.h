// What the orthogonalised update's two paths share: the update that is
// orthogonalised, read from the gradient and its momentum.
#pragma once

#include "moe_dense.h"

#include <math.h>

namespace moe {
namespace {

struct OrthoIn {
  const void* grad;
  float* momentum;   // or null
  float mu;
  int nesterov;
  int M, N, parts;
};

// Eight elements of the update from column c of a row on (n of them valid, 0 past).
// FIRST: the momentum takes its step; otherwise it has.
template <typename T, bool VEC, bool FIRST>
__device__ __forceinline__ void ortho_update8(const OrthoIn& in, int64_t at, int n, float (&u)[8]) {
  float m[8];
  if (VEC && n >= 8) {
    load8((const T*)in.grad + at, u);
    if (in.momentum) load8(in.momentum + at, m);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      u[i] = i < n ? load_as_f32((const T*)in.grad, at + i) : 0.f;
      m[i] = in.momentum && i < n ? in.momentum[at + i] : 0.f;
    }
  }
  if (!in.momentum) return;
  if (FIRST) {
#pragma unroll
    for (int i = 0; i < 8; ++i) m[i] = fmaf(in.mu, m[i], u[i]);
    if (VEC && n >= 8) {
      store8(in.momentum + at, m);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) in.momentum[at + i] = m[i];
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) u[i] = in.nesterov ? fmaf(in.mu, m[i], u[i]) : m[i];
}

// Largest power of two by which values up to v stay within half of fp16's range.
float f16_scale(double v) {
  const int e = 15 - (int)ceil(log2(v > 1e-6 ? v : 1e-6));
  return ldexpf(1.0f, e);
}

// Bound of |a + b s^2 + c s^4| for singular values up to `most`: of P's eigenvalues, and so of its elements.
double poly_bound(const float* coef, double most) {
  double v = 0.0;
  for (int i = 0; i <= 4096; ++i) {
    const double x = most * i / 4096, x2 = x * x;
    v = fmax(v, fabs((double)coef[0] + x2 * ((double)coef[1] + (double)coef[2] * x2)));
  }
  return 1.01 * v + 1e-6;
}

}  // namespace

// Matrices of up to 128 rows (or columns): moe_ortho_narrow.hip.
constexpr int kOrthoNarrow = 128;
size_t ortho_narrow_workspace_bytes(int mats, int m, int n);
hipError_t ortho_narrow(int dt, const void* grad, float* momentum, float mu, int nesterov, int batch, int M, int N,
                        int parts, int steps, const float* coef, const double* sigma, float eps, float scale,
                        float keep, void* out, void* workspace, hipStream_t s);

}  // namespace moe
