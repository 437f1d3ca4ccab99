// What the orthogonalised update's two paths share: the update that is
// orthogonalised, read from the gradient and its momentum.
#pragma once

#include "moe_dense.h"

#include <math.h>

#include <type_traits>

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

// Bounds over singular values s in [0, most], from the ends and the zeros of the
// derivative, which is a quadratic in s^2 at most; a hundredth is for rounding.
// (Sampling the range instead took 80 us of the host's time per call.)
//
// Of |a + b s^2 + c s^4|: of P's eigenvalues, and so of its elements.
double poly_bound(double a, double b, double c, double most) {
  const double end = most * most, y = -b / (2.0 * c);   // c = 0: not a number, or past the range
  double v = fmax(fabs(a), fabs(a + end * (b + c * end)));
  if (y > 0.0 && y < end) v = fmax(v, fabs(a + y * (b + c * y)));
  return 1.01 * v + 1e-6;
}
double poly_bound(const float* coef, double most) { return poly_bound(coef[0], coef[1], coef[2], most); }

// Of |a s + b s^3 + c s^5|: of the singular values after the step.
double step_bound(const float* coef, double most) {
  const double a = coef[0], b = coef[1], c = coef[2], end = most * most;
  double v = most * fabs(a + end * (b + c * end));
  const double disc = 9.0 * b * b - 20.0 * a * c;   // of 5 c y^2 + 3 b y + a = 0
  if (disc >= 0.0) {
    const double q = -0.5 * (3.0 * b + copysign(sqrt(disc), b));
    const double roots[2] = {q / (5.0 * c), a / q};
    for (const double y : roots)
      if (y > 0.0 && y < end) v = fmax(v, sqrt(y) * fabs(a + y * (b + c * y)));
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
