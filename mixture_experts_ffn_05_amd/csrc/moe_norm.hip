// The norms before and after the layer, fused with the branch's gate and the
// residual scales, and their backward.
//
// The layer sits in a residual block (PLENA_Compiler PR #69, section "Group B":
// residual_setup); with r(v) = 1 / sqrt(mean_h v^2 + eps):
//
//   n     = y r(y) (o + w_post)          (without w_post: n = y)
//   h'    = rs h + bs gate n             (stored in the stream's type; without y: h' = h)
//   x     = h' r(h') (o + w_pre)         (of h' as stored)
//
// and backward, with hat = h' r(h'), g = d_x (o + w_pre):
//
//   d       = d_h' + r(h') (g - hat mean(g hat))
//   d_w_pre = sum_t d_x hat
//   d_h     = rs d,  d_gate = sum_t bs d n,  d_n = bs d gate
//   d_w_post and d_y: as d_w_pre and the norm's part of d, with d_n and y
//
// Everything is bound by memory (4096 x 7168 forward: 56 us, 5.3 TB/s; 8192 x 2048
// backward: 59 us, 5.1), but for the backward of more than 4096 columns, whose
// registers do not suffice: one pass, a row's columns in registers (8 V
// columns of a lane, NW waves per row), statistics and sums in fp32.  The
// backward's two means are taken from one reduction of four sums: with q = bs
// gate (o + w_post) y r(y), the second mean's sum q d is
//
//   sum q d_h' + r (sum q g - mean(g hat) sum q hat)
//
// so a row costs one exchange between its waves and not two that depend on
// each other.
#include "moe_common.h"

#include <type_traits>

namespace moe {
namespace {

constexpr int kMaxNormWidth = 8192;   // 16 waves of 8 columns per lane

// Eight elements as they are stored.
template <typename T>
struct Raw8 {
  u32x4 v[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Raw8<T> raw8(const T* p, bool ok) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.v[i] = ok ? ((const u32x4*)p)[i] : u32x4{0u, 0u, 0u, 0u};
  return r;
}
__device__ __forceinline__ void unpack(const Raw8<float>& r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r.v[i / 4][i % 4]);
}
__device__ __forceinline__ void unpack(const Raw8<bf16_t>& r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_to_f32(r.v[0][i] & 0xffffu);
    v[2 * i + 1] = __uint_as_float(r.v[0][i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void st8(float* p, const float (&v)[8]) {
  *(f32x4*)p = f32x4{v[0], v[1], v[2], v[3]};
  *(f32x4*)(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
}
__device__ __forceinline__ void st8(bf16_t* p, const float (&v)[8]) {
  bf16x8 o;
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = (__bf16)v[i];
  *(bf16x8*)p = o;
}
// v as the type stores it
__device__ __forceinline__ void rnd8(float (&)[8], const float*) {}
__device__ __forceinline__ void rnd8(float (&v)[8], const bf16_t*) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = (float)(__bf16)v[i];
}

struct NormArgs {
  const void *h, *w_post, *gate, *w_pre;
  const float* y;
  void *h_out, *x;
  float *rstd_post, *rstd_pre;
  int T, H;
  float eps, offset, rs, bs;
};

// Sums of N values over the NW waves of a row, in the waves' order; `red` is
// [2][N][NW] and `phase` alternates between its halves, so that one barrier per
// reduction is enough.
template <int NW, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* red, int& phase) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if constexpr (NW > 1) {
    const int wave = threadIdx.x >> 6;
    float* r = red + phase * N * NW;
    phase ^= 1;
    if (lane_id() == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) r[i * NW + wave] = v[i];
    lds_barrier();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) v[i] += r[i * NW + w];
    }
  }
}

// Rows per workgroup: four waves with a row each, or one row over all waves.
template <int NW>
constexpr int norm_rows() { return NW == 1 ? 4 : 1; }
template <int NW>
constexpr int norm_threads() { return NW == 1 ? 256 : 64 * NW; }

// A workgroup takes every gridDim.x-th row (group of rows); the next row's loads are
// in flight while one is worked on, and the weights stay in registers.
template <typename R, typename X, int NW, int V>
__global__ __launch_bounds__(norm_threads<NW>()) void norm_fwd(NormArgs a) {
  __shared__ float red[2 * NW];
  int phase = 0;
  const int l = NW == 1 ? lane_id() : threadIdx.x, step = NW * 64 * 8;
  const float inv = 1.0f / a.H;
  bool ok[V];
  Raw8<X> w_post[V], gate[V], w_pre[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = 8 * l + i * step;
    ok[i] = c < a.H;
    w_post[i] = raw8((const X*)a.w_post + c, ok[i] && a.w_post);
    gate[i] = raw8((const X*)a.gate + c, ok[i] && a.gate);
    w_pre[i] = raw8((const X*)a.w_pre + c, ok[i] && a.w_pre);
  }
  Raw8<R> next_h[V];
  Raw8<float> next_y[V];
  auto fetch = [&](int64_t t) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int64_t at = t * a.H + 8 * l + i * step;
      next_h[i] = raw8((const R*)a.h + at, ok[i] && t < a.T);
      next_y[i] = raw8(a.y + at, ok[i] && t < a.T && a.y);
    }
  };
  const int64_t stride = (int64_t)gridDim.x * norm_rows<NW>();
  int64_t t = (int64_t)blockIdx.x * norm_rows<NW>() + (NW == 1 ? threadIdx.x >> 6 : 0);
  fetch(t);
  // whole waves leave the loop together, and with NW > 1 whole workgroups
  for (; t < a.T; t += stride) {
    const int64_t base = t * a.H;
    float s[V][8], n[V][8], w[8];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      unpack(next_h[i], s[i]);
      unpack(next_y[i], n[i]);
    }
    fetch(t + stride);
    if (a.y) {
      float f = 1.0f;
      if (a.w_post) {
        float m[1] = {0.f};
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
          for (int q = 0; q < 8; ++q) m[0] = fmaf(n[i][q], n[i][q], m[0]);
        row_sums<NW, 1>(m, red, phase);
        f = 1.0f / sqrtf(m[0] * inv + a.eps);
        if (l == 0 && a.rstd_post) a.rstd_post[t] = f;
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (a.w_post) {
          unpack(w_post[i], w);
#pragma unroll
          for (int q = 0; q < 8; ++q) n[i][q] *= f * (a.offset + w[q]);
        }
        if (a.gate) {
          unpack(gate[i], w);
#pragma unroll
          for (int q = 0; q < 8; ++q) n[i][q] *= w[q];
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) s[i][q] = fmaf(a.bs, n[i][q], a.rs * s[i][q]);
        rnd8(s[i], (const R*)nullptr);
        if (ok[i]) st8((R*)a.h_out + base + 8 * l + i * step, s[i]);
      }
    }
    if (!a.w_pre) continue;
    float m[1] = {0.f};
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int q = 0; q < 8; ++q) m[0] = fmaf(s[i][q], s[i][q], m[0]);
    row_sums<NW, 1>(m, red, phase);
    const float f = 1.0f / sqrtf(m[0] * inv + a.eps);
    if (l == 0 && a.rstd_pre) a.rstd_pre[t] = f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      unpack(w_pre[i], w);
#pragma unroll
      for (int q = 0; q < 8; ++q) s[i][q] *= f * (a.offset + w[q]);
      if (ok[i]) st8((X*)a.x + base + 8 * l + i * step, s[i]);
    }
  }
}

struct NormBwdArgs {
  const void *d_h_out, *stream, *w_pre, *w_post, *gate;
  const float *d_x, *rstd_pre, *y, *rstd_post;
  void* d_h;
  float* d_y;
  float* part;   // [blocks][3][H]: sums of d_w_pre, d_w_post, d_gate
  int T, H;
  float offset, rs, bs;
};

template <typename R, typename X, int NW, int V>
__global__ __launch_bounds__(norm_threads<NW>()) void norm_bwd(NormBwdArgs a) {
  __shared__ float red[2 * 4 * NW];
  extern __shared__ __attribute__((aligned(16))) float s_part[];   // NW == 1: [3][H]
  int phase = 0;
  const int l = NW == 1 ? lane_id() : threadIdx.x, step = NW * 64 * 8;
  const float inv = 1.0f / a.H;
  bool ok[V];
  // wide rows: the registers go to the sums, the weights are read again for every row
  constexpr bool kKeep = V == 1;
  Raw8<X> w_post[V], gate[V], w_pre[V];
  auto weights = [&](int i) {
    const int c = 8 * l + i * step;
    w_post[i] = raw8((const X*)a.w_post + c, ok[i] && a.w_post);
    gate[i] = raw8((const X*)a.gate + c, ok[i] && a.gate);
    w_pre[i] = raw8((const X*)a.w_pre + c, ok[i] && a.w_pre);
  };
  float wpre[V][8], wpost[V][8], wgate[V][8];   // the weights' sums
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = 8 * l + i * step;
    ok[i] = c < a.H;
    if (kKeep) weights(i);
#pragma unroll
    for (int q = 0; q < 8; ++q) wpre[i][q] = wpost[i][q] = wgate[i][q] = 0.f;
  }
  Raw8<R> next_d[V], next_h[V];
  Raw8<float> next_g[V], next_y[V];
  float next_rp = 0.f, next_ro = 1.0f;
  auto fetch = [&](int64_t t) {
    const bool in = t < a.T;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int64_t at = t * a.H + 8 * l + i * step;
      next_d[i] = raw8((const R*)a.d_h_out + at, ok[i] && in && a.d_h_out);
      next_h[i] = raw8((const R*)a.stream + at, ok[i] && in && a.d_x);
      next_g[i] = raw8(a.d_x + at, ok[i] && in && a.d_x);
      next_y[i] = raw8(a.y + at, ok[i] && in && a.y);
    }
    next_rp = in && a.d_x ? a.rstd_pre[t] : 0.f;
    next_ro = in && a.w_post ? a.rstd_post[t] : 1.0f;
  };
  const int64_t stride = (int64_t)gridDim.x * norm_rows<NW>();
  int64_t t = (int64_t)blockIdx.x * norm_rows<NW>() + (NW == 1 ? threadIdx.x >> 6 : 0);
  fetch(t);
  for (; t < a.T; t += stride) {
    const int64_t base = t * a.H;
    float d[V][8], hat[V][8], g[V][8], z[V][8], w[8], u[8];
    const float rp = next_rp, ro = next_ro;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      unpack(next_d[i], d[i]);
      unpack(next_h[i], hat[i]);
      unpack(next_g[i], g[i]);
      unpack(next_y[i], z[i]);
    }
    fetch(t + stride);
    float m[4] = {0.f, 0.f, 0.f, 0.f};   // sums of g hat, q d_h', q g, q hat
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (!kKeep) weights(i);
      unpack(w_pre[i], w);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        hat[i][q] *= rp;
        wpre[i][q] = fmaf(g[i][q], hat[i][q], wpre[i][q]);
        g[i][q] *= a.offset + w[q];
        m[0] = fmaf(g[i][q], hat[i][q], m[0]);
      }
      if (a.w_post) {
        unpack(w_post[i], w);
        unpack(gate[i], u);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          z[i][q] *= ro;
          const float k = a.bs * (a.offset + w[q]) * (a.gate ? u[q] : 1.0f) * z[i][q];
          m[1] = fmaf(k, d[i][q], m[1]);
          m[2] = fmaf(k, g[i][q], m[2]);
          m[3] = fmaf(k, hat[i][q], m[3]);
        }
      }
    }
    row_sums<NW, 4>(m, red, phase);
    const float m0 = m[0] * inv, m1 = (m[1] + rp * (m[2] - m0 * m[3])) * inv;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float o[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        d[i][q] = fmaf(rp, g[i][q] - hat[i][q] * m0, d[i][q]);
        o[q] = a.rs * d[i][q];
      }
      if (ok[i]) st8((R*)a.d_h + base + 8 * l + i * step, o);
      if (!a.d_y) continue;
      unpack(w_post[i], w);
      unpack(gate[i], u);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float b = a.bs * d[i][q];
        float dn = b;
        const float ow = a.w_post ? a.offset + w[q] : 1.0f;
        if (a.gate) {
          wgate[i][q] = fmaf(b, z[i][q] * ow, wgate[i][q]);
          dn = b * u[q];
        }
        if (a.w_post) {
          wpost[i][q] = fmaf(dn, z[i][q], wpost[i][q]);
          dn = ro * (dn * ow - z[i][q] * m1);
        }
        o[q] = dn;
      }
      if (ok[i]) st8(a.d_y + base + 8 * l + i * step, o);
    }
  }
  // the workgroup's partial sums of the weights that are there; its rows' waves in order
  float* part = a.part + (int64_t)blockIdx.x * 3 * a.H;
  const bool want[3] = {a.d_x != nullptr, a.w_post != nullptr, a.gate != nullptr};
  if constexpr (NW == 1) {
    for (int w = 0; w < 4; ++w) {
      if ((threadIdx.x >> 6) == w) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          if (!ok[i]) continue;
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            float* p = s_part + 8 * l + i * step + q;
            p[0] = (w ? p[0] : 0.f) + wpre[i][q];
            p[a.H] = (w ? p[a.H] : 0.f) + wpost[i][q];
            p[2 * a.H] = (w ? p[2 * a.H] : 0.f) + wgate[i][q];
          }
        }
      }
      __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < 3; ++k)
      if (want[k])
        for (int c = 4 * threadIdx.x; c < a.H; c += 1024)
          *(f32x4*)(part + k * a.H + c) = *(const f32x4*)(s_part + k * a.H + c);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (!ok[i]) continue;
      const int c = 8 * l + i * step;
      if (want[0]) st8(part + c, wpre[i]);
      if (want[1]) st8(part + a.H + c, wpost[i]);
      if (want[2]) st8(part + 2 * a.H + c, wgate[i]);
    }
  }
}

// The blocks' partial sums added in order: 16 columns per workgroup, 16 groups of
// threads with a run of blocks each.
template <typename X>
__global__ __launch_bounds__(256) void norm_bwd_sum(const float* __restrict__ part, int blocks, int H, X* d_w_pre,
                                                    X* d_w_post, X* d_gate) {
  __shared__ float s_q[16][17];
  X* out = blockIdx.y == 0 ? d_w_pre : blockIdx.y == 1 ? d_w_post : d_gate;
  if (!out) return;
  const int l = threadIdx.x & 15, g = threadIdx.x >> 4, c = blockIdx.x * 16 + l;
  const int per = (blocks + 15) / 16, b0 = g * per, n = max(min(per, blocks - b0), 0);
  s_q[g][l] = c < H ? sum_slices(part + ((int64_t)b0 * 3 + blockIdx.y) * H + c, 3 * (int64_t)H, n) : 0.f;
  __syncthreads();
  if (g == 0 && c < H) {
    float v = 0.f;
#pragma unroll
    for (int q = 0; q < 16; ++q) v += s_q[q][l];
    store_from_f32(out, c, v);
  }
}

// Waves of a row: eight columns per lane, in powers of two up to 16 waves.
int norm_waves(int H) {
  int w = 1;
  while (w < 16 && 512 * w < H) w *= 2;
  return w;
}

// Workgroups of the backward: 8 waves per CU (their loads, a row ahead, keep more
// than 90 KB per CU in flight), and no more partial sums than that.
int norm_blocks(int T, int H) {
  const int waves = norm_waves(H), rows = waves == 1 ? 4 : 1;
  const int most = waves == 1 ? 512 : waves <= 8 ? 2048 / waves : 256;
  const int64_t need = ((int64_t)T + rows - 1) / rows;
  return (int)(need < most ? need : most);
}

template <typename R, typename X, int NW, int V>
hipError_t run_fwd(const NormArgs& a, hipStream_t s) {
  const int rows = norm_rows<NW>();
  const int64_t need = ((int64_t)a.T + rows - 1) / rows, most = 4096 / (NW * rows);
  hipLaunchKernelGGL((norm_fwd<R, X, NW, V>), dim3((unsigned)(need < most ? need : most)), dim3(norm_threads<NW>()), 0,
                     s, a);
  return hipGetLastError();
}
template <typename R, typename X, int NW, int V>
hipError_t run_bwd(const NormBwdArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((norm_bwd<R, X, NW, V>), dim3(norm_blocks(a.T, a.H)), dim3(norm_threads<NW>()),
                     NW == 1 ? 3 * a.H * sizeof(float) : 0, s, a);
  return hipGetLastError();
}

// The forward of the widest rows takes 16 waves; the backward 8 with 16 columns per
// lane, whose sums would not fit the 128 registers that 16 waves leave a lane.  They do
// not all fit the 256 that 8 leave either: 12 are spilt with a bf16 stream, 31 to 43
// with a float32 one (4096 x 7168, all parts: 144 us, 104 of traffic; 233 and 138).
#define MOE_NORM_BY_WIDTH(fn, wide_waves, wide_v)      \
  switch (norm_waves(a.H)) {                           \
    case 1: return fn<R, X, 1, 1>(a, s);               \
    case 2: return fn<R, X, 2, 1>(a, s);               \
    case 4: return fn<R, X, 4, 1>(a, s);               \
    case 8: return fn<R, X, 8, 1>(a, s);               \
    default: return fn<R, X, wide_waves, wide_v>(a, s); \
  }

template <typename R, typename X>
hipError_t fwd_t(const NormArgs& a, hipStream_t s) {
  MOE_NORM_BY_WIDTH(run_fwd, 16, 1)
}
template <typename R, typename X>
hipError_t bwd_t(const NormBwdArgs& a, hipStream_t s) {
  MOE_NORM_BY_WIDTH(run_bwd, 8, 2)
}

}  // namespace
}  // namespace moe

namespace moe_launch {

int norm_max_width() { return moe::kMaxNormWidth; }

size_t norm_residual_backward_workspace_bytes(int T, int H) {
  return ((size_t)moe::norm_blocks(T, H) * 3 * H * sizeof(float) + 255) & ~(size_t)255;
}

hipError_t norm_residual(int dt, int res, const void* h, const float* y, const void* w_post, const void* gate,
                         const void* w_pre, int T, int H, float eps, float offset, float rs, float bs, void* h_out,
                         void* x, float* rstd_post, float* rstd_pre, hipStream_t s) {
  const moe::NormArgs a{h, w_post, gate, w_pre, y, h_out, x, rstd_post, rstd_pre, T, H, eps, offset, rs, bs};
  if (res == 1) return dt == 1 ? moe::fwd_t<moe::bf16_t, moe::bf16_t>(a, s) : moe::fwd_t<moe::bf16_t, float>(a, s);
  return dt == 1 ? moe::fwd_t<float, moe::bf16_t>(a, s) : moe::fwd_t<float, float>(a, s);
}

hipError_t norm_residual_backward(int dt, int res, const void* d_h_out, const float* d_x, const void* stream,
                                  const float* rstd_pre, const void* w_pre, const float* y, const float* rstd_post,
                                  const void* w_post, const void* gate, int T, int H, float offset, float rs, float bs,
                                  void* d_h, float* d_y, void* d_w_pre, void* d_w_post, void* d_gate, void* ws,
                                  hipStream_t s) {
  const moe::NormBwdArgs a{d_h_out, stream, w_pre, w_post, gate, d_x, rstd_pre, y, rstd_post, d_h, d_y,
                           (float*)ws, T, H, offset, rs, bs};
  hipError_t err;
  if (res == 1)
    err = dt == 1 ? moe::bwd_t<moe::bf16_t, moe::bf16_t>(a, s) : moe::bwd_t<moe::bf16_t, float>(a, s);
  else
    err = dt == 1 ? moe::bwd_t<float, moe::bf16_t>(a, s) : moe::bwd_t<float, float>(a, s);
  if (err != hipSuccess || !(d_w_pre || d_w_post || d_gate)) return err;
  const dim3 grid((H + 15) / 16, 3);
  if (dt == 1)
    hipLaunchKernelGGL(moe::norm_bwd_sum<moe::bf16_t>, grid, dim3(256), 0, s, (const float*)ws,
                       moe::norm_blocks(T, H), H, (moe::bf16_t*)d_w_pre, (moe::bf16_t*)d_w_post, (moe::bf16_t*)d_gate);
  else
    hipLaunchKernelGGL(moe::norm_bwd_sum<float>, grid, dim3(256), 0, s, (const float*)ws, moe::norm_blocks(T, H), H,
                       (float*)d_w_pre, (float*)d_w_post, (float*)d_gate);
  return hipGetLastError();
}

}  // namespace moe_launch
