// Backward of the router: from the route weights' gradient to x, the router
// weight and the logit bias, routes held fixed.
//
// PLENA_Simulator PR #97, section "C_SET_TOPK_REG" (topk_softmax): a token's
// route weights are the softmax over its top_k selected logits, so with
// dw[j] the gradient of w[j] the selected logits' gradient is
//
//   dl[j] = w[j] (dw[j] - sum_i w[i] dw[i])
//
// and every other logit's is zero.  With logits = x W_r + bias:
//
//   d_x[t]     (+)= sum_j dl[t, j] W_r[:, id_j]
//   d_W_r[:, e]  = sum over pairs with id = e of dl[t, j] x[t]
//   d_bias[e]    = sum over those pairs of dl[t, j]
//
// Steps: route_grad_logits computes dl (slots of one token that name the same
// expert are merged into the first, ids outside [0, E) are dropped) as (id, dl)
// pairs, as a dense [T, Ep] matrix in the element type (Ep = E rounded up to
// 8) and as partial bias sums; route_grad_x and the weight product follow;
// route_grad_finish adds partial sums in order.
//
// d_x only needs top_k of W_r's E columns per token, in fp32: it is bound by
// reading and writing d_x, so it is a gather from an LDS tile of W_r and not a
// matrix product (whose operand would have to be rounded).  d_W_r reads x once;
// it is a matrix product over the dense dl (rounded to the element type like
// the d_rows and d_h of the experts' weight gradients), whose zeros cost MFMAs
// that the reads hide, split over tokens to fill the chip.
#include "moe_common.h"

namespace moe {
namespace {

constexpr int kRgTokens = 16;  // tokens per workgroup of route_grad_logits

struct RoutePair {
  int32_t id;  // -1: none
  float dl;
};

template <typename T>
__global__ __launch_bounds__(256) void route_grad_logits(const int32_t* __restrict__ ids, const float* __restrict__ w,
                                                         const float* __restrict__ dw, int Tn, int E, int Ep, int k,
                                                         RoutePair* __restrict__ pairs, T* __restrict__ dense,
                                                         float* __restrict__ bias_part) {
  __shared__ int32_t s_id[kRgTokens][kMaxTopK];
  __shared__ float s_dl[kRgTokens][kMaxTopK];
  const int tid = threadIdx.x;
  const int64_t t0 = (int64_t)blockIdx.x * kRgTokens;
  const int nt = (int)min((int64_t)kRgTokens, Tn - t0);
  for (int i = tid; i < nt * k; i += 256) {
    const int64_t p = t0 * k + i;
    const int id = ids[p];
    s_id[i / k][i % k] = id >= 0 && id < E ? id : -1;
  }
  for (int64_t i = tid; i < (int64_t)nt * Ep; i += 256) store_from_f32(dense + t0 * Ep, i, 0.f);
  __syncthreads();
  if (tid < nt) {
    const float* wt = w + (t0 + tid) * k;
    const float* dt = dw + (t0 + tid) * k;
    float s = 0.f;
    for (int j = 0; j < k; ++j) s = fmaf(wt[j], dt[j], s);
    for (int j = 0; j < k; ++j) s_dl[tid][j] = wt[j] * (dt[j] - s);
    // merge repeated experts into the first slot that names them
    for (int j = 1; j < k; ++j)
      for (int i = 0; i < j; ++i)
        if (s_id[tid][j] >= 0 && s_id[tid][i] == s_id[tid][j]) {
          s_dl[tid][i] += s_dl[tid][j];
          s_id[tid][j] = -1;
        }
  }
  __syncthreads();
  for (int i = tid; i < nt * k; i += 256) {
    const int id = s_id[i / k][i % k];
    const float dl = s_dl[i / k][i % k];
    pairs[t0 * k + i] = RoutePair{id, dl};
    if (id >= 0) store_from_f32(dense + (t0 + i / k) * Ep, id, dl);
  }
  if (bias_part)
    for (int e = tid; e < E; e += 256) {
      float s = 0.f;
      for (int t = 0; t < nt; ++t)
        for (int j = 0; j < k; ++j)
          if (s_id[t][j] == e) s += s_dl[t][j];
      bias_part[(int64_t)blockIdx.x * E + e] = s;
    }
}

__device__ __forceinline__ void add8(float dl, const float* p, float (&v)[8]) {
  const f32x4 a = *(const f32x4*)p, b = *(const f32x4*)(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = fmaf(dl, a[i], v[i]);
    v[4 + i] = fmaf(dl, b[i], v[4 + i]);
  }
}
__device__ __forceinline__ void add8(float dl, const bf16_t* p, float (&v)[8]) {
  const u32x4 a = *(const u32x4*)p;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = fmaf(dl, bf16_to_f32(a[i] & 0xffffu), v[2 * i]);
    v[2 * i + 1] = fmaf(dl, __uint_as_float(a[i] & 0xffff0000u), v[2 * i + 1]);
  }
}

// One workgroup: hc columns of d_x (a power of two, 8..128) for a range of
// tokens.  Its hc rows of W_r ([H, E]) are transposed into LDS as [E][hc]; hc / 8
// lanes then serve one token, adding its pairs' LDS rows 16 bytes at a time in
// slot order.
template <typename T>
__global__ __launch_bounds__(256) void route_grad_x(const RoutePair* __restrict__ pairs, const T* __restrict__ wr,
                                                    int Tn, int H, int E, int k, int hc, int per, int accumulate,
                                                    float* __restrict__ d_x) {
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  T* sw = (T*)smem;
  const int tid = threadIdx.x;
  const int h0 = blockIdx.y * hc;
  for (int i = tid; i < hc * E; i += 256) {
    const int h = i % hc, e = i / hc;
    sw[i] = h0 + h < H ? wr[(int64_t)(h0 + h) * E + e] : (T)0;
  }
  __syncthreads();
  const int lanes = hc / 8, c = tid % lanes, slot = tid / lanes, step = 256 / lanes;
  const int h = h0 + 8 * c;
  if (h >= H) return;
  const int64_t t_lo = (int64_t)blockIdx.x * per, t_hi = min(t_lo + per, (int64_t)Tn);
  for (int64_t t = t_lo + slot; t < t_hi; t += step) {
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    const RoutePair* pt = pairs + t * k;
    for (int j = 0; j < k; ++j) {
      const RoutePair q = pt[j];
      if (q.id >= 0) add8(q.dl, sw + q.id * hc + 8 * c, v);
    }
    f32x4* o = (f32x4*)(d_x + t * H + h);
    f32x4 a{v[0], v[1], v[2], v[3]}, b{v[4], v[5], v[6], v[7]};
    if (accumulate) {
      a += o[0];
      b += o[1];
    }
    o[0] = a;
    o[1] = b;
  }
}

// d_w_router[h][e] (row length E) from the partial sums [splits][H][Ep], added in
// order; the workgroups past the weight's add the bias partials.
template <typename T>
__global__ __launch_bounds__(256) void route_grad_finish(const float* __restrict__ part, int splits, int H, int E,
                                                         int Ep, T* __restrict__ d_wr,
                                                         const float* __restrict__ bias_part, int bias_chunks,
                                                         float* __restrict__ d_bias, int w_blocks) {
  if ((int)blockIdx.x < w_blocks) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= (int64_t)H * E) return;
    const int64_t h = i / E;
    store_from_f32(d_wr, i, sum_slices(part + h * Ep + i % E, (int64_t)H * Ep, splits));
    return;
  }
  // 64 experts per workgroup, each wave a quarter of the chunks; quarters added in order
  __shared__ float s_q[4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int e = ((int)blockIdx.x - w_blocks) * 64 + lane;
  const int per = (bias_chunks + 3) / 4, c0 = wave * per, n = max(min(per, bias_chunks - c0), 0);
  s_q[wave][lane] = e < E ? sum_slices(bias_part + (int64_t)c0 * E + e, E, n) : 0.f;
  __syncthreads();
  if (wave == 0 && e < E) d_bias[e] = ((s_q[0][lane] + s_q[1][lane]) + s_q[2][lane]) + s_q[3][lane];
}

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

// Token ranges of the weight product: enough workgroups (128 x 128 output
// tiles, two per CU) to fill the chip, at least 256 tokens each.
struct RouteSplit {
  int splits, k_split;
};
RouteSplit route_split(int T, int H, int Ep, int cu_count) {
  const int64_t tiles = (int64_t)((H + 127) / 128) * ((Ep + 127) / 128);
  int64_t s = (2 * (int64_t)cu_count + tiles - 1) / tiles;
  const int64_t most = (T + 255) / 256;
  if (s > most) s = most;
  if (s < 1) s = 1;
  int64_t per = ((T + s - 1) / s + 63) / 64 * 64;
  return RouteSplit{(int)((T + per - 1) / per), (int)per};
}

struct RouteWs {
  size_t pairs, dense, bias, part, bytes;
  int Ep, chunks;
  RouteSplit sp;
};
RouteWs route_ws(int dt, int T, int H, int E, int k, int cu_count) {
  RouteWs w;
  w.Ep = (E + 7) / 8 * 8;
  w.chunks = (T + kRgTokens - 1) / kRgTokens;
  w.sp = route_split(T, H, w.Ep, cu_count);
  size_t at = 0;
  w.pairs = at;
  at += align256((size_t)T * k * sizeof(RoutePair));
  w.dense = at;
  at += align256((size_t)T * w.Ep * (dt == 1 ? 2 : 4));
  w.bias = at;
  at += align256((size_t)w.chunks * E * 4);
  w.part = at;
  at += align256((size_t)w.sp.splits * H * w.Ep * 4);
  w.bytes = at;
  return w;
}

template <typename T>
hipError_t route_backward_t(int dt, const void* x, const void* wr, const int32_t* ids, const float* w, const float* dw,
                            int Tn, int H, int E, int k, int accumulate, float* d_x, void* d_wr, float* d_bias,
                            void* workspace, int cu_count, hipStream_t s) {
  const RouteWs ws = route_ws(dt, Tn, H, E, k, cu_count);
  char* base = (char*)workspace;
  RoutePair* pairs = (RoutePair*)(base + ws.pairs);
  T* dense = (T*)(base + ws.dense);
  float* bias_part = (float*)(base + ws.bias);
  float* part = (float*)(base + ws.part);
  hipLaunchKernelGGL(route_grad_logits<T>, dim3(ws.chunks), dim3(256), 0, s, ids, w, dw, Tn, E, ws.Ep, k, pairs, dense,
                     d_bias ? bias_part : nullptr);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  int hc = 128;
  while (hc > 8 && (size_t)hc * E * sizeof(T) > 64 * 1024) hc /= 2;
  const int hb = (H + hc - 1) / hc, step = 256 / (hc / 8);
  int64_t tb = (2 * (int64_t)cu_count + hb - 1) / hb;
  const int64_t most = (Tn + step - 1) / step;
  if (tb > most) tb = most;
  const int per = (int)((Tn + tb - 1) / tb);
  tb = (Tn + per - 1) / per;
  hipLaunchKernelGGL(route_grad_x<T>, dim3((unsigned)tb, hb), dim3(256), (size_t)hc * E * sizeof(T), s, pairs,
                     (const T*)wr, Tn, H, E, k, hc, per, accumulate, d_x);
  err = hipGetLastError();
  if (err != hipSuccess) return err;
  err = moe_launch::router_wgrad_partials(dt, x, dense, Tn, H, ws.Ep, ws.sp.splits, ws.sp.k_split, part, s);
  if (err != hipSuccess) return err;
  const int w_blocks = (int)(((int64_t)H * E + 255) / 256);
  hipLaunchKernelGGL(route_grad_finish<T>, dim3(w_blocks + (d_bias ? (E + 63) / 64 : 0)), dim3(256), 0, s, part,
                     ws.sp.splits, H, E, ws.Ep, (T*)d_wr, bias_part, ws.chunks, d_bias, w_blocks);
  return hipGetLastError();
}

}  // namespace
}  // namespace moe

namespace moe_launch {

size_t route_backward_workspace_bytes(int dt, int T, int H, int E, int top_k, int cu_count) {
  return moe::route_ws(dt, T, H, E, top_k, cu_count).bytes;
}

hipError_t route_backward(int dt, const void* x, const void* w_router, const int32_t* ids, const float* weights,
                          const float* d_weights, int T, int H, int E, int top_k, int accumulate, float* d_x,
                          void* d_w_router, float* d_bias, void* workspace, int cu_count, hipStream_t s) {
  if (dt == 1)
    return moe::route_backward_t<moe::bf16_t>(dt, x, w_router, ids, weights, d_weights, T, H, E, top_k, accumulate,
                                              d_x, d_w_router, d_bias, workspace, cu_count, s);
  return moe::route_backward_t<float>(dt, x, w_router, ids, weights, d_weights, T, H, E, top_k, accumulate, d_x,
                                      d_w_router, d_bias, workspace, cu_count, s);
}

}  // namespace moe_launch
