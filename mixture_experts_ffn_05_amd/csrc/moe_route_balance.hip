// Backward of the router with its auxiliary losses: as moe_route_backward, with the
// gradients of the balance and z losses added to the logits'.
//
// With p[t] = softmax(logits[t]), c the counts, n the valid tokens and
//
//   balance = coef E / (top_k n^2) sum_e c[e] sum_t p[t, e],   z = z_coef / n sum_t lse[t]^2
//
// (c is a count: it has no gradient), a valid token's logits get
//
//   p[t, e] (coef E / (top_k n^2) (c[e] - sum_j p[t, j] c[j]) + 2 z_coef / n lse[t])
//
// on top of the route weights' dl[t, j] = w[j] (dw[j] - sum_i w[i] dw[i]) at the
// selected experts.  Every logit has a gradient then, so d_x is a matrix product
// and no longer a gather of top_k columns:
//
//   d_x (+)= d W_r^T,   d_W_r = x^T d,   d_bias = sum_t d[t]
//
// d is fp32; the products are bf16 MFMAs, so d is kept as the sum of bf16 planes:
// three (24 bits, fp32's own) for d_x, which is fp32, and two of them (16 bits) for
// d_W_r, which is stored as bf16.  E is small next to T and H, so the planes'
// products stay below the traffic of d_x and x, which bounds the call.  (4096 tokens, H
// 7168, 256 experts: 111 to 132 us for loss_main, 485 MB at 3.7 to 4.4 TB/s; d_x's tiles
// alone 80, the weight's 47.)
//
// Steps: loss_logits (d, its planes and partial bias sums; for E not a multiple of
// 8 a copy of W_r with zero columns), loss_main (both products and the bias in one
// launch, so that the weight product's chains run under d_x's traffic), and where
// the weight product's tokens were split, loss_finish.
#include "moe_dense.h"

namespace moe {
namespace {

// Tokens per workgroup of loss_logits: one per wave where there are few (4096 x 256:
// 10 us; four per wave: 16), four where the bias would have many partial sums.
int loss_tokens(int T) { return T <= 8192 ? 4 : 16; }

struct LossArgs {
  const float *logits, *lse, *w, *dw;
  const int32_t *ids, *counts, *tokens;
  const uint8_t* mask;
  const void* wr;
  void *dense, *wr_pad;
  float* bias_part;
  int T, E, Ep, k, H, chunks;
  float coef, z_coef;
};

// d of elements [e, e + 2) of token t into the planes.
__device__ __forceinline__ void store_planes(const LossArgs& a, int64_t t, int e, float v0, float v1, bf16_t) {
  bf16_t* row = (bf16_t*)a.dense + t * 3 * a.Ep + e;
#pragma unroll
  for (int z = 0; z < 3; ++z) {
    const uint32_t h0 = f32_to_bf16_rne(v0), h1 = f32_to_bf16_rne(v1);
    *(uint32_t*)(row + (int64_t)z * a.Ep) = h0 | (h1 << 16);
    v0 -= bf16_to_f32(h0);
    v1 -= bf16_to_f32(h1);
  }
}
__device__ __forceinline__ void store_planes(const LossArgs& a, int64_t t, int e, float v0, float v1, float) {
  float* row = (float*)a.dense + t * a.Ep + e;
  row[0] = v0;
  row[1] = v1;
}

// Workgroups [0, chunks): 4 kMine tokens, kMine per wave; a lane holds two neighbouring
// experts of every 128.  The rest copy rows of W_r [H, E] into rows
// of Ep elements.
template <typename T, int J, int kMine>
__global__ __launch_bounds__(256) void loss_logits(LossArgs a) {
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  if ((int)blockIdx.x >= a.chunks) {
    const int64_t h = (int64_t)(blockIdx.x - a.chunks) * 4 + wave;
    if (h >= a.H) return;
    for (int e = lane; e < a.Ep; e += 64)
      ((T*)a.wr_pad)[h * a.Ep + e] = e < a.E ? ((const T*)a.wr)[h * a.E + e] : T(0);
    return;
  }
  __shared__ float s_bias[4][J * 128];
  const int n = a.tokens[0];
  const float inv_n = 1.0f / (n > 1 ? (float)n : 1.0f);
  const float kb = a.coef * (float)a.E / (float)a.k * inv_n * inv_n, kz = 2.0f * a.z_coef * inv_n;
  float c[J][2], bias[J][2];
#pragma unroll
  for (int j = 0; j < J; ++j)
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int e = 128 * j + 2 * lane + q;
      c[j][q] = e < a.E ? (float)a.counts[e] : 0.f;
      bias[j][q] = 0.f;
    }
  // what a wave's tokens read first, so that it waits for memory once
  float l[kMine][J][2], lses[kMine], ws[kMine], dws[kMine];
  int ids[kMine];
  bool valids[kMine];
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int64_t t = (int64_t)blockIdx.x * 4 * kMine + wave + 4 * i;
    const bool in = t < a.T;
    valids[i] = in && (!a.mask || a.mask[t]);
    lses[i] = valids[i] ? a.lse[t] : 0.f;
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int e = 128 * j + 2 * lane + q;
        l[i][j][q] = valids[i] && e < a.E ? a.logits[t * a.E + e] : -INFINITY;
      }
    const bool have = in && a.dw && lane < a.k;   // top_k <= 32: a pair per lane
    ids[i] = have ? a.ids[t * a.k + lane] : -1;
    ws[i] = have ? a.w[t * a.k + lane] : 0.f;
    dws[i] = have ? a.dw[t * a.k + lane] : 0.f;
  }
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int64_t t = (int64_t)blockIdx.x * 4 * kMine + wave + 4 * i;
    if (t >= a.T) break;
    const float lse = lses[i];
    // lse brings the exponentials near 1 in all, but its rounding, a half step of |lse|, is
    // a factor of them all (of E where every logit is the type's lowest): their sum divides it out
    float d[J][2], dot = 0.f, total = 0.f;
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        d[j][q] = valids[i] && 128 * j + 2 * lane + q < a.E ? expf(l[i][j][q] - lse) : 0.f;
        dot = fmaf(d[j][q], c[j][q], dot);
        total += d[j][q];
      }
    const float inv = valids[i] ? 1.0f / wave_sum(total) : 0.f;
    dot = wave_sum(dot) * inv;
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int q = 0; q < 2; ++q) d[j][q] = d[j][q] * inv * fmaf(kb, c[j][q] - dot, kz * lse);
    if (a.dw) {
      const float dl = ws[i] * (dws[i] - wave_sum(lane < a.k ? ws[i] * dws[i] : 0.f));
      for (int j = 0; j < a.k; ++j) {
        const int e = __builtin_amdgcn_readlane(ids[i], j);
        const float v = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(dl), j));
        if (e < 0 || e >= a.E) continue;
#pragma unroll
        for (int u = 0; u < J; ++u)
#pragma unroll
          for (int q = 0; q < 2; ++q)
            if (e == 128 * u + 2 * lane + q) d[u][q] += v;
      }
    }
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int e = 128 * j + 2 * lane;
      if (e < a.Ep) store_planes(a, t, e, d[j][0], d[j][1], T{});
      bias[j][0] += d[j][0];
      bias[j][1] += d[j][1];
    }
  }
  if (!a.bias_part) return;
#pragma unroll
  for (int j = 0; j < J; ++j)
#pragma unroll
    for (int q = 0; q < 2; ++q) s_bias[wave][128 * j + 2 * lane + q] = bias[j][q];
  __syncthreads();
  for (int e = tid; e < a.E; e += 256)
    a.bias_part[(int64_t)blockIdx.x * a.E + e] = s_bias[0][e] + s_bias[1][e] + s_bias[2][e] + s_bias[3][e];
}

// 16 experts of the bias: 16 groups of threads add a run of the chunks' partial
// sums each, in order, and the runs are added in order.
__device__ __forceinline__ void loss_bias(int block, const float* __restrict__ part, int chunks, int E,
                                          float* __restrict__ d_bias, float* s_q) {
  const int l = threadIdx.x & 15, g = threadIdx.x >> 4, e = block * 16 + l;
  const int per = (chunks + 15) / 16, c0 = g * per, n = max(min(per, chunks - c0), 0);
  s_q[g * 16 + l] = e < E ? sum_slices(part + (int64_t)c0 * E + e, E, n) : 0.f;
  __syncthreads();
  if (g == 0 && e < E) {
    float v = 0.f;
#pragma unroll
    for (int q = 0; q < 16; ++q) v += s_q[q * 16 + l];
    d_bias[e] = v;
  }
}

struct LossMain {
  const float* bias_part;
  float* d_bias;
  int E, chunks;
};

// Workgroups [0, nw): the weight product's tiles; [nw, nw + nx): d_x's; the rest
// the bias.
template <typename T, class CW, class CX>
__global__ __launch_bounds__(256, 2) void loss_main(LossMain a, DenseProblem w, DenseProblem x, DensePlanes pw,
                                                    DensePlanes px, int nw, int nx) {
  extern __shared__ __attribute__((aligned(1024))) unsigned char smem[];
  const int u = blockIdx.x;
  if (u < nw) {
    if constexpr (sizeof(T) == 2)
      dense_tile_at<CW, true, true, kEStoreCols>(w, dense_unit(w, u), smem, pw, PlanesEpi{});
    else
      dense_f32_tile<true, true, kEStoreCols>(w, u, (float*)smem);
  } else if (u < nw + nx) {
    if constexpr (sizeof(T) == 2)
      dense_tile_at<CX, false, false, kEInputGrad>(x, dense_unit(x, u - nw), smem, px, PlanesEpi{});
    else
      dense_f32_tile<false, false, kEInputGrad>(x, u - nw, (float*)smem);
  } else {
    loss_bias(u - nw - nx, a.bias_part, a.chunks, a.E, a.d_bias, (float*)smem);
  }
}

// d_w_router [H, E] from the partial sums [splits][H][Ep], added in order, eight
// experts per thread.
template <typename T>
__global__ __launch_bounds__(256) void loss_finish(DenseProblem w) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, ps = (int64_t)w.M * w.N;
  const int oct = w.N / 8;
  if (i >= w.M * (int64_t)oct) return;
  const int64_t h = i / oct;
  const int e0 = 8 * (int)(i % oct);
  float v[8] = {0, 0, 0, 0, 0, 0, 0, 0}, x[8];
#pragma unroll 4
  for (int z = 0; z < w.splits; ++z) {
    load8(w.partial + z * ps + h * w.N + e0, x);
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] += x[q];
  }
  epi8_now<T, kEStoreCols>(w.e, h, e0, w.N, v, v);
}

typedef DenseCfg<128, 128, 2, 2, 1, false, true> LossM;   // 4 waves of 64 x 64, two workgroups per CU
typedef DenseCfg<128, 64, 4, 1, 1, false, true> LossN;    // 4 waves of 32 x 64, two per CU

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

struct LossWs {
  size_t dense, bias, part, wr, bytes;
  int Ep, chunks, splits, k_split;
};

// The weight product's token ranges: chains of 64-token slices, two planes each,
// that run under d_x's traffic; more than one range costs the adding launch and the
// partial sums' trip through memory.
LossWs loss_ws(int dt, int T, int H, int E, int cu_count) {
  LossWs w;
  w.Ep = (E + 7) / 8 * 8;
  w.chunks = (T + loss_tokens(T) - 1) / loss_tokens(T);
  const int64_t tiles = (int64_t)((H + 127) / 128) * (w.Ep <= 64 ? 1 : (w.Ep + 127) / 128);
  const double slice = dt != 1 ? 2.0 : w.Ep <= 64 ? 1.2 : 2.0;
  const double x_us = 4.0 + (double)T * H * 8 / 4.6e6, part_us = (double)H * w.Ep * 8 / 3.5e6;
  const int slices = (T + 63) / 64;
  double best = 1e30;
  w.splits = 1;
  w.k_split = slices * 64;
  for (int s = 1; s <= 16 && s <= (T + 127) / 128 && (s == 1 || s * tiles <= 2 * cu_count); ++s) {
    const int per = (slices + s - 1) / s;
    if ((slices + per - 1) / per != s) continue;
    const double w_us = 3.0 + per * slice;
    const double us = (w_us > x_us ? w_us : x_us) + (s > 1 ? 3.0 + s * part_us : 0.0);
    if (us < best) {
      best = us;
      w.splits = s;
      w.k_split = per * 64;
    }
  }
  size_t at = 0;
  w.dense = at;
  at += align256((size_t)T * w.Ep * (dt == 1 ? 6 : 4));
  w.bias = at;
  at += align256((size_t)w.chunks * E * 4);
  w.part = at;
  at += align256(w.splits > 1 ? (size_t)w.splits * H * w.Ep * 4 : 0);
  w.wr = at;
  at += align256(E % 8 ? (size_t)H * w.Ep * (dt == 1 ? 2 : 4) : 0);
  w.bytes = at;
  return w;
}

template <typename T, int J>
hipError_t launch_logits(const LossArgs& a, hipStream_t s) {
  const unsigned blocks = a.chunks + (a.wr_pad ? (a.H + 3) / 4 : 0);
  if (loss_tokens(a.T) == 4)
    hipLaunchKernelGGL((loss_logits<T, J, 1>), dim3(blocks), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((loss_logits<T, J, 4>), dim3(blocks), dim3(256), 0, s, a);
  return hipGetLastError();
}

template <typename T, class CW, class CX>
hipError_t launch_main(const LossMain& m, DenseProblem w, DenseProblem x, const DensePlanes& pw, const DensePlanes& px,
                       int nb, hipStream_t s) {
  constexpr bool F32 = sizeof(T) == 4;
  constexpr int f_lds = dense_f32_lds<kEStoreCols>() * 4;
  constexpr int lds = F32 ? f_lds : CW::kLds > CX::kLds ? CW::kLds : CX::kLds;
  static std::atomic<uint64_t> lds_done{0};
  const hipError_t err = allow_lds(reinterpret_cast<const void*>(&loss_main<T, CW, CX>), lds, lds_done);
  if (err != hipSuccess) return err;
  w.m_tiles = (w.M + (F32 ? 31 : CW::BM - 1)) / (F32 ? 32 : CW::BM);
  w.n_tiles = (w.N + (F32 ? 31 : CW::BN - 1)) / (F32 ? 32 : CW::BN);
  x.m_tiles = (x.M + (F32 ? 31 : CX::BM - 1)) / (F32 ? 32 : CX::BM);
  x.n_tiles = (x.N + (F32 ? 31 : CX::BN - 1)) / (F32 ? 32 : CX::BN);
  const int nw = w.m_tiles * w.n_tiles * w.splits, nx = x.m_tiles * x.n_tiles;
  hipLaunchKernelGGL((loss_main<T, CW, CX>), dim3(nw + nx + nb), dim3(256), lds, s, m, w, x, pw, px, nw, nx);
  return hipGetLastError();
}

template <typename T>
hipError_t route_balance_backward_t(LossArgs a, int dt, const void* x, int accumulate, float* d_x, void* d_wr,
                                    float* d_bias, void* workspace, int cu_count, hipStream_t s) {
  const LossWs ws = loss_ws(dt, a.T, a.H, a.E, cu_count);
  char* base = (char*)workspace;
  a.Ep = ws.Ep;
  a.chunks = ws.chunks;
  a.dense = base + ws.dense;
  a.bias_part = d_bias ? (float*)(base + ws.bias) : nullptr;
  a.wr_pad = a.E % 8 ? base + ws.wr : nullptr;
  hipError_t err = a.E <= 128   ? launch_logits<T, 1>(a, s)
                   : a.E <= 256 ? launch_logits<T, 2>(a, s)
                   : a.E <= 512 ? launch_logits<T, 4>(a, s)
                                : launch_logits<T, 8>(a, s);
  if (err != hipSuccess) return err;
  const int planes = dt == 1 ? 3 : 1;
  DenseProblem w{x, a.dense, a.H, ws.Ep, a.T, a.H, planes * ws.Ep, ws.splits, ws.k_split};
  w.partial = ws.splits > 1 ? (float*)(base + ws.part) : nullptr;
  w.e.out = d_wr;
  w.e.cols = a.E;
  DenseProblem p{a.dense, a.wr_pad ? a.wr_pad : a.wr, a.T, a.H, ws.Ep, planes * ws.Ep, ws.Ep, 1,
                 (ws.Ep + kDBK - 1) / kDBK * kDBK};
  p.partial = nullptr;
  p.e.out = d_x;
  p.e.accumulate = accumulate;
  DensePlanes pw, px;
  pw.count = 2;
  pw.b[1] = ws.Ep;
  px.count = 3;
  px.a[1] = ws.Ep;
  px.a[2] = 2 * ws.Ep;
  const LossMain m{a.bias_part, d_bias, a.E, ws.chunks};
  const int nb = d_bias ? (a.E + 15) / 16 : 0;
  if (sizeof(T) == 2 && ws.Ep > 64)
    err = launch_main<T, LossM, LossM>(m, w, p, pw, px, nb, s);
  else
    err = launch_main<T, LossN, LossM>(m, w, p, pw, px, nb, s);
  if (err != hipSuccess || !w.partial) return err;
  const int blocks = (int)(((int64_t)a.H * (ws.Ep / 8) + 255) / 256);
  hipLaunchKernelGGL(loss_finish<T>, dim3(blocks), dim3(256), 0, s, w);
  return hipGetLastError();
}

}  // namespace
}  // namespace moe

namespace moe_launch {

size_t route_balance_backward_workspace_bytes(int dt, int T, int H, int E, int cu_count) {
  return moe::loss_ws(dt, T, H, E, cu_count).bytes;
}

int64_t route_balance_backward_blocks(int dt, int T, int H, int E) {
  const int64_t t = dt == 1 ? 128 : 32, hp = (H + t - 1) / t, ep = dt == 1 ? (E + 63) / 64 : (E + 31) / 32;
  const int64_t main = (T + t - 1) / t * hp + 16 * ep * hp + 64;
  const int64_t first = ((int64_t)T + moe::loss_tokens(T) - 1) / moe::loss_tokens(T) + (H + 3) / 4;
  return main > first ? main : first;
}

hipError_t route_balance_backward(int dt, const void* x, const void* w_router, const float* logits, const float* lse,
                                  const int32_t* ids, const float* weights, const float* d_weights,
                                  const uint8_t* mask, const int32_t* counts, const int32_t* tokens, int T, int H,
                                  int E, int top_k, float coef, float z_coef, int accumulate, float* d_x,
                                  void* d_w_router, float* d_bias, void* workspace, int cu_count, hipStream_t s) {
  moe::LossArgs a{};
  a.logits = logits;
  a.lse = lse;
  a.w = weights;
  a.dw = d_weights;
  a.ids = ids;
  a.counts = counts;
  a.tokens = tokens;
  a.mask = mask;
  a.wr = w_router;
  a.T = T;
  a.E = E;
  a.k = top_k;
  a.H = H;
  a.coef = coef;
  a.z_coef = z_coef;
  if (dt == 1)
    return moe::route_balance_backward_t<moe::bf16_t>(a, dt, x, accumulate, d_x, d_w_router, d_bias, workspace,
                                                      cu_count, s);
  return moe::route_balance_backward_t<float>(a, dt, x, accumulate, d_x, d_w_router, d_bias, workspace, cu_count, s);
}

}  // namespace moe_launch
