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
// 8) and as partial bias sums, and transposes W_r; route_grad_main takes the
// weight product, d_x and the bias; where the product's tokens were split,
// route_grad_finish adds the partial sums in order.  One launch for the three:
// the product's chains of MFMAs run under d_x's traffic (4096 tokens, H = 7168,
// 256 experts, top 8: 84 us against 93 one after the other; 1021 tokens, 2048, 60
// experts, top 4: 16 against 20).
//
// d_x only needs top_k of W_r's E columns per token, in fp32: it is bound by
// reading and writing d_x, so it is a gather from an LDS tile of W_r^T and not a
// matrix product (whose operand would have to be rounded).  d_W_r reads x once;
// it is a matrix product over the dense dl (rounded to the element type like
// the d_rows and d_h of the experts' weight gradients: a bf16 d_W_r has a relative
// error of 0.0023 against float64, its store alone 0.0017), whose zeros cost MFMAs
// that the reads hide, split over tokens to fill the chip.
#include "moe_dense.h"

namespace moe {
namespace {

constexpr int kRgTokens = 16;  // tokens per workgroup of route_grad_logits

struct RoutePair {
  int32_t id;  // E: none (the gather's row of zeros)
  float dl;
};

// Workgroups [0, chunks): kRgTokens tokens each.  The rest: 64 x 64 tiles of
// W_r [H, E] into wt [E, H].
template <typename T>
__global__ __launch_bounds__(256) void route_grad_logits(const int32_t* __restrict__ ids, const float* __restrict__ w,
                                                         const float* __restrict__ dw, int Tn, int E, int Ep, int k,
                                                         RoutePair* __restrict__ pairs, T* __restrict__ dense,
                                                         float* __restrict__ bias_part, int chunks,
                                                         const T* __restrict__ wr, int H, T* __restrict__ wt) {
  const int tid = threadIdx.x;
  if ((int)blockIdx.x >= chunks) {
    __shared__ T s_t[64][65];
    const int b = blockIdx.x - chunks, et = (E + 63) / 64;
    const int e0 = (b % et) * 64, h0 = (b / et) * 64, l = tid & 63;
    T v[16];   // all loads in flight at once: clamped, not predicated
#pragma unroll
    for (int i = 0; i < 16; ++i)
      v[i] = wr[(int64_t)min(h0 + (tid >> 6) + 4 * i, H - 1) * E + min(e0 + l, E - 1)];
#pragma unroll
    for (int i = 0; i < 16; ++i) s_t[(tid >> 6) + 4 * i][l] = v[i];
    __syncthreads();
    for (int r = tid >> 6; r < 64; r += 4)
      if (e0 + r < E && h0 + l < H) wt[(int64_t)(e0 + r) * H + h0 + l] = s_t[l][r];
    return;
  }
  __shared__ int32_t s_id[kRgTokens * kMaxTopK], s_mid[kRgTokens * kMaxTopK];
  __shared__ float s_w[kRgTokens * kMaxTopK], s_dw[kRgTokens * kMaxTopK], s_dl[kRgTokens * kMaxTopK];
  __shared__ float s_bias[kMaxExperts];
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  T* s_dense = (T*)smem;   // [kRgTokens][Ep]
  const int64_t t0 = (int64_t)blockIdx.x * kRgTokens;
  const int nt = (int)min((int64_t)kRgTokens, Tn - t0), n = nt * k;
  for (int i = tid; i < n; i += 256) {
    const int id = ids[t0 * k + i];
    s_id[i] = id >= 0 && id < E ? id : -1;
    s_w[i] = w[t0 * k + i];
    s_dw[i] = dw[t0 * k + i];
  }
  // Ep is a multiple of 8: whole 16-byte pieces
  const int pieces = (int)(nt * Ep * sizeof(T) / 16);
  for (int i = tid; i < pieces; i += 256) ((u32x4*)smem)[i] = u32x4{0u, 0u, 0u, 0u};
  if (bias_part)
    for (int e = tid; e < E; e += 256) s_bias[e] = 0.f;
  __syncthreads();
  // one pair per thread: its own logit gradient
  for (int i = tid; i < n; i += 256) {
    const int b = i / k * k;
    float s = 0.f;
    for (int j = 0; j < k; ++j) s = fmaf(s_w[b + j], s_dw[b + j], s);
    s_dl[i] = s_w[i] * (s_dw[i] - s);
  }
  __syncthreads();
  // slots that repeat an expert: the first takes the sum, in slot order
  for (int i = tid; i < n; i += 256) {
    const int b = i / k * k, id = s_id[i];
    float v = s_dl[i];
    bool first = id >= 0;
    for (int j = 0; j < k; ++j) {
      if (id < 0 || s_id[b + j] != id || b + j == i) continue;
      if (b + j < i) first = false; else v += s_dl[b + j];
    }
    s_mid[i] = first ? id : -1;
    s_w[i] = v;
    pairs[t0 * k + i] = RoutePair{first ? id : E, first ? v : 0.f};
    if (first) store_from_f32(s_dense + (i / k) * Ep, id, v);
  }
  __syncthreads();
  for (int i = tid; i < pieces; i += 256) ((u32x4*)(dense + t0 * Ep))[i] = ((const u32x4*)smem)[i];
  if (!bias_part) return;
  // one token after the other; a token's merged slots name different experts
  if (tid < 64)
    for (int t = 0; t < nt; ++t) {
      if (tid < k && s_mid[t * k + tid] >= 0) s_bias[s_mid[t * k + tid]] += s_w[t * k + tid];
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    }
  __syncthreads();
  for (int e = tid; e < E; e += 256) bias_part[(int64_t)blockIdx.x * E + e] = s_bias[e];
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

// One workgroup: hc columns of d_x (a power of two, 16..128) for a range of
// tokens, with its slice [E][hc] of W_r^T and a row of zeros in LDS; hc / 8 lanes
// serve one token, adding its pairs' LDS rows 16 bytes at a time in slot order.
// Tokens go in chunks of U per thread (four; one where many experts make hc
// small and a chunk's pairs large, or where two such chunks per workgroup would
// not fill the chip); the next chunk's old d_x values and pairs (KP per thread)
// are loaded while a chunk is worked on.  Reading W_r^T's rows from L2 instead, a
// whole row of d_x per wave, takes 77 us where this takes about 60 (4096 tokens,
// H = 7168, 256 experts, top 8): d_x streams through L2 and evicts them.
template <typename T, int U, int KP>
__device__ __forceinline__ void route_grad_x(int block, const RoutePair* __restrict__ pairs, const T* __restrict__ wt,
                                             int Tn, int H, int E, int k, int hc, int per, int h_blocks, int accumulate,
                                             float* __restrict__ d_x, unsigned char* __restrict__ smem) {
  T* sw = (T*)smem;
  RoutePair* sp = (RoutePair*)(smem + (size_t)hc * (E + 1) * sizeof(T));   // two chunks of pairs
  const int tid = threadIdx.x;
  const int h0 = block % h_blocks * hc;
  const int lanes = hc / 8, c = tid % lanes, slot = tid / lanes, step = 256 / lanes;
  const int h = h0 + 8 * c;
  const bool live = h < H;
  const int64_t t_lo = (int64_t)(block / h_blocks) * per, t_hi = min(t_lo + per, (int64_t)Tn);
  const int chunk = U * step, cp = chunk * k;   // tokens and pairs of a chunk
  RoutePair next[KP];
  auto fetch = [&](int64_t t) {
#pragma unroll
    for (int i = 0; i < KP; ++i) {
      const int64_t q = t * k + tid + 256 * i;
      next[i] = tid + 256 * i < cp && q < t_hi * k ? pairs[q] : RoutePair{E, 0.f};
    }
  };
  auto put = [&](RoutePair* dst) {
#pragma unroll
    for (int i = 0; i < KP; ++i)
      if (tid + 256 * i < cp) dst[tid + 256 * i] = next[i];
  };
  const f32x4 kZero{0.f, 0.f, 0.f, 0.f};
  f32x4 old[U][2];
#define MOE_FETCH_OLD(t0)                                          \
  _Pragma("unroll") for (int u = 0; u < U; ++u) {                  \
    const int64_t t = (t0) + slot + u * step;                      \
    const f32x4* o = (const f32x4*)(d_x + t * H + h);              \
    const bool ok = accumulate && live && t < t_hi;                \
    old[u][0] = ok ? __builtin_nontemporal_load(o) : kZero;        \
    old[u][1] = ok ? __builtin_nontemporal_load(o + 1) : kZero;    \
  }
  fetch(t_lo);
  MOE_FETCH_OLD(t_lo)
  constexpr int V = 8 * sizeof(T) / 16;   // 16-byte pieces of 8 columns
  if (live)
    for (int e = slot; e < E; e += step)
#pragma unroll
      for (int v = 0; v < V; ++v)
        ((u32x4*)(sw + e * hc + 8 * c))[v] = ((const u32x4*)(wt + (int64_t)e * H + h))[v];
  if (tid < lanes)
#pragma unroll
    for (int v = 0; v < V; ++v) ((u32x4*)(sw + E * hc + 8 * tid))[v] = u32x4{0u, 0u, 0u, 0u};
  put(sp);
  int buf = 0;
  for (int64_t t0 = t_lo; t0 < t_hi; t0 += chunk) {
    lds_barrier();   // LDS only: __syncthreads would also wait for the stores and for the next chunk's loads
    float v[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[u][i] = old[u][i / 4][i % 4];
    fetch(t0 + chunk);   // past the range: nothing
    MOE_FETCH_OLD(t0 + chunk)
    const RoutePair* mine = sp + buf * cp + slot * k;
    for (int j = 0; j < k; ++j)
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const RoutePair q = mine[u * step * k + j];
        add8(q.dl, sw + q.id * hc + 8 * c, v[u]);
      }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t t = t0 + slot + u * step;
      if (live && t < t_hi) {
        f32x4* o = (f32x4*)(d_x + t * H + h);
        __builtin_nontemporal_store(f32x4{v[u][0], v[u][1], v[u][2], v[u][3]}, o);
        __builtin_nontemporal_store(f32x4{v[u][4], v[u][5], v[u][6], v[u][7]}, o + 1);
      }
    }
    buf ^= 1;
    put(sp + buf * cp);
  }
#undef MOE_FETCH_OLD
}

// 16 experts of the bias: 16 groups of threads add a run of the chunks' partial
// sums each, in order, and the runs are added in order.
__device__ __forceinline__ void route_grad_bias(int block, const float* __restrict__ part, int chunks, int E,
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

struct RouteMain {
  const RoutePair* pairs;
  const void* wt;
  const float* bias_part;
  float* d_x;
  float* d_bias;
  int Tn, H, E, k, hc, per, h_blocks, accumulate, chunks;
};

// Everything that follows from the logits' gradients, in one launch: workgroups
// [0, nw) take the weight product's tiles, [nw, nw + nx) d_x, the rest the bias.
template <typename T, int U, int KP, class C>
__global__ __launch_bounds__(256, 2) void route_grad_main(RouteMain a, DenseProblem w, int nw, int nx) {
  extern __shared__ __attribute__((aligned(1024))) unsigned char smem[];
  const int u = blockIdx.x;
  if (u < nw) {
    if constexpr (sizeof(T) == 2)
      dense_tile<C, true, true, kEStoreCols>(w, u, smem);
    else
      dense_f32_tile<true, true, kEStoreCols>(w, u, (float*)smem);
  } else if (u < nw + nx) {
    route_grad_x<T, U, KP>(u - nw, a.pairs, (const T*)a.wt, a.Tn, a.H, a.E, a.k, a.hc, a.per, a.h_blocks, a.accumulate,
                           a.d_x, smem);
  } else {
    route_grad_bias(u - nw - nx, a.bias_part, a.chunks, a.E, a.d_bias, (float*)smem);
  }
}

// d_w_router [H, E] from the partial sums [splits][H][Ep], added in order, eight
// experts per thread.
template <typename T>
__global__ __launch_bounds__(256) void route_grad_finish(DenseProblem w) {
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

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

// Token ranges of the weight product.  A range is a chain of 64-token slices
// (microseconds each, measured beside d_x's traffic) that runs under d_x; more
// than one range costs the adding launch and the partial sums' trip through
// memory.  Few tokens take one range (300 tokens, H = 4096, 128 experts: 12.4 us
// against 16.3 with two), many tokens over a narrow weight several (4096, 2048, 64:
// 30 with four, 42 with one).
struct RouteSplit {
  int splits, k_split;
};
RouteSplit route_split(int dt, int T, int H, int Ep, int cu_count) {
  const int64_t tiles = (int64_t)((H + 127) / 128) * (Ep <= 64 ? 1 : (Ep + 127) / 128);
  const double slice = dt != 1 ? 2.0 : Ep <= 64 ? 0.6 : 1.0;
  const double x_us = 4.0 + (double)T * H * 8 / 4.6e6, part_us = (double)H * Ep * 8 / 3.5e6;
  const int slices = (T + 63) / 64;
  RouteSplit best{1, slices * 64};
  double best_us = 1e30;
  for (int s = 1; s <= 16 && s <= (T + 127) / 128 && (s == 1 || s * tiles <= cu_count); ++s) {
    const int per = (slices + s - 1) / s;
    if ((slices + per - 1) / per != s) continue;
    const double w_us = 3.0 + per * slice;
    const double us = (w_us > x_us ? w_us : x_us) + (s > 1 ? 3.0 + s * part_us : 0.0);
    if (us < best_us) {
      best_us = us;
      best = RouteSplit{s, per * 64};
    }
  }
  return best;
}

struct RouteWs {
  size_t pairs, dense, bias, part, wt, bytes;
  int Ep, chunks;
  RouteSplit sp;
};
RouteWs route_ws(int dt, int T, int H, int E, int k, int cu_count) {
  RouteWs w;
  w.Ep = (E + 7) / 8 * 8;
  w.chunks = (T + kRgTokens - 1) / kRgTokens;
  w.sp = route_split(dt, T, H, w.Ep, cu_count);
  size_t at = 0;
  w.pairs = at;
  at += align256((size_t)T * k * sizeof(RoutePair));
  w.dense = at;
  at += align256((size_t)T * w.Ep * (dt == 1 ? 2 : 4));
  w.bias = at;
  at += align256((size_t)w.chunks * E * 4);
  w.part = at;
  at += align256((size_t)w.sp.splits * H * w.Ep * 4);
  w.wt = at;
  at += align256((size_t)E * H * (dt == 1 ? 2 : 4));
  w.bytes = at;
  return w;
}

// route_grad_x's W_r^T slice takes up to kRouteSlice bytes of LDS and a row of
// zeros, its pairs up to two chunks of 256 / (kMinHc / 8) tokens.
constexpr int kRouteSlice = 64 * 1024, kMinHc = 16, kRoutePairs = 256 / (kMinHc / 8) * kMaxTopK;
constexpr int kRouteXLds = kRouteSlice + 128 * 4 + 2 * kRoutePairs * (int)sizeof(RoutePair);
static_assert(kMinHc * kMaxExperts * 4 <= kRouteSlice, "the narrowest slice fits for every number of experts");
static_assert(kRoutePairs <= 16 * 256, "a thread carries at most 16 pairs");

template <int N>
using Int = std::integral_constant<int, N>;

template <typename T, int U, int KP, class C>
hipError_t launch_route_main(const RouteMain& a, DenseProblem w, int nx, int nb, size_t x_lds, hipStream_t s) {
  constexpr bool F32 = sizeof(T) == 4;
  constexpr int w_lds = F32 ? dense_f32_lds<kEStoreCols>() * 4 : C::kLds;
  constexpr int most = w_lds > kRouteXLds ? w_lds : kRouteXLds;
  static std::atomic<uint64_t> lds_done{0};
  const hipError_t err = allow_lds(reinterpret_cast<const void*>(&route_grad_main<T, U, KP, C>), most, lds_done);
  if (err != hipSuccess) return err;
  w.m_tiles = (w.M + (F32 ? 31 : C::BM - 1)) / (F32 ? 32 : C::BM);
  w.n_tiles = (w.N + (F32 ? 31 : C::BN - 1)) / (F32 ? 32 : C::BN);
  const int nw = w.m_tiles * w.n_tiles * w.splits;
  hipLaunchKernelGGL((route_grad_main<T, U, KP, C>), dim3(nw + nx + nb), dim3(256), x_lds > w_lds ? x_lds : w_lds, s, a,
                     w, nw, nx);
  return hipGetLastError();
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
  T* wt = (T*)(base + ws.wt);
  const size_t dense_lds = (size_t)kRgTokens * ws.Ep * sizeof(T);
  static std::atomic<uint64_t> lds_done{0};
  hipError_t err = allow_lds(reinterpret_cast<const void*>(&route_grad_logits<T>),
                             kRgTokens * kMaxExperts * (int)sizeof(T), lds_done);
  if (err != hipSuccess) return err;
  hipLaunchKernelGGL(route_grad_logits<T>, dim3((unsigned)moe_launch::route_backward_blocks(Tn, H, E)), dim3(256), dense_lds, s, ids, w, dw,
                     Tn, E, ws.Ep, k, pairs, dense, d_bias ? bias_part : nullptr, ws.chunks, (const T*)wr, H, wt);
  err = hipGetLastError();
  if (err != hipSuccess) return err;
  int hc = 128;   // columns per workgroup
  while (hc > kMinHc && (size_t)hc * E * sizeof(T) > kRouteSlice) hc /= 2;
  const int hb = (H + hc - 1) / hc, step = 256 / (hc / 8);
  const int unroll = hc == 128 && (int64_t)Tn * hb >= 2 * 64 * 2 * (int64_t)cu_count ? 4 : 1, chunk = unroll * step;
  const size_t lds = (size_t)hc * (E + 1) * sizeof(T) + 2 * (size_t)chunk * k * sizeof(RoutePair);
  // one wave of workgroups at two per CU, in whole chunks of tokens
  int64_t tb = 2 * (int64_t)cu_count / hb;
  const int64_t most = (Tn + chunk - 1) / chunk;
  if (tb > most) tb = most;
  if (tb < 1) tb = 1;
  const int64_t per = ((Tn + tb - 1) / tb + chunk - 1) / chunk * chunk;
  tb = (Tn + per - 1) / per;
  const RouteMain a{pairs, wt, bias_part, d_x, d_bias, Tn, H, E, k, hc, (int)per, hb, accumulate, ws.chunks};
  DenseProblem p{x, dense, H, ws.Ep, Tn, H, ws.Ep, ws.sp.splits, ws.sp.k_split};
  p.partial = ws.sp.splits > 1 ? part : nullptr;
  p.e.out = d_wr;
  p.e.cols = E;
  const int nx = (int)(tb * hb), nb = d_bias ? (E + 15) / 16 : 0;
  auto go = [&](auto u, auto kp) {
    constexpr int U = decltype(u)::value, KP = decltype(kp)::value;
    if (sizeof(T) == 2 && ws.Ep > 64) return launch_route_main<T, U, KP, DenseM>(a, p, nx, nb, lds, s);
    return launch_route_main<T, U, KP, DenseN>(a, p, nx, nb, lds, s);
  };
  const int kp = (chunk * k + 255) / 256;
  err = unroll == 1 ? (kp <= 4 ? go(Int<1>{}, Int<4>{}) : go(Int<1>{}, Int<16>{}))
        : kp <= 2   ? go(Int<4>{}, Int<2>{})
                    : go(Int<4>{}, Int<8>{});
  if (err != hipSuccess || !p.partial) return err;
  const int blocks = (int)(((int64_t)H * (ws.Ep / 8) + 255) / 256);
  hipLaunchKernelGGL(route_grad_finish<T>, dim3(blocks), dim3(256), 0, s, p);
  return hipGetLastError();
}

}  // namespace
}  // namespace moe

namespace moe_launch {

size_t route_backward_workspace_bytes(int dt, int T, int H, int E, int top_k, int cu_count) {
  return moe::route_ws(dt, T, H, E, top_k, cu_count).bytes;
}

int64_t route_backward_blocks(int T, int H, int E) {
  return (int64_t)((T + moe::kRgTokens - 1) / moe::kRgTokens) + (int64_t)((E + 63) / 64) * ((H + 63) / 64);
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
