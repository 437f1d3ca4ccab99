// Dense GEMMs of the shared expert in training: both forward halves and the
// input and weight gradients of both, with their elementwise work fused in.
//
// PLENA_Compiler PR #69, section "Group C -- shared experts": the shared expert
// is a dense FFN over every token.  Its training passes are the chain rule of
//
//   h = x Ws1 = [g | u],   a = silu(g) u,   ys = a Ws2,   y (+)= gate ys
//
// so they need six products: x Ws1 (SwiGLU epilogue, h and a stored), a Ws2
// (gate epilogue), D Ws2^T (SwiGLU' epilogue), d_h Ws1^T (gate gradient added),
// and the two weight gradients A^T D; moe_dense.h holds the product itself.
//
//  * A reduction can be split over workgroups when the output has too few
//    tiles to fill the chip: partial sums go to the workspace in fp32 and
//    dense_finish adds them in split order and runs the same epilogue, so
//    results do not depend on timing.
#include "moe_dense.h"

namespace moe {
namespace {

template <class C, bool ACOL, bool BCOL, int EPI>
__global__ __launch_bounds__(C::NT, dense_min_waves<C>()) void dense_bf16(DenseProblem p) {
  extern __shared__ __attribute__((aligned(1024))) unsigned char smem[];
  dense_tile<C, ACOL, BCOL, EPI>(p, blockIdx.x, smem);
}

// The gate weight's gradient, sum over t of d_z[t] x[t, h]: `blocks` workgroups
// (0: no gate), one per chunk of kGateRows rows and 64 columns.  8 lanes hold a
// row's columns (16 bytes each in bf16), NT / 8 groups take every NT / 8th row, eight
// rows at a time, and their sums are added in group order.  One chunk: the result,
// in the element type; more: partial sums [chunks, H].
constexpr int kGateRows = 512;
struct GateGrad {
  const float* d_z;
  const void* x;
  int Tn, H, chunks, blocks;
  float* part;
  void* d_wg;
};
template <typename T, int NT>
__device__ __forceinline__ void dense_gate_grad(const GateGrad& p, int unit, float* s_part) {
  constexpr int G = NT / 8;
  const int c = threadIdx.x & 7, g = threadIdx.x >> 3;
  const int chunk = unit % p.chunks, h0 = unit / p.chunks * 64, h = h0 + 8 * c, H = p.H;
  const T* x = (const T*)p.x;
  const int64_t t0 = (int64_t)chunk * kGateRows, t1 = min(t0 + kGateRows, (int64_t)p.Tn);
  float s[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (h < H)
    for (int64_t t = t0 + g; t < t1; t += 8 * G) {
      float a[8][8], z[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int64_t tu = min(t + G * u, t1 - 1);
        load8(x + tu * H + h, a[u]);
        z[u] = p.d_z[tu];
      }
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (t + G * u < t1)
#pragma unroll
          for (int i = 0; i < 8; ++i) s[i] = fmaf(z[u], a[u][i], s[i]);
    }
  store8(s_part + g * 64 + 8 * c, s);
  __syncthreads();
  const int col = h0 + threadIdx.x;
  if (threadIdx.x >= 64 || col >= H) return;
  float v = 0.f;
#pragma unroll
  for (int q = 0; q < G; ++q) v += s_part[q * 64 + threadIdx.x];
  if (p.chunks == 1)
    store_from_f32((T*)p.d_wg, col, v);
  else
    p.part[(int64_t)chunk * H + col] = v;
}

// The two products of a half's backward in one launch: the input gradient (d)
// and the weight gradient (w).  Their tiles have different reduction lengths;
// the host puts the longer ones first (n_first units of them), so the
// dispatcher fills the CUs that finish early with the shorter ones, and the
// epilogues of the two kinds do not run at the same time on every CU.  The gate
// weight's gradient fills in at the end (its own launch took 4 us).
template <class CD, class CW, bool BCOL, int EPI>
__global__ __launch_bounds__(CD::NT, dense_min_waves<CW>()) void dense_pair_bf16(DenseProblem d, DenseProblem w,
                                                                                 int n_first, int w_first, int n_all,
                                                                                 GateGrad g) {
  static_assert(CD::NT == CW::NT, "one workgroup size");
  extern __shared__ __attribute__((aligned(1024))) unsigned char smem[];
  const int u = blockIdx.x;
  if (EPI == kEInputGrad && u >= n_all)
    dense_gate_grad<bf16_t, CD::NT>(g, u - n_all, (float*)smem);
  else if ((u < n_first) != (w_first != 0))
    dense_tile<CD, false, BCOL, EPI>(d, w_first ? u - n_first : u, smem);
  else
    dense_tile<CW, true, true, kEStore>(w, w_first ? u : u - n_first, smem);
}

// Adds the splits' partial sums in split order and runs the epilogue.
template <typename T, int EPI>
__global__ __launch_bounds__(256) void dense_finish(DenseProblem p) {
  constexpr bool PAIRED = dense_paired<EPI>();
  const int per_row = p.N / 8;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)p.M * per_row) return;
  const int64_t m = i / per_row;
  const int n = 8 * (int)(i % per_row);
  const int64_t ps = (int64_t)p.M * (PAIRED ? 2 * p.N : p.N);
  const float* s = p.partial + m * (PAIRED ? 2 * p.N : p.N) + n;
  // U splits' loads in flight together (clamped, not predicated).  Whole calls:
  // first half at 8 tokens, 4096 x 2816, 14.5 -> 13.7 us against one split after the
  // other, second half at 16 tokens, 4096 x 2048, 12.8 -> 10.5.
  constexpr int NB = PAIRED ? 2 : 1, U = PAIRED ? 4 : 8;
  float v[NB][8];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int q = 0; q < 8; ++q) v[b][q] = 0.f;
  for (int z = 0; z < p.splits; z += U) {
    f32x4 x[U][NB][2];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const f32x4* at = (const f32x4*)(s + min(z + u, p.splits - 1) * ps + b * p.N);
        x[u][b][0] = at[0];
        x[u][b][1] = at[1];
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (z + u < p.splits)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int q = 0; q < 8; ++q) v[b][q] += x[u][b][q / 4][q % 4];
  }
  epi8_now<T, EPI>(p.e, m, n, p.N, v[0], v[NB - 1]);
}

template <bool ACOL, bool BCOL, int EPI>
__global__ __launch_bounds__(256) void dense_f32(DenseProblem p) {
  __shared__ __attribute__((aligned(16))) float smem[dense_f32_lds<EPI>()];
  dense_f32_tile<ACOL, BCOL, EPI>(p, blockIdx.x, smem);
}

// Both products of a half's backward, and the gate weight's gradient, in one launch.
template <bool BCOL, int EPI>
__global__ __launch_bounds__(256) void dense_f32_pair(DenseProblem d, DenseProblem w, int nd, int n_all, GateGrad g) {
  __shared__ __attribute__((aligned(16))) float smem[dense_f32_lds<EPI>()];
  const int u = blockIdx.x;
  if (EPI == kEInputGrad && u >= n_all)
    dense_gate_grad<float, 256>(g, u - n_all, smem);
  else if (u < nd)
    dense_f32_tile<false, BCOL, EPI>(d, u, smem);
  else
    dense_f32_tile<true, true, kEStore>(w, u - nd, smem);
}

// ------------------------------------------------------------------------------------------
// Elementwise and reduction steps
// ------------------------------------------------------------------------------------------
// Workgroups of dense_gate and dense_dy, a wave per token, looping past 2^24 tokens:
// without the cap 2^26 tokens would need more than a launch's 2^32 - 1 threads.
constexpr int kTokenBlocks = 1 << 22;
unsigned token_blocks(int T) { return (unsigned)min((T + 3) / 4, kTokenBlocks); }

// One wave per token.  gate[t] = sigmoid(x[t] . w_gate), fp32.
template <typename T>
__global__ __launch_bounds__(256) void dense_gate(const T* __restrict__ x, const T* __restrict__ wg, int Tn, int H,
                                                  float* __restrict__ gate) {
  const int lane = threadIdx.x & 63;
  for (int64_t t = blockIdx.x * 4 + (threadIdx.x >> 6); t < Tn; t += 4 * (int64_t)gridDim.x) {
    float s = 0.f;
    for (int h = 8 * lane; h < H; h += 512) {
      float a[8], b[8];
      load8(x + t * H + h, a);
      load8(wg + h, b);
#pragma unroll
      for (int i = 0; i < 8; ++i) s = fmaf(a[i], b[i], s);
    }
    s = wave_sum(s);
    if (lane == 0) gate[t] = sigmoidf_(s);
  }
}

// One wave per token: d_rows[t] = gate[t] * dy[t] in the element type (null: not
// wanted), and the gate logit's gradient gate (1 - gate) (dy[t] . ys[t]).
//
// In bf16 this rounds an fp32 input of both products, as moe_scatter_grad does for
// the routed experts: bf16 MFMAs take no wider operand, fp32's run at a sixteenth of
// their rate, and a high and a low bf16 part would double both products (4096 tokens,
// 2048 x 5632: 158 us of them).  d_h and d_ws2 then carry this rounding and that of
// their own store: relative error 0.0023 against float64, where the store alone has
// 0.0017 (517 and 4096 tokens).
template <typename T>
__global__ __launch_bounds__(256) void dense_dy(const float* __restrict__ dy, const float* __restrict__ ys,
                                                const float* __restrict__ gate, int Tn, int H, T* __restrict__ d_rows,
                                                float* __restrict__ d_z) {
  const int lane = threadIdx.x & 63;
  for (int64_t t = blockIdx.x * 4 + (threadIdx.x >> 6); t < Tn; t += 4 * (int64_t)gridDim.x) {
    const float g = gate ? gate[t] : 1.0f;
    const int64_t base = t * H;
    float s = 0.f;
    for (int h = 8 * lane; h < H; h += 512) {
      float a[8], b[8];
      load8(dy + base + h, a);
      if (gate) {
        load8(ys + base + h, b);
#pragma unroll
        for (int i = 0; i < 8; ++i) s = fmaf(a[i], b[i], s);
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] *= g;
      }
      if (d_rows) store8(d_rows + base + h, a);
    }
    if (!gate) continue;
    s = wave_sum(s);
    if (lane == 0) d_z[t] = g * (1.0f - g) * s;
  }
}

template <typename T>
__global__ __launch_bounds__(256) void dense_gate_grad_sum(const float* __restrict__ part, int chunks, int H,
                                                           T* __restrict__ d_wg) {
  const int h = blockIdx.x * 256 + threadIdx.x;
  if (h < H) store_from_f32(d_wg, h, sum_slices(part + h, H, chunks));
}

// ------------------------------------------------------------------------------------------
// Host: configurations and their choice
// ------------------------------------------------------------------------------------------
typedef DenseCfg<256, 256, 2, 2> DenseL;      // 4 waves of 128 x 128, one workgroup per CU
typedef DenseCfg<256, 256, 2, 4> DenseL8;     // 8 waves of 128 x 64
typedef DenseCfg<64, 128, 2, 2> DenseS;       // 4 waves of 32 x 64, two per CU
typedef DenseCfg<64, 128, 2, 2, 2> DenseS2;   // two such groups on alternate slices, one workgroup per CU
typedef DenseCfg<128, 128, 2, 2, 2> DenseM2;  // two groups of DenseM's waves, one workgroup per CU
typedef DenseCfg<64, 64, 2, 1, 4> DenseS4;    // four groups of 2 waves of 32 x 64, one workgroup per CU

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

// The 256 x 256 tile has four waves, whose 128 x 128 pieces read a third less
// LDS than eight waves' 128 x 64 (measured, Scout-shaped fc2 forward at 2048
// tokens 165 against 178 us; fc1 backward at 4096 tokens 330 against 336), except
// with SwiGLU's gradient as the epilogue, whose loads and arithmetic want two
// waves per SIMD (fc2 backward at 4096 tokens 218 against 253 us: the input
// gradient's tiles alone 141 against 161, the weight's, which share its launch and
// so its workgroup size, 89 against 84).
template <int EPI>
using DenseLarge = std::conditional_t<EPI == kESwigluBwd, DenseL8, DenseL>;

// A configuration's tile, its workgroups per CU, and microseconds: per 64-deep
// slice with one workgroup on a CU and with every slot taken, and per tile
// besides its slices.  Fitted to 25000 measured times: 600 random layers (1 to
// 8192 tokens, widths 128 to 8192) with every choice and split, most of them with
// inputs that change from pass to pass.  What the model picks takes 2 to 3 %
// longer than the best choice (geometric mean; 100 layers that the fit had not
// seen); without S4, M2 and the fit it was 4 to 9 %.
// kShapeL stands for both 256 x 256 tiles: with SwiGLU's gradient a tile takes about
// 20 us more than its `fixed` says (fc2 backward at 4096 tokens: 200 us, 160 by the
// model, which picks the best of its choices all the same).
struct DenseShape {
  int bm, bn, slots;
  double alone, full, fixed;
};
constexpr DenseShape kShapeL{256, 256, 1, 1.04, 1.45, 7.0}, kShapeM{128, 128, 2, 0.69, 0.89, 2.2},
    kShapeS{64, 128, 2, 0.49, 0.70, 2.2}, kShapeS2{64, 128, 1, 0.31, 0.33, 3.5},
    kShapeM2{128, 128, 1, 0.30, 0.48, 4.8}, kShapeS4{64, 64, 1, 0.18, 0.194, 4.2};
// `full` of S4 where its 32 gate and 32 up columns are 64-byte pieces of a stored
// row: half a cache line each, the other half another workgroup's.
constexpr double kS4HalfLines = 0.45;
// Choices for one product, for the input and the weight gradient of a pair
// (which share a launch, so their workgroups have as many threads), or for
// either.  The groups of S2, M2 and S4 work on alternate slices, which shortens a
// tile's chain where there are fewer tiles than CUs.
struct DenseChoice {
  DenseShape d, w;
  bool one, pair;
};
constexpr DenseChoice kChoices[8] = {{kShapeL, kShapeL, true, true},    {kShapeM, kShapeM, true, true},
                                     {kShapeS, kShapeS, true, true},    {kShapeS2, kShapeS2, true, false},
                                     {kShapeS, kShapeM, false, true},   {kShapeM2, kShapeM2, true, false},
                                     {kShapeS4, kShapeS4, true, false}, {kShapeS4, kShapeM2, false, true}};
// A split product's second launch, and its partial sums' trip through memory.
constexpr double kFinishUs = 3.2, kFinishUsPaired = 4.2, kFinishUsPerMb = 0.34;

// One product's tiles: M x Ns outputs (Ns counts the staged columns: both halves
// of a paired product), K reduced.  half_lines: paired, the weight stored [K, 2N].
struct DenseWork {
  int M, Ns, K;
  bool paired = false, half_lines = false;
};
int64_t work_tiles(const DenseWork& w, const DenseShape& c) {
  return (int64_t)((w.M + c.bm - 1) / c.bm) * ((w.Ns + c.bn - 1) / c.bn);
}
int work_slices(const DenseWork& w) { return (w.K + kDBK - 1) / kDBK; }

// Time of nl tiles of length l followed by ns tiles of length s (l >= s) on P
// slots, each slot taking the next tile when it is free: the smallest time by
// which the slots without a last long tile (free from t0) and those with one
// (free from t1) have room for all the short tiles.
double two_class_time(int64_t nl, double l, int64_t ns, double s, int64_t P) {
  const int64_t nr = nl % P, nf = P - nr;
  const double t0 = (double)(nl / P) * l, t1 = nr ? t0 + l : t0;
  if (ns == 0) return t1;
  double est = t0 + (double)ns * s / nf;                              // all in the free slots
  if (est > t1) est = ((double)ns * s + nf * t0 + nr * t1) / P;       // else spread over all
  int64_t kf = (int64_t)((est - t0) / s), kr = est > t1 ? (int64_t)((est - t1) / s) : 0;
  double end = est;
  for (int it = 0; it < 64 && kf * nf + kr * nr < ns; ++it) {
    const double a = t0 + (kf + 1) * s, b = nr ? t1 + (kr + 1) * s : a;
    if (a <= b) ++kf; else ++kr;
    end = a < b ? a : b;
  }
  return end > t1 ? end : t1;
}

struct DensePlan {
  int choice;
  int splits[2], k_split[2];
  bool w_first;   // the weight gradient's tiles are the longer ones
  double us;
};

// Bytes of partial sums a call may use: up to 16 splits of its widest product, at
// most 64 MiB (a product that large fills the chip without splitting).
size_t partial_cap(int T, int H, int I_s) {
  const int64_t a = (int64_t)T * 2 * I_s, b = (int64_t)T * H, c = (int64_t)H * 2 * I_s;
  const int64_t most = a > b ? (a > c ? a : c) : (b > c ? b : c);
  const int64_t bytes = 16 * 4 * most, cap = (int64_t)64 << 20;
  return align256((size_t)(bytes < cap ? bytes : cap));
}

size_t split_bytes(const DenseWork& w, int splits) {
  return splits > 1 ? align256((size_t)splits * w.M * w.Ns * 4) : 0;
}

// Cheapest tiles and reduction splits for one product, or for two that share a
// launch (w[1].M > 0), by a model of the dispatch: slots take tiles in order,
// longer ones first, and slow down as a CU's slots fill; a split product pays
// for writing and adding its partial sums (at most `cap` bytes).
DensePlan dense_plan(const DenseWork (&w)[2], size_t cap, int cu_count) {
  static constexpr int kSplits[2][8] = {{1, 2, 3, 4, 6, 8, 12, 16}, {1, 2, 4, 8, 0, 0, 0, 0}};
  DensePlan best{1, {1, 1}, {kDBK, kDBK}, false, 1e30};
  const int products = w[1].M > 0 ? 2 : 1;
  for (int c = 0; c < 8; ++c) {
    if (!(products == 2 ? kChoices[c].pair : kChoices[c].one)) continue;
    const DenseShape* sh[2] = {&kChoices[c].d, &kChoices[c].w};
    const int64_t slots = (int64_t)cu_count * sh[0]->slots;
    for (int s0 : kSplits[0])
      for (int s1 : kSplits[1]) {
        if (s1 == 0 || (products == 1 && s1 > 1)) break;
        const int sp[2] = {s0, s1};
        if (split_bytes(w[0], s0) + split_bytes(w[1], s1) > cap) break;
        double len[2] = {0, 0}, extra = 0;
        int64_t units[2] = {0, 0};
        int per[2] = {1, 1};
        bool ok = true;
        for (int q = 0; q < products; ++q) {
          const int n = work_slices(w[q]);
          per[q] = (n + sp[q] - 1) / sp[q];
          if (sp[q] > 1 && (per[q] < 4 || (n + per[q] - 1) / per[q] != sp[q])) ok = false;
          units[q] = work_tiles(w[q], *sh[q]) * sp[q];
          if (sp[q] > 1)
            extra += (w[q].paired ? kFinishUsPaired : kFinishUs) +
                     kFinishUsPerMb * sp[q] * ((double)w[q].M * w[q].Ns * 4e-6);
        }
        if (!ok) continue;
        // average share of the slots at work while the longest tile runs
        double work = 0, chain = 0;
        double full[2];
        for (int q = 0; q < products; ++q) {
          full[q] = w[q].half_lines && sh[q]->bn == kShapeS4.bn ? kS4HalfLines : sh[q]->full;
          const double one = per[q] * full[q];
          work += one * units[q];
          chain = one > chain ? one : chain;
        }
        double occ = work / (chain * slots);
        occ = occ < 1.0 ? occ : 1.0;
        const double shared = (occ * slots - cu_count) / (slots - cu_count + 1e-9);
        const double busy = sh[0]->slots == 1 ? occ : shared > 0 ? shared : 0.0;
        for (int q = 0; q < products; ++q)
          len[q] = per[q] * (sh[q]->alone + busy * (full[q] - sh[q]->alone)) + sh[q]->fixed;
        const int a = len[0] >= len[1] ? 0 : 1;
        const double us =
            two_class_time(units[a], len[a], units[1 - a], len[1 - a] > 0 ? len[1 - a] : 1.0, slots) + extra;
        if (us < best.us)
          best = DensePlan{c, {s0, s1}, {per[0] * kDBK, per[1] * kDBK}, a == 1, us};
      }
  }
  return best;
}

template <class C, bool PAIRED>
void set_tiles(DenseProblem& p) {
  const int out = PAIRED ? C::BN / 2 : C::BN;
  p.m_tiles = (p.M + C::BM - 1) / C::BM;
  p.n_tiles = (p.N + out - 1) / out;
}

template <typename T, int EPI>
hipError_t launch_finish(const DenseProblem& p, hipStream_t s) {
  const int64_t n = (int64_t)p.M * (p.N / 8);
  hipLaunchKernelGGL((dense_finish<T, EPI>), dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, p);
  return hipGetLastError();
}

template <class C, bool ACOL, bool BCOL, int EPI>
hipError_t launch_dense_cfg(DenseProblem p, hipStream_t s) {
  static std::atomic<uint64_t> lds_done{0};
  hipError_t err = allow_lds(reinterpret_cast<const void*>(&dense_bf16<C, ACOL, BCOL, EPI>), C::kLds, lds_done);
  if (err != hipSuccess) return err;
  set_tiles<C, dense_paired<EPI>()>(p);
  hipLaunchKernelGGL((dense_bf16<C, ACOL, BCOL, EPI>), dim3(p.m_tiles * p.n_tiles * p.splits), dim3(C::NT), C::kLds, s,
                     p);
  return hipGetLastError();
}

template <class CD, class CW, bool BCOL, int EPI>
hipError_t launch_pair_cfg(DenseProblem d, DenseProblem w, bool w_first, const GateGrad& g, hipStream_t s) {
  constexpr int lds = CD::kLds > CW::kLds ? CD::kLds : CW::kLds;
  static std::atomic<uint64_t> lds_done{0};
  hipError_t err = allow_lds(reinterpret_cast<const void*>(&dense_pair_bf16<CD, CW, BCOL, EPI>), lds, lds_done);
  if (err != hipSuccess) return err;
  set_tiles<CD, false>(d);
  set_tiles<CW, false>(w);
  const int nd = d.m_tiles * d.n_tiles * d.splits, nw = w.m_tiles * w.n_tiles * w.splits;
  hipLaunchKernelGGL((dense_pair_bf16<CD, CW, BCOL, EPI>), dim3(nd + nw + g.blocks), dim3(CD::NT), lds, s, d, w,
                     w_first ? nw : nd, w_first ? 1 : 0, nd + nw, g);
  return hipGetLastError();
}

void set_tiles_f32(DenseProblem& p) {
  p.m_tiles = (p.M + 31) / 32;
  p.n_tiles = (p.N + 31) / 32;
}

template <bool ACOL, bool BCOL, int EPI>
hipError_t launch_f32(DenseProblem p, hipStream_t s) {
  set_tiles_f32(p);
  hipLaunchKernelGGL((dense_f32<ACOL, BCOL, EPI>), dim3(p.m_tiles * p.n_tiles * p.splits), dim3(256), 0, s, p);
  return hipGetLastError();
}

template <bool BCOL, int EPI>
hipError_t launch_f32_pair(DenseProblem d, DenseProblem w, const GateGrad& g, hipStream_t s) {
  set_tiles_f32(d);
  set_tiles_f32(w);
  const int nd = d.m_tiles * d.n_tiles, n_all = nd + w.m_tiles * w.n_tiles;
  hipLaunchKernelGGL((dense_f32_pair<BCOL, EPI>), dim3(n_all + g.blocks), dim3(256), 0, s, d, w, nd, n_all, g);
  return hipGetLastError();
}

void whole_reduction(DenseProblem& p) {
  p.splits = 1;
  p.k_split = (p.K + kDBK - 1) / kDBK * kDBK;
}

template <int EPI>
DenseWork work_of(const DenseProblem& p) {
  return DenseWork{p.M, dense_paired<EPI>() ? 2 * p.N : p.N, p.K, dense_paired<EPI>()};
}

// One product; B is the weight (b_col: stored [K, N], else [N, K]).
template <int EPI>
hipError_t launch_forward(int dt, bool b_col, DenseProblem p, float* partial, size_t cap, int cu_count, hipStream_t s) {
  whole_reduction(p);
  if (dt != 1) return b_col ? launch_f32<false, true, EPI>(p, s) : launch_f32<false, false, EPI>(p, s);
  DenseWork w[2] = {work_of<EPI>(p), {0, 0, 0}};
  w[0].half_lines = dense_paired<EPI>() && b_col;
  const DensePlan plan = dense_plan(w, cap, cu_count);
  p.splits = plan.splits[0];
  p.k_split = plan.k_split[0];
  p.partial = p.splits > 1 ? partial : nullptr;
  auto go = [&](auto c) {
    typedef decltype(c) C;
    return b_col ? launch_dense_cfg<C, false, true, EPI>(p, s) : launch_dense_cfg<C, false, false, EPI>(p, s);
  };
  const hipError_t err = plan.choice == 0   ? go(DenseLarge<EPI>{})
                         : plan.choice == 1 ? go(DenseM{})
                         : plan.choice == 2 ? go(DenseS{})
                         : plan.choice == 3 ? go(DenseS2{})
                         : plan.choice == 5 ? go(DenseM2{})
                                            : go(DenseS4{});
  if (err != hipSuccess || !p.partial) return err;
  return launch_finish<bf16_t, EPI>(p, s);
}

// The two products of a half's backward: d (epilogue EPI, B the weight) and w (the weight's gradient).
template <int EPI>
hipError_t launch_backward(int dt, bool b_col, DenseProblem d, DenseProblem w, const GateGrad& g, float* partial,
                           size_t cap, int cu_count, hipStream_t s) {
  whole_reduction(d);
  whole_reduction(w);
  if (dt != 1) return b_col ? launch_f32_pair<true, EPI>(d, w, g, s) : launch_f32_pair<false, EPI>(d, w, g, s);
  const DenseWork work[2] = {work_of<EPI>(d), work_of<kEStore>(w)};
  const DensePlan plan = dense_plan(work, cap, cu_count);
  d.splits = plan.splits[0];
  d.k_split = plan.k_split[0];
  w.splits = plan.splits[1];
  w.k_split = plan.k_split[1];
  d.partial = d.splits > 1 ? partial : nullptr;
  w.partial = w.splits > 1 ? partial + split_bytes(work[0], d.splits) / 4 : nullptr;
  auto go = [&](auto cd, auto cw) {
    typedef decltype(cd) CD;
    typedef decltype(cw) CW;
    return b_col ? launch_pair_cfg<CD, CW, true, EPI>(d, w, plan.w_first, g, s)
                 : launch_pair_cfg<CD, CW, false, EPI>(d, w, plan.w_first, g, s);
  };
  typedef DenseLarge<EPI> Large;
  hipError_t err = plan.choice == 0   ? go(Large{}, Large{})
                   : plan.choice == 1 ? go(DenseM{}, DenseM{})
                   : plan.choice == 2 ? go(DenseS{}, DenseS{})
                   : plan.choice == 4 ? go(DenseS{}, DenseM{})
                                      : go(DenseS4{}, DenseM2{});
  if (err == hipSuccess && d.partial) err = launch_finish<bf16_t, EPI>(d, s);
  if (err == hipSuccess && w.partial) err = launch_finish<bf16_t, kEStore>(w, s);
  return err;
}

}  // namespace
}  // namespace moe

namespace moe_launch {

using moe::DenseEpiArgs;
using moe::DenseProblem;

// Workspace: d_rows [T, H] of fc2's backward or d_w_gate's partial sums of fc1's,
// then the partial sums of split products.
size_t shared_front_bytes(int dt, int T, int H) {
  const size_t rows = moe::align256((size_t)T * H * (dt == 1 ? 2 : 4));
  const size_t part = moe::align256((size_t)((T + moe::kGateRows - 1) / moe::kGateRows) * H * 4);
  return rows > part ? rows : part;
}

size_t shared_train_workspace_bytes(int dt, int T, int H, int I_s) {
  return shared_front_bytes(dt, T, H) + (dt == 1 ? moe::partial_cap(T, H, I_s) : 0);
}

float* shared_partials(void* ws, int dt, int T, int H) { return (float*)((char*)ws + shared_front_bytes(dt, T, H)); }

int shared_train_tiles(int dt, int call, int wl, int T, int H, int I_s, int cu_count, int32_t* splits) {
  using namespace moe;
  splits[0] = splits[1] = 1;
  if (dt != 1) return MOE_DENSE_F32;
  DenseWork w[2] = {{T, 2 * I_s, H, true, wl == 0}, {0, 0, 0}};
  if (call == 1) w[0] = DenseWork{T, H, I_s};
  if (call == 2) {
    w[0] = DenseWork{T, I_s, H};
    w[1] = wl ? DenseWork{H, I_s, T} : DenseWork{I_s, H, T};
  }
  if (call == 3) {
    w[0] = DenseWork{T, H, 2 * I_s};
    w[1] = wl ? DenseWork{2 * I_s, H, T} : DenseWork{H, 2 * I_s, T};
  }
  const DensePlan p = dense_plan(w, partial_cap(T, H, I_s), cu_count);
  splits[0] = p.splits[0];
  splits[1] = p.splits[1];
  return MOE_DENSE_256x256 + p.choice;
}

int64_t shared_f32_blocks(int call, int T, int H, int I_s) {
  auto tiles = [](int64_t m, int64_t n) { return ((m + 31) / 32) * ((n + 31) / 32); };
  switch (call) {
    case 0: return tiles(T, I_s);
    case 1: return tiles(T, H);
    case 2: return tiles(T, I_s) + tiles(I_s, H);
    default:
      return tiles(T, H) + tiles(2 * (int64_t)I_s, H) +
             (int64_t)((T + moe::kGateRows - 1) / moe::kGateRows) * ((H + 63) / 64);
  }
}

hipError_t shared_fc1_save(int dt, int wl, const void* x, const void* ws1, int T, int H, int I_s, void* act,
                           void* h_pre, void* ws, int cu_count, hipStream_t s) {
  DenseProblem p{x, ws1, T, I_s, H, H, wl ? H : 2 * I_s};
  p.e = DenseEpiArgs{act, h_pre, nullptr, nullptr, nullptr, 0};
  return moe::launch_forward<moe::kESwigluSave>(dt, wl == 0, p, shared_partials(ws, dt, T, H),
                                               moe::partial_cap(T, H, I_s), cu_count, s);
}

hipError_t shared_fc2_save(int dt, int wl, const void* act, const void* ws2, const void* x, const void* w_gate, int T,
                           int H, int I_s, int accumulate, float* y, float* y_shared, float* gate, void* ws,
                           int cu_count, hipStream_t s) {
  using namespace moe;
  if (w_gate) {
    const dim3 grid(token_blocks(T));
    if (dt == 1)
      hipLaunchKernelGGL(dense_gate<bf16_t>, grid, dim3(256), 0, s, (const bf16_t*)x, (const bf16_t*)w_gate, T, H,
                         gate);
    else
      hipLaunchKernelGGL(dense_gate<float>, grid, dim3(256), 0, s, (const float*)x, (const float*)w_gate, T, H, gate);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  DenseProblem p{act, ws2, T, H, I_s, I_s, wl ? I_s : H};
  p.e = DenseEpiArgs{y, w_gate ? y_shared : nullptr, nullptr, w_gate ? gate : nullptr, nullptr, accumulate};
  return launch_forward<kEGateAdd>(dt, wl == 0, p, shared_partials(ws, dt, T, H), partial_cap(T, H, I_s), cu_count, s);
}

hipError_t shared_fc2_backward(int dt, int wl, const float* dy, const void* act, const void* h_pre, const void* ws2,
                               const float* y_shared, const float* gate, int T, int H, int I_s, void* d_h, void* d_ws2,
                               float* d_z, void* ws, int cu_count, hipStream_t s) {
  using namespace moe;
  const void* rows = ws;
  const dim3 grid(token_blocks(T));
  if (dt == 1)
    hipLaunchKernelGGL(dense_dy<bf16_t>, grid, dim3(256), 0, s, dy, y_shared, gate, T, H, (bf16_t*)ws, d_z);
  else if (gate)
    hipLaunchKernelGGL(dense_dy<float>, grid, dim3(256), 0, s, dy, y_shared, gate, T, H, (float*)ws, d_z);
  else
    rows = dy;
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  // da = d_rows Ws2^T: reduction H, outputs I_s; Ws2 [I_s, H] is the "row" form here
  DenseProblem d{rows, ws2, T, I_s, H, H, wl ? I_s : H};
  d.e = DenseEpiArgs{d_h, nullptr, h_pre, nullptr, nullptr, 0};
  DenseProblem w = wl ? DenseProblem{rows, act, H, I_s, T, H, I_s} : DenseProblem{act, rows, I_s, H, T, I_s, H};
  w.e = DenseEpiArgs{d_ws2, nullptr, nullptr, nullptr, nullptr, 0};
  return launch_backward<kESwigluBwd>(dt, wl == 1, d, w, GateGrad{}, shared_partials(ws, dt, T, H),
                                      partial_cap(T, H, I_s), cu_count, s);
}

hipError_t shared_fc1_backward(int dt, int wl, const void* d_h, const void* x, const void* ws1, const float* d_z,
                               const void* w_gate, int T, int H, int I_s, int accumulate, float* d_x, void* d_ws1,
                               void* d_w_gate, void* ws, int cu_count, hipStream_t s) {
  using namespace moe;
  // d_x = d_h Ws1^T: reduction 2 I_s, outputs H; Ws1 [H, 2 I_s] is the "row" form here
  DenseProblem d{d_h, ws1, T, H, 2 * I_s, 2 * I_s, wl ? H : 2 * I_s};
  d.e = DenseEpiArgs{d_x, nullptr, nullptr, w_gate ? d_z : nullptr, w_gate, accumulate};
  DenseProblem w = wl ? DenseProblem{d_h, x, 2 * I_s, H, T, 2 * I_s, H}
                      : DenseProblem{x, d_h, H, 2 * I_s, T, H, 2 * I_s};
  w.e = DenseEpiArgs{d_ws1, nullptr, nullptr, nullptr, nullptr, 0};
  GateGrad g{d_z, x, T, H, (T + kGateRows - 1) / kGateRows, 0, (float*)ws, d_w_gate};
  if (w_gate) g.blocks = g.chunks * ((H + 63) / 64);
  const hipError_t err = launch_backward<kEInputGrad>(dt, wl == 1, d, w, g, shared_partials(ws, dt, T, H),
                                                      partial_cap(T, H, I_s), cu_count, s);
  if (err != hipSuccess || !w_gate || g.chunks == 1) return err;
  const dim3 grid((H + 255) / 256);
  if (dt == 1)
    hipLaunchKernelGGL(dense_gate_grad_sum<bf16_t>, grid, dim3(256), 0, s, g.part, g.chunks, H, (bf16_t*)d_w_gate);
  else
    hipLaunchKernelGGL(dense_gate_grad_sum<float>, grid, dim3(256), 0, s, g.part, g.chunks, H, (float*)d_w_gate);
  return hipGetLastError();
}

}  // namespace moe_launch
