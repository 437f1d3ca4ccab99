// The router's auxiliary losses, forward.
//
// With p[t] = softmax(logits[t]) over all experts, c[e] the slots of valid tokens
// that name expert e, S[e] the sum of p[t, e] over valid tokens and n their number:
//
//   balance = coef E / (top_k n^2) sum_e c[e] S[e]       (1 x coef when both are even)
//   z       = z_coef / n sum_t lse[t]^2,  lse[t] = log sum_e exp(logits[t, e])
//
// A router that sends many slots to an expert it also gives much probability has
// a large balance loss (VeOmni docs "Fused MoE Kernel Notes": skewed and duplicate
// routes make groups far larger than the mean).
//
// One pass over the logits, bound by reading them: 64 / G tokens per wave, G
// lanes and J values per lane for a token's experts, so a lane's probability sums
// stay in registers over all its tokens.  A workgroup leaves its sums in the
// workspace; one workgroup adds them in order.
#include "moe_common.h"

namespace moe {
namespace {

constexpr int kBalanceBlocks = 512;

// What a workgroup leaves: E probability sums, E counts, its sum of lse^2 and its valid tokens.
__host__ __device__ constexpr int balance_stride(int E) { return 2 * E + 2; }

struct BalanceArgs {
  const float* logits;
  const int32_t* ids;
  const uint8_t* mask;
  float* lse;
  float* part;
  int T, E, k;
};

template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int d = G / 2; d >= 1; d >>= 1) v += __shfl_xor(v, d, kWave);
  return v;
}
template <int G>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int d = G / 2; d >= 1; d >>= 1) v = fmaxf(v, __shfl_xor(v, d, kWave));
  return v;
}

template <int G, int J>
__global__ __launch_bounds__(256) void balance_sums(BalanceArgs a) {
  constexpr int P = kWave / G;   // tokens of a wave at a time
  __shared__ int32_t s_cnt[kMaxExperts];
  __shared__ float s_p[G * J], s_z[4 * P];
  __shared__ int32_t s_n[4 * P];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, g = lane % G, slot = lane / G;
  for (int e = tid; e < a.E; e += 256) s_cnt[e] = 0;
  __syncthreads();
  float sum[J], z = 0.f;
  int n = 0;
#pragma unroll
  for (int j = 0; j < J; ++j) sum[j] = 0.f;
  const int64_t step = (int64_t)gridDim.x * 4 * P;
  // every lane makes the same number of turns: the shuffles need all of a group
  for (int64_t t0 = (int64_t)blockIdx.x * 4 * P; t0 < a.T; t0 += step) {
    const int64_t t = t0 + wave * P + slot;
    const bool in = t < a.T;
    const bool valid = in && (!a.mask || a.mask[t]);
    const float* row = a.logits + t * a.E;
    float v[J];
#pragma unroll
    for (int j = 0; j < J; ++j) v[j] = valid && g + G * j < a.E ? row[g + G * j] : -INFINITY;
    float m = v[0];
#pragma unroll
    for (int j = 1; j < J; ++j) m = fmaxf(m, v[j]);
    m = group_max<G>(m);
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      v[j] = g + G * j < a.E ? expf(v[j] - m) : 0.f;
      s += v[j];
    }
    s = group_sum<G>(s);
    const float lse = valid ? m + logf(s) : 0.f;
    if (valid) {
      const float inv = 1.0f / s;
#pragma unroll
      for (int j = 0; j < J; ++j) sum[j] += v[j] * inv;
      if (g == 0) {
        z = fmaf(lse, lse, z);
        ++n;
      }
      for (int j = g; j < a.k; j += G) {
        const int id = a.ids[t * a.k + j];
        if (id >= 0 && id < a.E) atomicAdd(&s_cnt[id], 1);   // whole numbers: the order changes nothing
      }
    }
    if (in && g == 0 && a.lse) a.lse[t] = lse;
  }
  // a workgroup's sums: its groups of lanes in order
  for (int q = 0; q < 4 * P; ++q) {
    if (wave * P + slot == q) {
#pragma unroll
      for (int j = 0; j < J; ++j) s_p[g + G * j] = (q ? s_p[g + G * j] : 0.f) + sum[j];
      if (g == 0) {
        s_z[q] = z;
        s_n[q] = n;
      }
    }
    __syncthreads();
  }
  float* out = a.part + (int64_t)blockIdx.x * balance_stride(a.E);
  for (int e = tid; e < a.E; e += 256) {
    out[e] = s_p[e];
    out[a.E + e] = __int_as_float(s_cnt[e]);
  }
  if (tid == 0) {
    float zz = 0.f;
    int nn = 0;
    for (int q = 0; q < 4 * P; ++q) {
      zz += s_z[q];
      nn += s_n[q];
    }
    out[2 * a.E] = zz;
    out[2 * a.E + 1] = __int_as_float(nn);
  }
}

// One workgroup: the blocks' sums in order, then the losses (their last sums in
// fp64: their terms span many binades and there are few of them).
__global__ __launch_bounds__(1024) void balance_finish(const float* __restrict__ part, int blocks, int E, int k,
                                                       float coef, float z_coef, float* __restrict__ losses,
                                                       int32_t* __restrict__ counts, int32_t* __restrict__ tokens,
                                                       float* __restrict__ prob_sums) {
  __shared__ double s_loss[16];
  __shared__ double s_z;
  __shared__ int32_t s_n;
  const int tid = threadIdx.x, ld = balance_stride(E);
  double term = 0.0;
  for (int e = tid; e < E; e += 1024) {
    const float s = sum_slices(part + e, ld, blocks);
    int c = 0;
    for (int b = 0; b < blocks; ++b) c += __float_as_int(part[(int64_t)b * ld + E + e]);
    prob_sums[e] = s;
    counts[e] = c;
    term += (double)c * (double)s;
  }
  if (tid == 1023) {
    double z = 0.0;
    int n = 0;
    for (int b = 0; b < blocks; ++b) {
      z += (double)part[(int64_t)b * ld + 2 * E];
      n += __float_as_int(part[(int64_t)b * ld + 2 * E + 1]);
    }
    s_z = z;
    s_n = n;
  }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) term += __shfl_xor(term, d, kWave);
  if ((tid & 63) == 0) s_loss[tid >> 6] = term;
  __syncthreads();
  if (tid == 0) {
    double v = 0.0;
    for (int w = 0; w < 16; ++w) v += s_loss[w];
    const double n = s_n > 0 ? (double)s_n : 1.0;
    losses[0] = (float)((double)coef * E / k * v / (n * n));
    losses[1] = (float)((double)z_coef * s_z / n);
    tokens[0] = s_n;
  }
}

int balance_blocks(int T, int E) {
  const int g = E <= 8 ? 8 : E <= 16 ? 16 : E <= 32 ? 32 : 64;
  const int64_t per = 4 * (kWave / g), need = ((int64_t)T + per - 1) / per;
  return (int)(need < kBalanceBlocks ? need : kBalanceBlocks);
}

template <int G, int J>
void launch_sums(const BalanceArgs& a, int blocks, hipStream_t s) {
  hipLaunchKernelGGL((balance_sums<G, J>), dim3(blocks), dim3(256), 0, s, a);
}

}  // namespace
}  // namespace moe

namespace moe_launch {

size_t balance_loss_workspace_bytes(int T, int E) {
  return ((size_t)moe::balance_blocks(T, E) * moe::balance_stride(E) * sizeof(float) + 255) & ~(size_t)255;
}

hipError_t balance_loss(const float* logits, const int32_t* ids, const uint8_t* mask, int T, int E, int top_k,
                        float coef, float z_coef, float* losses, int32_t* counts, int32_t* tokens, float* prob_sums,
                        float* lse, void* ws, hipStream_t s) {
  const moe::BalanceArgs a{logits, ids, mask, lse, (float*)ws, T, E, top_k};
  const int blocks = moe::balance_blocks(T, E);
  if (E <= 8) moe::launch_sums<8, 1>(a, blocks, s);
  else if (E <= 16) moe::launch_sums<16, 1>(a, blocks, s);
  else if (E <= 32) moe::launch_sums<32, 1>(a, blocks, s);
  else if (E <= 64) moe::launch_sums<64, 1>(a, blocks, s);
  else if (E <= 128) moe::launch_sums<64, 2>(a, blocks, s);
  else if (E <= 256) moe::launch_sums<64, 4>(a, blocks, s);
  else if (E <= 512) moe::launch_sums<64, 8>(a, blocks, s);
  else moe::launch_sums<64, 16>(a, blocks, s);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  hipLaunchKernelGGL(moe::balance_finish, dim3(1), dim3(1024), 0, s, (const float*)ws, blocks, E, top_k, coef, z_coef,
                     losses, counts, tokens, prob_sums);
  return hipGetLastError();
}

}  // namespace moe_launch
