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
// One pass over the logits (32768 tokens, 256 experts: 13 us, 2.7 TB/s, and 6 for the
// sums; with 512 workgroups 12 and 7), bound by reading them: G lanes share a token, four
// neighbouring experts per lane, up to four times (few lanes: the softmax's maximum
// and sum take log2 G exchanges for 64 / G tokens at once), and U such groups of
// tokens are in flight; a lane's probability sums stay in registers over all its
// tokens.  A workgroup leaves its sums in the workspace; balance_finish adds them
// in order, 16 experts per workgroup, and the last workgroup to finish adds up the
// losses (its order of addition does not depend on which one that is).
#include "moe_common.h"

namespace moe {
namespace {

constexpr int kBalanceBlocks = 256, kBalanceThreads = 512, kBalanceWaves = kBalanceThreads / kWave;
constexpr int kFinishExperts = 16;   // experts of a workgroup of balance_finish

// What a workgroup leaves: E probability sums, E counts, its sum of lse^2 and its valid tokens.
__host__ __device__ constexpr int balance_stride(int E) { return 2 * E + 2; }

struct BalanceArgs {
  const float* logits;
  const int32_t* ids;
  const uint8_t* mask;
  float* lse;
  float* part;
  uint32_t* done;
  int T, E, k;
};

// Rows of logits start at any multiple of four bytes.
typedef float f32x4_u __attribute__((ext_vector_type(4), aligned(4)));

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

template <int G, int K, int U>
__global__ __launch_bounds__(kBalanceThreads) void balance_sums(BalanceArgs a) {
  constexpr int P = kWave / G;   // tokens of a wave at a time
  __shared__ int32_t s_cnt[G * K * 4];
  __shared__ float s_p[kBalanceWaves][G * K * 4], s_z[kBalanceWaves];
  __shared__ int32_t s_n[kBalanceWaves];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, g = lane % G, slot = lane / G;
  if (blockIdx.x == 0 && tid == 0) *a.done = 0;   // for balance_finish
  for (int e = tid; e < G * K * 4; e += kBalanceThreads) s_cnt[e] = 0;
  __syncthreads();
  float sum[K][4], z = 0.f;
  int n = 0;
#pragma unroll
  for (int j = 0; j < K; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q) sum[j][q] = 0.f;
  constexpr int R = kBalanceWaves * P;   // tokens of a workgroup at a time
  const int64_t step = (int64_t)gridDim.x * R * U;
  // every lane makes the same number of turns: the shuffles need all of a group
  for (int64_t t0 = (int64_t)blockIdx.x * R * U; t0 < a.T; t0 += step) {
    float v[U][K][4];
    bool valid[U];
    int id[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t t = t0 + u * R + wave * P + slot;
      valid[u] = t < a.T && (!a.mask || a.mask[t]);
      const float* row = a.logits + t * a.E;
#pragma unroll
      for (int j = 0; j < K; ++j) {
        const int e = 4 * (g + G * j);
        f32x4_u x = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        if (valid[u] && e + 4 <= a.E) {
          x = *(const f32x4_u*)(row + e);
        } else if (valid[u]) {
#pragma unroll
          for (int q = 0; q < 3; ++q)
            if (e + q < a.E) x[q] = row[e + q];
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) v[u][j][q] = x[q];
      }
      id[u] = valid[u] && g < a.k ? a.ids[t * a.k + g] : -1;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t t = t0 + u * R + wave * P + slot;
      float m = -INFINITY;
#pragma unroll
      for (int j = 0; j < K; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) m = fmaxf(m, v[u][j][q]);
      m = group_max<G>(m);
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < K; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          v[u][j][q] = 4 * (g + G * j) + q < a.E ? expf(v[u][j][q] - m) : 0.f;
          s += v[u][j][q];
        }
      s = group_sum<G>(s);
      const float lse = valid[u] ? m + logf(s) : 0.f;
      if (valid[u]) {
        const float inv = 1.0f / s;
#pragma unroll
        for (int j = 0; j < K; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) sum[j][q] = fmaf(v[u][j][q], inv, sum[j][q]);
        if (g == 0) {
          z = fmaf(lse, lse, z);
          ++n;
        }
        // whole numbers: the order of the atomics changes nothing
        if (id[u] >= 0 && id[u] < a.E) atomicAdd(&s_cnt[id[u]], 1);
        for (int j = g + G; j < a.k; j += G) {
          const int more = a.ids[t * a.k + j];
          if (more >= 0 && more < a.E) atomicAdd(&s_cnt[more], 1);
        }
      }
      if (t < a.T && g == 0) a.lse[t] = lse;
    }
  }
  // the groups of a wave, then the waves in order
#pragma unroll
  for (int d = G; d < kWave; d <<= 1) {
#pragma unroll
    for (int j = 0; j < K; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) sum[j][q] += __shfl_xor(sum[j][q], d, kWave);
    z += __shfl_xor(z, d, kWave);
    n += __shfl_xor(n, d, kWave);
  }
  if (slot == 0) {
#pragma unroll
    for (int j = 0; j < K; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) s_p[wave][4 * (g + G * j) + q] = sum[j][q];
    if (g == 0) {
      s_z[wave] = z;
      s_n[wave] = n;
    }
  }
  __syncthreads();
  float* out = a.part + (int64_t)blockIdx.x * balance_stride(a.E);
  for (int e = tid; e < a.E; e += kBalanceThreads) {
    float p = 0.f;
#pragma unroll
    for (int w = 0; w < kBalanceWaves; ++w) p += s_p[w][e];
    out[e] = p;
    out[a.E + e] = __int_as_float(s_cnt[e]);
  }
  if (tid == 0) {
    float zz = 0.f;
    int nn = 0;
    for (int w = 0; w < kBalanceWaves; ++w) {
      zz += s_z[w];
      nn += s_n[w];
    }
    out[2 * a.E] = zz;
    out[2 * a.E + 1] = __int_as_float(nn);
  }
}

// kFinishExperts experts per workgroup: 16 groups of threads add a run of the
// blocks' sums each, eight loads in flight, and the runs are added in order.  The
// last workgroup adds the experts' terms, the blocks' sums of lse^2 (fp64: the terms
// span many binades and there are few of them) and their tokens.
__global__ __launch_bounds__(256) void balance_finish(const float* __restrict__ part, int blocks, int E, int k,
                                                      float coef, float z_coef, double* terms, uint32_t* done,
                                                      float* __restrict__ losses, int32_t* __restrict__ counts,
                                                      int32_t* __restrict__ tokens, float* __restrict__ prob_sums) {
  __shared__ float s_p[16][kFinishExperts];
  __shared__ int32_t s_c[16][kFinishExperts];
  __shared__ double s_z[4];
  __shared__ int32_t s_n[4];
  __shared__ uint32_t s_last;
  const int tid = threadIdx.x, l = tid % kFinishExperts, g = tid / kFinishExperts, ld = balance_stride(E);
  const int e = blockIdx.x * kFinishExperts + l;
  static_assert(kMaxExperts <= kFinishExperts * kWave, "a lane of the last workgroup per workgroup");
  const int per = (blocks + 15) / 16, b0 = g * per, n = max(min(per, blocks - b0), 0);
  float p = 0.f;
  int c = 0;
  if (e < E) {
    const float* q = part + (int64_t)b0 * ld + e;
    for (int b = 0; b < n; b += 8) {
      float x[8];
      int y[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        x[u] = b + u < n ? q[(int64_t)(b + u) * ld] : 0.f;
        y[u] = b + u < n ? __float_as_int(q[(int64_t)(b + u) * ld + E]) : 0;
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        p += x[u];
        c += y[u];
      }
    }
  }
  s_p[g][l] = p;
  s_c[g][l] = c;
  // this workgroup's run of the blocks' sums of lse^2 and tokens
  {
    const int run = (blocks + gridDim.x - 1) / gridDim.x, at = blockIdx.x * run, len = min(run, blocks - at);
    double z = 0.0;
    int m = 0;
    for (int b = tid; b < len; b += 256) {
      z += (double)part[(int64_t)(at + b) * ld + 2 * E];
      m += __float_as_int(part[(int64_t)(at + b) * ld + 2 * E + 1]);
    }
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) {
      z += __shfl_xor(z, d, kWave);
      m += __shfl_xor(m, d, kWave);
    }
    if ((tid & 63) == 0) {
      s_z[tid >> 6] = z;
      s_n[tid >> 6] = m;
    }
  }
  __syncthreads();
  if (tid < kFinishExperts) {
    float v = 0.f;
    int w = 0;
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      v += s_p[q][l];
      w += s_c[q][l];
    }
    if (e < E) {
      prob_sums[e] = v;
      counts[e] = w;
    }
    double term = e < E ? (double)w * (double)v : 0.0;
#pragma unroll
    for (int d = kFinishExperts / 2; d >= 1; d >>= 1) term += __shfl_xor(term, d, kWave);
    if (tid == 0) {
      double* mine = terms + 3 * blockIdx.x;
      const double z = s_z[0] + s_z[1] + s_z[2] + s_z[3], m = (double)(s_n[0] + s_n[1] + s_n[2] + s_n[3]);
      __hip_atomic_store(mine, term, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      __hip_atomic_store(mine + 1, z, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      __hip_atomic_store(mine + 2, m, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      s_last = __hip_atomic_fetch_add(done, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == gridDim.x - 1;
    }
  }
  __syncthreads();
  if (!s_last || tid >= kWave) return;
  // at most 64 workgroups: a lane takes one, and the lanes are added in a fixed tree
  double v[3];
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    v[i] = (unsigned)tid < gridDim.x
               ? __hip_atomic_load(&terms[3 * tid + i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)
               : 0.0;
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) v[i] += __shfl_xor(v[i], d, kWave);
  }
  if (tid == 0) {
    const double n = v[2] > 0.0 ? v[2] : 1.0;
    losses[0] = (float)((double)coef * E / k * v[0] / (n * n));
    losses[1] = (float)((double)z_coef * v[1] / n);
    tokens[0] = (int32_t)v[2];
  }
}

// Lanes that share a token: the power of two that up to 16 experts each fill.
int balance_lanes(int E) {
  int g = 4;
  while (g < kWave && 16 * g < E) g *= 2;
  return g;
}

// One group of tokens per wave and turn where there are few tokens, two where that
// still fills every block.
int balance_unroll(int T, int E) {
  return (int64_t)T * balance_lanes(E) >= (int64_t)kBalanceBlocks * kBalanceThreads * 2 ? 2 : 1;
}
int balance_blocks(int T, int E) {
  const int64_t per = (int64_t)kBalanceWaves * (kWave / balance_lanes(E)) * balance_unroll(T, E);
  const int64_t need = ((int64_t)T + per - 1) / per;
  return (int)(need < kBalanceBlocks ? need : kBalanceBlocks);
}

struct BalanceWs {
  size_t terms, done, part, bytes;
};
BalanceWs balance_ws(int T, int E) {
  const size_t groups = (E + kFinishExperts - 1) / kFinishExperts;
  BalanceWs w;
  w.terms = 0;
  w.done = 3 * groups * sizeof(double);
  w.part = (w.done + sizeof(uint32_t) + 255) & ~(size_t)255;
  w.bytes = (w.part + (size_t)balance_blocks(T, E) * balance_stride(E) * sizeof(float) + 255) & ~(size_t)255;
  return w;
}

template <int G, int K>
void launch_sums(const BalanceArgs& a, int blocks, int unroll, hipStream_t s) {
  if (unroll == 2)
    hipLaunchKernelGGL((balance_sums<G, K, 2>), dim3(blocks), dim3(kBalanceThreads), 0, s, a);
  else
    hipLaunchKernelGGL((balance_sums<G, K, 1>), dim3(blocks), dim3(kBalanceThreads), 0, s, a);
}

}  // namespace
}  // namespace moe

namespace moe_launch {

size_t balance_loss_workspace_bytes(int T, int E) { return moe::balance_ws(T, E).bytes; }

hipError_t balance_loss(const float* logits, const int32_t* ids, const uint8_t* mask, int T, int E, int top_k,
                        float coef, float z_coef, float* losses, int32_t* counts, int32_t* tokens, float* prob_sums,
                        float* lse, void* ws, hipStream_t s) {
  const moe::BalanceWs w = moe::balance_ws(T, E);
  char* base = (char*)ws;
  float* part = (float*)(base + w.part);
  uint32_t* done = (uint32_t*)(base + w.done);
  const moe::BalanceArgs a{logits, ids, mask, lse, part, done, T, E, top_k};
  const int blocks = moe::balance_blocks(T, E), unroll = moe::balance_unroll(T, E);
  switch (moe::balance_lanes(E)) {
    case 4:
      if (E <= 16) moe::launch_sums<4, 1>(a, blocks, unroll, s);
      else if (E <= 32) moe::launch_sums<4, 2>(a, blocks, unroll, s);
      else moe::launch_sums<4, 4>(a, blocks, unroll, s);
      break;
    case 8: moe::launch_sums<8, 4>(a, blocks, unroll, s); break;
    case 16: moe::launch_sums<16, 4>(a, blocks, unroll, s); break;
    case 32: moe::launch_sums<32, 4>(a, blocks, unroll, s); break;
    default: moe::launch_sums<64, 4>(a, blocks, unroll, s);
  }
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  hipLaunchKernelGGL(moe::balance_finish, dim3((E + moe::kFinishExperts - 1) / moe::kFinishExperts), dim3(256), 0, s,
                     part, blocks, E, top_k, coef, z_coef, (double*)(base + w.terms), done, losses, counts, tokens,
                     prob_sums);
  return hipGetLastError();
}

}  // namespace moe_launch
