// Norm of all gradients together, and the gradients scaled to at most a given
// norm.
//
//   norm = sqrt(sum over all elements of all tensors of g^2)
//   coef = min(1, max_norm / (norm + 1e-6)),   out = coef * g
//
// Both are bound by memory: the norm reads every gradient once, the scaling
// reads and writes it once (in place with coef == 1 nothing moves).  Squares are
// taken and added in fp64: a float's square can overflow or vanish in fp32
// where the norm itself is representable, and the conversion and FMA cost less
// than the loads they follow.
//
// The tensors are cut into chunks; a launch carries the table of up to
// kGradBatch tensors in its arguments (nothing to upload, nothing that a
// captured graph would find changed), finds a chunk's tensor by bisection, and
// writes one partial sum per workgroup.  Partial sums are added in a fixed
// order by one workgroup, so the norm does not depend on timing.  The scaling
// walks the chunks backwards: those the norm read last may still be in the
// last-level cache.
#include "moe_common.h"

namespace moe {
namespace {

constexpr int kGradBatch = 112;
constexpr int kGradChunk = 16384;  // elements; a multiple of 8, so every chunk of a tensor has its alignment
constexpr int kGradBlocks = 2048;  // workgroups (and partial sums) per launch

struct GradBatchArgs {
  const void* in[kGradBatch];
  void* out[kGradBatch];
  int64_t numel[kGradBatch];
  int32_t chunk0[kGradBatch + 1];  // first chunk of each tensor
  uint8_t bf16[kGradBatch];
  int32_t n;
};
static_assert(sizeof(GradBatchArgs) + 64 <= 4096, "kernel arguments");

struct GradChunk {
  int i;
  int64_t at;
  int len;
};
__device__ __forceinline__ GradChunk grad_chunk(const GradBatchArgs& b, int c) {
  int lo = 0, hi = b.n - 1;  // largest i with chunk0[i] <= c: a tensor that is not empty
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (b.chunk0[mid] <= c) lo = mid; else hi = mid - 1;
  }
  GradChunk g;
  g.i = lo;
  g.at = (int64_t)(c - b.chunk0[lo]) * kGradChunk;
  g.len = (int)min((int64_t)kGradChunk, b.numel[lo] - g.at);
  return g;
}

// Elements before p reaches 16-byte alignment, at most len.
template <typename T>
__device__ __forceinline__ int head_of(const T* p, int len) {
  return min((int)(((16 - ((uintptr_t)p & 15)) & 15) / sizeof(T)), len);
}

__device__ __forceinline__ void sq(double& s, float v) { s = fma((double)v, (double)v, s); }

__device__ __forceinline__ double sum_squares(const float* __restrict__ p, int len, int tid) {
  const int head = head_of(p, len), nv = (len - head) / 4, done = head + 4 * nv;
  double s[4] = {0, 0, 0, 0};
  if (tid < head) sq(s[0], p[tid]);
  const f32x4* q = (const f32x4*)(p + head);
  for (int i = tid; i < nv; i += 256) {
    const f32x4 v = q[i];
#pragma unroll
    for (int j = 0; j < 4; ++j) sq(s[j], v[j]);
  }
  if (tid < len - done) sq(s[1], p[done + tid]);
  return (s[0] + s[1]) + (s[2] + s[3]);
}
__device__ __forceinline__ double sum_squares(const bf16_t* __restrict__ p, int len, int tid) {
  const int head = head_of(p, len), nv = (len - head) / 8, done = head + 8 * nv;
  double s[4] = {0, 0, 0, 0};
  if (tid < head) sq(s[0], bf16_to_f32(p[tid]));
  const u32x4* q = (const u32x4*)(p + head);
  for (int i = tid; i < nv; i += 256) {
    const u32x4 v = q[i];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      sq(s[j], bf16_to_f32(v[j] & 0xffffu));
      sq(s[j], __uint_as_float(v[j] & 0xffff0000u));
    }
  }
  if (tid < len - done) sq(s[1], bf16_to_f32(p[done + tid]));
  return (s[0] + s[1]) + (s[2] + s[3]);
}

// Sum over the workgroup in a fixed order (lanes, then waves), in thread 0.
__device__ __forceinline__ double block_sum(double v) {
  __shared__ double s_w[4];
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, kWave);
  if ((threadIdx.x & 63) == 0) s_w[threadIdx.x >> 6] = v;
  __syncthreads();
  return ((s_w[0] + s_w[1]) + s_w[2]) + s_w[3];
}

__global__ __launch_bounds__(256) void grad_sq(GradBatchArgs b, double* __restrict__ part) {
  const int chunks = b.chunk0[b.n];
  double s = 0.0;
  for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
    const GradChunk g = grad_chunk(b, c);
    s += b.bf16[g.i] ? sum_squares((const bf16_t*)b.in[g.i] + g.at, g.len, threadIdx.x)
                     : sum_squares((const float*)b.in[g.i] + g.at, g.len, threadIdx.x);
  }
  s = block_sum(s);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

__global__ __launch_bounds__(256) void grad_norm_sum(const double* __restrict__ part, int n, float* __restrict__ norm,
                                                     double* __restrict__ sum_sq) {
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += 256) s += part[i];
  s = block_sum(s);
  if (threadIdx.x == 0) {
    *norm = (float)sqrt(s);
    if (sum_sq) *sum_sq = s;
  }
}

__device__ __forceinline__ void scale(const float* __restrict__ p, float* o, int len, float c, int tid) {
  if ((((uintptr_t)p ^ (uintptr_t)o) & 15) == 0) {
    const int head = head_of(p, len), nv = (len - head) / 4, done = head + 4 * nv;
    if (tid < head) o[tid] = c * p[tid];
    for (int i = tid; i < nv; i += 256) ((f32x4*)(o + head))[i] = c * ((const f32x4*)(p + head))[i];
    if (tid < len - done) o[done + tid] = c * p[done + tid];
  } else {
    for (int i = tid; i < len; i += 256) o[i] = c * p[i];
  }
}
__device__ __forceinline__ bf16_t scale1(float c, uint32_t v) { return (bf16_t)f32_to_bf16_rne(c * bf16_to_f32(v)); }
__device__ __forceinline__ void scale(const bf16_t* __restrict__ p, bf16_t* o, int len, float c, int tid) {
  if ((((uintptr_t)p ^ (uintptr_t)o) & 15) == 0) {
    const int head = head_of(p, len), nv = (len - head) / 8, done = head + 8 * nv;
    if (tid < head) o[tid] = scale1(c, p[tid]);
    for (int i = tid; i < nv; i += 256) {
      const u32x4 v = ((const u32x4*)(p + head))[i];
      bf16x8 r;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        r[2 * j] = (__bf16)(c * bf16_to_f32(v[j] & 0xffffu));
        r[2 * j + 1] = (__bf16)(c * __uint_as_float(v[j] & 0xffff0000u));
      }
      ((bf16x8*)(o + head))[i] = r;
    }
    if (tid < len - done) o[done + tid] = scale1(c, p[done + tid]);
  } else {
    for (int i = tid; i < len; i += 256) o[i] = scale1(c, p[i]);
  }
}

// max_norm / (norm + 1e-6) where that is below 1 or not a number, else 1.
__device__ __forceinline__ float clip_coef(float norm, float max_norm) {
  const float c = (float)((double)max_norm / ((double)norm + 1e-6));
  return c >= 1.0f ? 1.0f : c;
}

__global__ __launch_bounds__(256) void grad_scale(GradBatchArgs b, const float* __restrict__ norm, float max_norm,
                                                  float* __restrict__ coef) {
  const float c = clip_coef(*norm, max_norm);
  if (coef && blockIdx.x == 0 && threadIdx.x == 0) *coef = c;
  const int chunks = b.chunk0[b.n];
  for (int k = blockIdx.x; k < chunks; k += gridDim.x) {
    const GradChunk g = grad_chunk(b, chunks - 1 - k);
    if (c == 1.0f && b.in[g.i] == b.out[g.i]) continue;
    if (b.bf16[g.i])
      scale((const bf16_t*)b.in[g.i] + g.at, (bf16_t*)b.out[g.i] + g.at, g.len, c, threadIdx.x);
    else
      scale((const float*)b.in[g.i] + g.at, (float*)b.out[g.i] + g.at, g.len, c, threadIdx.x);
  }
}

// Tensors [first, first + n) of a list; returns the number of chunks.
int fill_batch(GradBatchArgs& b, const void* const* in, void* const* out, const int64_t* numel, const int32_t* dts,
               int first, int n) {
  int64_t chunks = 0;
  for (int i = 0; i < n; ++i) {
    b.in[i] = in[first + i];
    b.out[i] = out ? out[first + i] : nullptr;
    b.numel[i] = numel[first + i];
    b.bf16[i] = dts[first + i] == 1;
    b.chunk0[i] = (int32_t)chunks;
    chunks += (numel[first + i] + kGradChunk - 1) / kGradChunk;
  }
  b.chunk0[n] = (int32_t)chunks;
  b.n = n;
  return (int)chunks;
}

}  // namespace
}  // namespace moe

namespace moe_launch {

size_t grad_norm_workspace_bytes(int n) {
  return (size_t)((n + moe::kGradBatch - 1) / moe::kGradBatch) * moe::kGradBlocks * sizeof(double);
}

hipError_t grad_norm(int n, const void* const* grads, const int64_t* numel, const int32_t* dts, float* norm,
                     double* sum_sq, void* workspace, hipStream_t s) {
  using namespace moe;
  double* part = (double*)workspace;
  int parts = 0;
  for (int first = 0; first < n; first += kGradBatch) {
    GradBatchArgs b;
    const int chunks = fill_batch(b, grads, nullptr, numel, dts, first, n - first < kGradBatch ? n - first : kGradBatch);
    if (chunks == 0) continue;
    const int grid = chunks < kGradBlocks ? chunks : kGradBlocks;
    hipLaunchKernelGGL(grad_sq, dim3(grid), dim3(256), 0, s, b, part + parts);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    parts += grid;
  }
  hipLaunchKernelGGL(grad_norm_sum, dim3(1), dim3(256), 0, s, part, parts, norm, sum_sq);
  return hipGetLastError();
}

hipError_t grad_clip(int n, const void* const* grads, void* const* outs, const int64_t* numel, const int32_t* dts,
                     const float* norm, float max_norm, float* coef, hipStream_t s) {
  using namespace moe;
  const int batches = (n + kGradBatch - 1) / kGradBatch;
  for (int q = batches - 1; q >= 0; --q) {
    const int first = q * kGradBatch;
    GradBatchArgs b;
    const int chunks = fill_batch(b, grads, outs, numel, dts, first, n - first < kGradBatch ? n - first : kGradBatch);
    // the first batch's launch also stores the coefficient
    if (chunks == 0 && !(q == 0 && coef)) continue;
    const int grid = chunks < 1 ? 1 : (chunks < kGradBlocks ? chunks : kGradBlocks);
    hipLaunchKernelGGL(grad_scale, dim3(grid), dim3(256), 0, s, b, norm, max_norm, q == 0 ? coef : nullptr);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

}  // namespace moe_launch
