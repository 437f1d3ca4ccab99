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
// The tensors are cut into chunks of kGradChunk elements; a launch carries the
// table of its tensors in its arguments (nothing to upload, nothing that a
// captured graph would find changed) and writes one partial sum per workgroup.
// A chunk's tensor is found by comparing the chunk with every tensor's first one,
// a table entry per lane.  A thread loads all its 16-byte pieces of a chunk
// before it uses them: with a loop of one load at a time, a chunk took eight
// memory latencies (300 tensors of 13 M elements in all: 57 us, now 31).
// Partial sums are added in a fixed order by one workgroup, so the norm does not
// depend on timing.  The scaling is a copy and bound as one: a workgroup per chunk
// (0.38 G bf16 elements into others: 242 us, 6.3 TB/s; 2048 workgroups that loop
// 334), its loads and stores past the caches (non-temporal; cached loads: 5 %
// slower).  Norm and scaling of a layer's 0.571 G elements: 533 us, of them the
// norm 186 (6.1 TB/s) and the scaling 342 (6.7 TB/s); in place 557, and 195 where
// the factor is 1.
#include "moe_common.h"

namespace moe {
namespace {

constexpr int kGradChunk = 8192;   // elements; a multiple of 8, so every chunk of a tensor has its alignment
constexpr int kGradBlocks = 2048;  // workgroups (and partial sums) per launch of the norm
// Workgroups per launch of the scaling.  In place most of them find a factor of
// 1 and end, which costs 46000 of them 13 us, 8192 of them 5.
constexpr int kScaleBlocks = 1 << 20, kScaleBlocksInPlace = 8192;

// Up to N tensors in a kernel's arguments: 14 bytes each, 22 with an output of
// their own.  A tensor's length is its chunks and the elements of its last one.
template <int N, bool OUT>
struct GradTable {
  static constexpr int kMost = N;
  static constexpr bool kOut = OUT;
  const void* in[N];
  void* out[OUT ? N : 1];
  int32_t chunk0[N];      // first chunk of each tensor; INT32_MAX past the last tensor
  uint16_t tail[N];       // elements of the last chunk (0: the tensor is empty), and kBf16
  int32_t chunks;
  int32_t n;
};
constexpr uint16_t kBf16 = 0x8000;
typedef GradTable<280, false> GradTableIn;   // the norm, and scaling in place
typedef GradTable<180, true> GradTableInOut;
static_assert(sizeof(GradTableIn) <= 4000 && sizeof(GradTableInOut) <= 4000, "kernel arguments: at most 4 KiB");

// First chunks of the table, 64 tensors per register.
template <class B>
struct GradLookup {
  static constexpr int kRegs = (B::kMost + 63) / 64;
  int32_t first[kRegs];
};
template <class B>
__device__ __forceinline__ void grad_lookup_init(const B& b, GradLookup<B>& l) {
#pragma unroll
  for (int q = 0; q < GradLookup<B>::kRegs; ++q) {
    const int i = 64 * q + lane_id();
    l.first[q] = i < B::kMost ? b.chunk0[i] : 0x7fffffff;
  }
}

struct GradChunk {
  int i;        // tensor
  int64_t at;   // first element
  int len;
  bool bf16;
};
template <class B>
__device__ __forceinline__ GradChunk grad_chunk(const B& b, const GradLookup<B>& l, int c) {
  // tensors that start at or before c; an empty tensor shares its successor's
  // first chunk, so the last of them is one that holds c
  int n = 0;
#pragma unroll
  for (int q = 0; q < GradLookup<B>::kRegs; ++q) n += __popcll(__ballot(l.first[q] <= c));
  GradChunk g;
  g.i = __builtin_amdgcn_readfirstlane(n - 1);
  const int first = b.chunk0[g.i];
  const int next = g.i + 1 < b.n ? b.chunk0[g.i + 1] : b.chunks;
  const int tail = b.tail[g.i];
  g.bf16 = (tail & kBf16) != 0;
  g.at = (int64_t)(c - first) * kGradChunk;
  g.len = c + 1 == next ? (tail & (kBf16 - 1)) : kGradChunk;
  return g;
}

// Elements before p reaches 16-byte alignment, at most len.
template <typename T>
__device__ __forceinline__ int head_of(const T* p, int len) {
  return min((int)(((16 - ((uintptr_t)p & 15)) & 15) / sizeof(T)), len);
}

__device__ __forceinline__ void sq(double& s, float v) { s = fma((double)v, (double)v, s); }

__device__ __forceinline__ void sq_piece(const u32x4& v, double (&s)[4], float) {
#pragma unroll
  for (int j = 0; j < 4; ++j) sq(s[j], __uint_as_float(v[j]));
}
__device__ __forceinline__ void sq_piece(const u32x4& v, double (&s)[4], bf16_t) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    sq(s[j], bf16_to_f32(v[j] & 0xffffu));
    sq(s[j], __uint_as_float(v[j] & 0xffff0000u));
  }
}

// The calling thread's part of a chunk's sum of squares: a 16-byte aligned
// middle, and up to one piece's elements before and after it.
template <typename T>
__device__ __forceinline__ double sum_squares(const T* __restrict__ p, int len, int tid) {
  constexpr int E = 16 / sizeof(T), P = kGradChunk / E / 256;   // elements per piece, pieces per thread
  const int head = head_of(p, len), nv = (len - head) / E, done = head + E * nv;
  const u32x4* q = (const u32x4*)(p + head);
  u32x4 v[P];
#pragma unroll
  for (int i = 0; i < P; ++i) v[i] = tid + 256 * i < nv ? q[tid + 256 * i] : u32x4{0u, 0u, 0u, 0u};
  const float a = tid < head ? load_as_f32(p, tid) : 0.f;
  const float b = tid < len - done ? load_as_f32(p, done + tid) : 0.f;
  double s[4] = {0, 0, 0, 0};
  sq(s[0], a);
  sq(s[1], b);
#pragma unroll
  for (int i = 0; i < P; ++i) sq_piece(v[i], s, T{});
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

__global__ __launch_bounds__(256) void grad_sq(GradTableIn b, double* __restrict__ part) {
  GradLookup<GradTableIn> l;
  grad_lookup_init(b, l);
  double s = 0.0;
  for (int c = blockIdx.x; c < b.chunks; c += gridDim.x) {
    const GradChunk g = grad_chunk(b, l, c);
    s += g.bf16 ? sum_squares((const bf16_t*)b.in[g.i] + g.at, g.len, threadIdx.x)
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

__device__ __forceinline__ u32x4 scale_piece(const u32x4& v, float c, float) {
  u32x4 r;
#pragma unroll
  for (int j = 0; j < 4; ++j) r[j] = __float_as_uint(c * __uint_as_float(v[j]));
  return r;
}
__device__ __forceinline__ u32x4 scale_piece(const u32x4& v, float c, bf16_t) {
  bf16x8 r;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    r[2 * j] = (__bf16)(c * bf16_to_f32(v[j] & 0xffffu));
    r[2 * j + 1] = (__bf16)(c * __uint_as_float(v[j] & 0xffff0000u));
  }
  return __builtin_bit_cast(u32x4, r);
}

// p and o may be the same tensor.
template <typename T>
__device__ __forceinline__ void scale(const T* p, T* o, int len, float c, int tid) {
  if ((((uintptr_t)p ^ (uintptr_t)o) & 15) == 0) {
    constexpr int E = 16 / sizeof(T), P = kGradChunk / E / 256;
    const int head = head_of(p, len), nv = (len - head) / E, done = head + E * nv;
    const u32x4* q = (const u32x4*)(p + head);
    u32x4 v[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
      v[i] = u32x4{0u, 0u, 0u, 0u};
      if (tid + 256 * i < nv) v[i] = __builtin_nontemporal_load(q + tid + 256 * i);
    }
    const float a = tid < head ? load_as_f32(p, tid) : 0.f;
    const float b = tid < len - done ? load_as_f32(p, done + tid) : 0.f;
    u32x4* r = (u32x4*)(o + head);
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (tid + 256 * i < nv) __builtin_nontemporal_store(scale_piece(v[i], c, T{}), r + tid + 256 * i);
    if (tid < head) store_from_f32(o, tid, c * a);
    if (tid < len - done) store_from_f32(o, done + tid, c * b);
  } else {   // alignments differ: element by element, sixteen in flight per thread
    for (int i0 = tid; i0 < len; i0 += 16 * 256) {
      float v[16];
#pragma unroll
      for (int u = 0; u < 16; ++u) v[u] = i0 + 256 * u < len ? load_as_f32(p, i0 + 256 * u) : 0.f;
#pragma unroll
      for (int u = 0; u < 16; ++u)
        if (i0 + 256 * u < len) store_from_f32(o, i0 + 256 * u, c * v[u]);
    }
  }
}

// max_norm / (norm + 1e-6) where that is below 1 or not a number, else 1.
__device__ __forceinline__ float clip_coef(float norm, float max_norm) {
  const float c = (float)((double)max_norm / ((double)norm + 1e-6));
  return c >= 1.0f ? 1.0f : c;
}

template <class B>
__global__ __launch_bounds__(256) void grad_scale(B b, const float* __restrict__ norm, float max_norm,
                                                  float* __restrict__ coef) {
  const float c = clip_coef(*norm, max_norm);
  if (coef && blockIdx.x == 0 && threadIdx.x == 0) *coef = c;
  if (!B::kOut && c == 1.0f) return;   // in place: nothing to move
  GradLookup<B> l;
  grad_lookup_init(b, l);
  for (int64_t k = blockIdx.x; k < b.chunks; k += gridDim.x) {
    const GradChunk g = grad_chunk(b, l, (int)k);
    const void* in = b.in[g.i];
    void* out = B::kOut ? b.out[g.i] : const_cast<void*>(in);
    if (c == 1.0f && in == out) continue;
    if (g.bf16)
      scale((const bf16_t*)in + g.at, (bf16_t*)out + g.at, g.len, c, threadIdx.x);
    else
      scale((const float*)in + g.at, (float*)out + g.at, g.len, c, threadIdx.x);
  }
}

// Fills a table from tensor `first` on; returns the tensor after its last.  Fewer
// than 2^43 elements in all are at most 2^30 + kMost chunks of a table.
template <class B>
int fill_table(B& b, const void* const* in, void* const* out, const int64_t* numel, const int32_t* dts, int first,
               int n) {
  int64_t chunks = 0;
  int i = 0;
  for (; i < B::kMost && first + i < n; ++i) {
    const int64_t len = numel[first + i], c = (len + kGradChunk - 1) / kGradChunk;
    b.in[i] = in[first + i];
    if (B::kOut) b.out[i] = out[first + i];
    b.chunk0[i] = (int32_t)chunks;
    b.tail[i] = (uint16_t)((len - (c > 0 ? c - 1 : 0) * kGradChunk) | (dts[first + i] == 1 ? kBf16 : 0));
    chunks += c;
  }
  b.n = i;
  b.chunks = (int32_t)chunks;
  for (; i < B::kMost; ++i) {
    b.in[i] = nullptr;
    if (B::kOut) b.out[i] = nullptr;
    b.chunk0[i] = 0x7fffffff;
    b.tail[i] = 0;
  }
  return first + b.n;
}

template <class B>
hipError_t scale_list(int n, const void* const* grads, void* const* outs, const int64_t* numel, const int32_t* dts,
                      const float* norm, float max_norm, float* coef, hipStream_t s) {
  B b;
  for (int first = 0; first < n;) {
    const bool head = first == 0;   // the first launch also stores the coefficient
    first = fill_table(b, grads, outs, numel, dts, first, n);
    if (b.chunks == 0 && !(head && coef)) continue;
    const int most = B::kOut ? kScaleBlocks : kScaleBlocksInPlace;
    const int grid = b.chunks < 1 ? 1 : (b.chunks < most ? b.chunks : most);
    hipLaunchKernelGGL(grad_scale<B>, dim3(grid), dim3(256), 0, s, b, norm, max_norm, head ? coef : nullptr);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

}  // namespace
}  // namespace moe

namespace moe_launch {

// One partial sum per workgroup, at most kGradBlocks per launch.
size_t grad_norm_workspace_bytes(int n) {
  const int64_t tables = ((int64_t)n + moe::GradTableIn::kMost - 1) / moe::GradTableIn::kMost;
  return (size_t)tables * moe::kGradBlocks * sizeof(double);
}

hipError_t grad_norm(int n, const void* const* grads, const int64_t* numel, const int32_t* dts, float* norm,
                     double* sum_sq, void* workspace, hipStream_t s) {
  using namespace moe;
  double* part = (double*)workspace;
  int parts = 0;
  GradTableIn b;
  for (int first = 0; first < n;) {
    first = fill_table(b, grads, nullptr, numel, dts, first, n);
    if (b.chunks == 0) continue;
    const int grid = b.chunks < kGradBlocks ? b.chunks : kGradBlocks;
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
  bool in_place = true;
  for (int i = 0; i < n && in_place; ++i) in_place = numel[i] == 0 || grads[i] == outs[i];
  if (in_place)
    return moe::scale_list<moe::GradTableIn>(n, grads, nullptr, numel, dts, norm, max_norm, coef, s);
  return moe::scale_list<moe::GradTableInOut>(n, grads, outs, numel, dts, norm, max_norm, coef, s);
}

}  // namespace moe_launch
