// Dense bf16 products on MFMAs: one output tile per workgroup, shared by the
// shared expert's training calls and the router's weight gradient.
//
//   C[m, n] = sum_k A(m, k) B(k, n)
//
// where an operand is stored either with k contiguous ("row": A [M, K],
// B [N, K]) or with its other index contiguous ("col": A [K, M], B [K, N]).
//
//  * One workgroup per output tile (BM x BN) and reduction range; slices of 64
//    along k travel HBM -> LDS with buffer_load ... lds into a ring of five
//    slots of one operand slice each (two whole slices and the next A: what 160
//    KiB hold of a 256 x 256 tile), so half of a slice's loads are issued two
//    slices ahead and half one slice ahead.  Rows, columns and k past an
//    operand's end are out of the buffer descriptor's range (or given an
//    out-of-range offset), which the hardware turns into zeros in LDS, so no
//    size has a special path.
//  * "row" operands sit in LDS as 128-byte rows whose 16-byte chunks are XORed
//    with (row >> 1) & 7: an MFMA fragment is one ds_read_b128.  "col" operands
//    sit as k rows with chunks XORed by the k row; a fragment is two
//    ds_read_b64_tr_b16 transpose reads.
//  * v_mfma_f32_16x16x32_bf16: on random data the chip is bound by power, and a
//    register-only loop of it sustains 1985 TFLOP/s against 1750 of 32x32x16,
//    which moves four times the accumulators per instruction.
//  * Each wave alternates between two fragment sets: the next 32-deep
//    substep's LDS reads run under the current substep's MFMAs, across slice
//    boundaries too.
//  * The product is taken swapped (B's fragment as the MFMA's first operand),
//    so a lane holds four consecutive columns of one row; the tile goes through
//    the idle ring, a wave's 32 x 64 piece at a time, and the epilogue works on
//    eight consecutive columns per lane with 16-byte loads and stores.
#pragma once

#include "moe_common.h"

#include <type_traits>

namespace moe {
namespace {

constexpr int kDBK = 64;          // reduction slice
constexpr int kSlots = 5;         // ring slots, one operand slice each
constexpr int kDXcds = 8;
constexpr int kOob = 0x7ffffff0;  // byte offset past every descriptor's range

// Epilogues.  v holds eight consecutive output columns of one row (for the
// paired one: g and u columns of the same outputs).
// kEStoreCols: rows of `cols` <= N elements are stored.
enum DenseEpi { kESwigluSave = 0, kEGateAdd = 1, kESwigluBwd = 2, kEInputGrad = 3, kEStore = 4, kEStoreCols = 5 };

struct DenseEpiArgs {
  void* out;
  void* out2;
  const void* aux;
  const float* row;   // per-row factor, or null
  const void* col;    // per-column factor (kEInputGrad), or null
  int accumulate;
  int cols;
};

struct DenseProblem {
  const void* a;
  const void* b;
  int M, N, K;          // N: output columns (paired: B holds 2N, gate columns first)
  int lda, ldb;         // elements between stored rows
  int splits, k_split;  // reduction ranges of k_split (a multiple of kDBK)
  int m_tiles, n_tiles;
  float* partial;       // [splits, M, N or 2N], or null: the epilogue runs in the kernel (one split)
  DenseEpiArgs e;
};

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const f32x4 a = *(const f32x4*)p, b = *(const f32x4*)(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = a[i];
    v[4 + i] = b[i];
  }
}
__device__ __forceinline__ void load8(const bf16_t* p, float (&v)[8]) {
  const u32x4 a = *(const u32x4*)p;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_to_f32(a[i] & 0xffffu);
    v[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  *(f32x4*)p = f32x4{v[0], v[1], v[2], v[3]};
  *(f32x4*)(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
}
// Round to nearest even, the storage rounding of every bf16 tensor of the layer.
__device__ __forceinline__ void store8(bf16_t* p, const float (&v)[8]) {
  bf16x8 o;
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = (__bf16)v[i];
  *(bf16x8*)p = o;
}

// The pre-activations are not read before the backward pass: their stores do not
// stay in the caches, where what the next product reads then has more room (8192
// tokens, H = 2048, I_s = 2816: 168 -> 165 us, weights stored transposed 167 -> 163).
__device__ __forceinline__ void store8nt(float* p, const float (&v)[8]) {
  __builtin_nontemporal_store(f32x4{v[0], v[1], v[2], v[3]}, (f32x4*)p);
  __builtin_nontemporal_store(f32x4{v[4], v[5], v[6], v[7]}, (f32x4*)p + 1);
}
__device__ __forceinline__ void store8nt(bf16_t* p, const float (&v)[8]) {
  bf16x8 o;
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = (__bf16)v[i];
  __builtin_nontemporal_store(__builtin_bit_cast(u32x4, o), (u32x4*)p);
}

// Sigmoid of an epilogue.  bf16 results (half a step is 2^-9 of the value or
// more) take v_exp_f32 and v_rcp_f32, each within about 1 ulp of fp32: the
// correctly rounded division and expf cost five times the instructions, and with
// them the epilogue of a 256 x 256 tile was as long as a quarter of its products.
template <typename T>
__device__ __forceinline__ float epi_sigmoid(float z) {
  if constexpr (sizeof(T) == 2)
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * z));
  else
    return sigmoidf_(z);
}

// What the epilogue of outputs [n, n + 8) of row m reads besides the sums
// (16-byte pieces, not converted): the pre-activation of kESwigluBwd, or what
// the output is added to.  Loaded apart from its use, so that the loads of
// several rows are in flight together.
template <typename T, int EPI>
struct EpiIn {
  static constexpr int kAdd = EPI == kEGateAdd || EPI == kEInputGrad ? 2 : 0;
  static constexpr int N = EPI == kESwigluBwd ? (sizeof(T) == 2 ? 2 : 4) : kAdd;
  u32x4 v[N ? N : 1];
};

template <typename T, int EPI>
__device__ __forceinline__ void epi_load(const DenseEpiArgs& e, int64_t m, int n, int N, EpiIn<T, EPI>& in) {
  if constexpr (EPI == kESwigluBwd) {
    const T* h = (const T*)e.aux + m * 2 * N + n;
    constexpr int half = EpiIn<T, EPI>::N / 2;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      in.v[i] = ((const u32x4*)h)[i];
      in.v[half + i] = ((const u32x4*)(h + N))[i];
    }
  } else if constexpr (EPI == kEGateAdd || EPI == kEInputGrad) {
    if (e.accumulate) {
      const u32x4* o = (const u32x4*)((const float*)e.out + m * N + n);
      in.v[0] = o[0];
      in.v[1] = o[1];
    }
  }
}

__device__ __forceinline__ void unpack8(const u32x4* v, float (&o)[8], float) {
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = __uint_as_float(v[i / 4][i % 4]);
}
__device__ __forceinline__ void unpack8(const u32x4* v, float (&o)[8], bf16_t) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o[2 * i] = bf16_to_f32(v[0][i] & 0xffffu);
    o[2 * i + 1] = __uint_as_float(v[0][i] & 0xffff0000u);
  }
}

// Outputs [n, n + 8) of row m from their accumulated sums v (paired: g = v, u = v2).
template <typename T, int EPI>
__device__ __forceinline__ void epi8(const DenseEpiArgs& e, int64_t m, int n, int N, const float (&v)[8],
                                     const float (&v2)[8], const EpiIn<T, EPI>& in) {
  float o[8], p[8];
  if constexpr (EPI == kESwigluSave) {
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = v[i] * epi_sigmoid<T>(v[i]) * v2[i];
    store8((T*)e.out + m * N + n, o);
    T* h = (T*)e.out2 + m * 2 * N + n;
    store8nt(h, v);
    store8nt(h + N, v2);
  } else if constexpr (EPI == kEGateAdd) {
    if (e.out2) store8((float*)e.out2 + m * N + n, v);
    const float sc = e.row ? e.row[m] : 1.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = sc * v[i];
    if (e.accumulate) {
      unpack8(in.v, p, 0.f);
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] += p[i];
    }
    store8((float*)e.out + m * N + n, o);
  } else if constexpr (EPI == kESwigluBwd) {
    // dg = da u s (1 + g (1 - s)), du = da g s, s = sigmoid(g).  The sigmoid's factor goes
    // to u and g before da does: s = 0 would turn an overflow of da u or da g into a NaN
    // where the value is 0, and any other small s into an infinity.
    float g[8], u[8];
    unpack8(in.v, g, T{});
    unpack8(in.v + EpiIn<T, EPI>::N / 2, u, T{});
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float s = epi_sigmoid<T>(g[i]);
      o[i] = v[i] * (u[i] * s * (1.0f + g[i] * (1.0f - s)));
      p[i] = v[i] * (g[i] * s);
    }
    T* d = (T*)e.out + m * 2 * N + n;
    store8(d, o);
    store8(d + N, p);
  } else if constexpr (EPI == kEInputGrad) {
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = v[i];
    if (e.row) {
      const float z = e.row[m];
      load8((const T*)e.col + n, p);
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = fmaf(z, p[i], o[i]);
    }
    if (e.accumulate) {
      unpack8(in.v, p, 0.f);
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = p[i] + o[i];
    }
    store8((float*)e.out + m * N + n, o);
  } else if constexpr (EPI == kEStore) {
    store8((T*)e.out + m * N + n, v);
  } else if constexpr (EPI == kEStoreCols) {
    T* d = (T*)e.out + m * e.cols + n;
    if (e.cols == N) {   // N is a multiple of 8: aligned
      store8(d, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (n + i < e.cols) store_from_f32(d, i, v[i]);
    }
  }
}

// Load and use in one step.
template <typename T, int EPI>
__device__ __forceinline__ void epi8_now(const DenseEpiArgs& e, int64_t m, int n, int N, const float (&v)[8],
                                         const float (&v2)[8]) {
  EpiIn<T, EPI> in;
  epi_load<T, EPI>(e, m, n, N, in);
  epi8<T, EPI>(e, m, n, N, v, v2, in);
}

template <int EPI>
constexpr bool dense_paired() { return EPI == kESwigluSave; }

// ------------------------------------------------------------------------------------------
// bf16
// ------------------------------------------------------------------------------------------
// KW > 1: KW groups of WM x WN waves take every KW-th slice, each with a ring of
// its own; their sums are added in group order before the epilogue.
template <int BM_, int BN_, int WM_, int WN_, int KW_ = 1>
struct DenseCfg {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, KW = KW_;
  static constexpr int kPos = WM * WN, kWaves = kPos * KW, NT = kWaves * kWave;
  static constexpr int kMB = BM / WM / 16, kNB = BN / WN / 16;   // 16 x 16 MFMA blocks of a wave
  static constexpr int kABytes = BM * kDBK * 2, kBBytes = BN * kDBK * 2;   // one operand slice
  static constexpr int kALoads = kABytes / 1024 / kPos, kBLoads = kBBytes / 1024 / kPos;
  static constexpr int kSlot = kABytes > kBBytes ? kABytes : kBBytes;
  static constexpr int kRing = kSlots * kSlot, kLds = KW * kRing;
  static constexpr int kFit = (160 * 1024) / kLds;
  static constexpr int kWgs0 = kFit < 1 ? 1 : kFit;
  // waves per SIMD that the registers allow: 128-accumulator waves fit two
  static constexpr int kWgsPerCu = kWgs0 * kWaves > 8 ? (8 / kWaves < 1 ? 1 : 8 / kWaves) : kWgs0;
  static_assert(kABytes % (1024 * kPos) == 0 && kBBytes % (1024 * kPos) == 0, "slices split into 1 KiB loads");
  static_assert(kMB % 2 == 0 && kNB % 4 == 0, "a wave holds pairs of 16-row blocks and 64-column pieces");
  static_assert(kPos * 8192 <= kRing, "epilogue: 8 KiB of a ring per wave");
  static_assert((KW - 1) * BM * BN * 4 <= kRing * (KW - 1), "the groups' sums fit their rings");
};

// Column (in the staged tile) of 16-column block nb of wave column wn; four
// blocks make a 64-column piece.  Paired: a piece is 32 gate columns and the
// matching 32 up columns.
template <class C, bool PAIRED>
__device__ __forceinline__ int dense_col(int nb, int wn) {
  return PAIRED ? ((nb % 4 / 2) * (C::BN / 2) + wn * (C::BN / 2 / C::WN) + 32 * (nb / 4) + 16 * (nb % 2))
                : (wn * (C::BN / C::WN) + 16 * nb);
}

// Swizzle of 16-byte chunks of a k-major ("col") LDS row of CHUNKS chunks.  A
// 32-lane phase of a transpose read touches 4 consecutive k rows of two octets
// of k, 32 bytes of each: the 4 rows go to different 64-byte quarters of the
// 256-byte bank window (128-byte rows: two rows share a window, so only the
// second row bit needs moving), the octets to different halves of a quarter.
template <int CHUNKS>
__device__ __forceinline__ int col_swz(int k) {
  return (CHUNKS >= 16 ? 4 * (k & 3) : 4 * ((k >> 1) & 1)) ^ (2 * ((k >> 3) & 1));
}

// Byte offsets (from the slice's base) of a wave's 1 KiB loads of one operand
// tile of W rows/columns.
template <int W, bool COL, int LOADS>
__device__ __forceinline__ void dense_offsets(int (&off)[LOADS], int ld, int valid, bool paired, int half_valid,
                                              int up_off, int wave, int lane) {
#pragma unroll
  for (int i = 0; i < LOADS; ++i) {
    const int piece = wave * LOADS + i;
    if constexpr (COL) {
      constexpr int CH = W / 8;                      // chunks per k row
      const int kr = (piece * 64 + lane) / CH;
      const int c = 8 * (((piece * 64 + lane) % CH) ^ col_swz<CH>(kr));
      if (paired) {
        const int half = W / 2, cc = c % half;
        off[i] = cc < half_valid ? 2 * (kr * ld + cc + (c < half ? 0 : up_off)) : kOob;
      } else {
        off[i] = c < valid ? 2 * (kr * ld + c) : kOob;
      }
    } else {
      const int r = piece * 8 + lane / 8;
      const int chunk = (lane % 8) ^ ((r >> 1) & 7);
      if (paired) {
        const int half = W / 2, rr = r % half;
        off[i] = rr < half_valid ? 2 * ((rr + (r < half ? 0 : up_off)) * ld + 8 * chunk) : kOob;
      } else {
        off[i] = r < valid ? 2 * (r * ld + 8 * chunk) : kOob;
      }
    }
  }
}

struct DenseSpan {
  const bf16_t* base;
  int bytes;
  int kv;   // valid k of the slice
};

// One 1 KiB direct load: piece `piece` of the slice into the slot at st.
template <bool COL>
__device__ __forceinline__ void dense_load(const DenseSpan& d, int off, int piece, int lane, unsigned char* st) {
  if constexpr (!COL) {  // chunks past the valid k hold the next row's elements
    const int r = piece * 8 + lane / 8;
    off = 8 * ((lane % 8) ^ ((r >> 1) & 7)) < d.kv ? off : kOob;
  }
  __builtin_amdgcn_raw_ptr_buffer_load_lds(__builtin_amdgcn_make_buffer_rsrc((void*)d.base, 0, d.bytes, 0x00027000),
                                           MOE_LDS(void, st + piece * 1024), 16, off, 0, 0, 0);
}

// Fragment of 16 rows/columns at `blk`, k [32 ks, 32 ks + 32), of an LDS tile:
// lane L gets row/column blk + L % 16, k = 8 (L / 16) .. + 7.
template <int W, bool COL>
__device__ __forceinline__ u32x4 dense_frag(const unsigned char* __restrict__ tile, int blk, int ks, int lane) {
  const int grp = lane >> 4, s16 = lane & 15;
  if constexpr (COL) {
    constexpr int CH = W / 8;
    const int row = 32 * ks + 8 * grp + (s16 >> 2);
    const int chunk = (blk / 8 + ((s16 & 3) >> 1)) ^ col_swz<CH>(8 * grp + (s16 >> 2));
    const unsigned char* p = tile + row * (16 * CH) + chunk * 16 + (s16 & 1) * 8;
    const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(MOE_LDS(i16x4, p));
    const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(MOE_LDS(i16x4, p + 4 * 16 * CH));
    return pack_tr_pair(lo, hi);
  } else {
    const int r = blk + s16;
    const int chunk = (4 * ks + grp) ^ ((r >> 1) & 7);
    return *(const u32x4*)(tile + r * 128 + chunk * 16);
  }
}

__device__ __forceinline__ f32x4 dmfma(const u32x4& a, const u32x4& b, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                 0);
}

// A wave's fragments of one 32-deep substep.
template <class C>
struct DenseFrags {
  u32x4 a[C::kMB], b[C::kNB];
};

// Fragment i of a substep (B's first: every MFMA of a row block needs them).
template <class C, bool ACOL, bool BCOL, bool PAIRED>
__device__ __forceinline__ void dense_read1(const unsigned char* __restrict__ ta, const unsigned char* __restrict__ tb,
                                            int ks, int i, int wm, int wn, int lane, DenseFrags<C>& f) {
  if (i < C::kNB)
    f.b[i] = dense_frag<C::BN, BCOL>(tb, dense_col<C, PAIRED>(i, wn), ks, lane);
  else
    f.a[i - C::kNB] = dense_frag<C::BM, ACOL>(ta, wm * (C::BM / C::WM) + 16 * (i - C::kNB), ks, lane);
}
template <class C, bool ACOL, bool BCOL, bool PAIRED>
__device__ __forceinline__ void dense_read(const unsigned char* __restrict__ ta, const unsigned char* __restrict__ tb,
                                           int ks, int wm, int wn, int lane, DenseFrags<C>& f) {
#pragma unroll
  for (int i = 0; i < C::kNB + C::kMB; ++i) dense_read1<C, ACOL, BCOL, PAIRED>(ta, tb, ks, i, wm, wn, lane, f);
}

// The MFMAs of one substep in groups of two, with the next substep's fragment
// reads (read(i)) under the first three quarters of them and L direct loads
// (load(i)) spread over all; the scheduling barriers keep the compiler to this
// order.
template <class C, int L, class Read, class Load>
__device__ __forceinline__ void dense_substep(const DenseFrags<C>& f, f32x4 (&acc)[C::kMB][C::kNB], const Read& read,
                                              const Load& load) {
  constexpr int M = C::kMB * C::kNB, G = M / 2, R = C::kMB + C::kNB, GR = G * 3 / 4;
#pragma unroll
  for (int g = 0; g < G; ++g) {
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (i * GR / R == g) read(i);
#pragma unroll
    for (int i = 0; i < L; ++i)
      if ((2 * i + 1) * G / (2 * L) == g) load(i);
#pragma unroll
    for (int q = 2 * g; q < 2 * g + 2; ++q)
      acc[q / C::kNB][q % C::kNB] = dmfma(f.b[q % C::kNB], f.a[q / C::kNB], acc[q / C::kNB][q % C::kNB]);
    __builtin_amdgcn_sched_barrier(0);
  }
}

__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Tile and reduction range of unit `u` of a problem.  Units are dealt to the
// XCDs in contiguous runs (workgroups go to the 8 XCDs round-robin), and a run
// walks bands of up to 8 row tiles, so that the workgroups of one XCD share
// operand tiles in its L2.  The splits of a tile are runs apart.
struct DenseUnit {
  int mt, nt, split;
};
__device__ __forceinline__ DenseUnit dense_unit(const DenseProblem& p, int u) {
  const int tiles = p.m_tiles * p.n_tiles;
  const int n = tiles * p.splits;
  const int q = n / kDXcds, r = n % kDXcds, x = u % kDXcds;
  const int id = x * q + min(x, r) + u / kDXcds;
  DenseUnit t;
  t.split = id / tiles;
  const int tile = id % tiles;
  const int band = tile / (8 * p.n_tiles), in = tile % (8 * p.n_tiles);
  const int rows = min(8, p.m_tiles - 8 * band);
  t.mt = 8 * band + in % rows;
  t.nt = in / rows;
  return t;
}

template <class C, bool ACOL, bool BCOL, int EPI>
__device__ __forceinline__ void dense_tile(const DenseProblem& p, int unit, unsigned char* __restrict__ smem0) {
  constexpr bool PAIRED = dense_paired<EPI>();
  constexpr int OUT = PAIRED ? C::BN / 2 : C::BN;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave_all = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int kw = C::KW > 1 ? wave_all / C::kPos : 0, wave = C::KW > 1 ? wave_all % C::kPos : wave_all;
  unsigned char* __restrict__ smem = smem0 + kw * C::kRing;   // this group's ring
  const int wm = wave / C::WN, wn = wave % C::WN;
  const DenseUnit t = dense_unit(p, unit);
  const int m0 = t.mt * C::BM, n0 = t.nt * OUT;
  const int k_lo = t.split * p.k_split, k_hi = min(k_lo + p.k_split, p.K);
  // slices of a group (the last may lie past the range for some groups: zeros)
  const int nk = ((k_hi - k_lo + kDBK - 1) / kDBK + C::KW - 1) / C::KW;
  const bf16_t* __restrict__ A = (const bf16_t*)p.a;
  const bf16_t* __restrict__ B = (const bf16_t*)p.b;

  int a_off[C::kALoads], b_off[C::kBLoads];
  dense_offsets<C::BM, ACOL, C::kALoads>(a_off, p.lda, p.M - m0, false, 0, 0, wave, lane);
  dense_offsets<C::BN, BCOL, C::kBLoads>(b_off, p.ldb, p.N - n0, PAIRED, p.N - n0, p.N, wave, lane);
  // bytes a slice's descriptor spans past its base, less the k part
  const int a_rows = min(C::BM, p.M - m0);
  const int b_rows = PAIRED ? min(OUT, p.N - n0) + p.N : min(C::BN, p.N - n0);

  // An operand's slice kt: its first element and the bytes its descriptor
  // spans.  Slices past the last one span nothing: zeros land in a free slot.
  auto a_span = [&](int kt) {
    const int k0 = k_lo + (kt * C::KW + kw) * kDBK, kv = min(kDBK, k_hi - k0);
    return DenseSpan{ACOL ? A + (int64_t)k0 * p.lda + m0 : A + (int64_t)m0 * p.lda + k0,
                     kv > 0 ? 2 * (ACOL ? (kv - 1) * p.lda + a_rows : (a_rows - 1) * p.lda + kv) : 0, kv};
  };
  auto b_span = [&](int kt) {
    const int k0 = k_lo + (kt * C::KW + kw) * kDBK, kv = min(kDBK, k_hi - k0);
    return DenseSpan{BCOL ? B + (int64_t)k0 * p.ldb + n0 : B + (int64_t)n0 * p.ldb + k0,
                     kv > 0 ? 2 * (BCOL ? (kv - 1) * p.ldb + b_rows : (b_rows - 1) * p.ldb + kv) : 0, kv};
  };
  auto load_a = [&](const DenseSpan& d, int i, unsigned char* st) {
    dense_load<ACOL>(d, a_off[i], wave * C::kALoads + i, lane, st);
  };
  auto load_b = [&](const DenseSpan& d, int i, unsigned char* st) {
    dense_load<BCOL>(d, b_off[i], wave * C::kBLoads + i, lane, st);
  };
  auto issue_a = [&](int kt, unsigned char* st) {
    const DenseSpan d = a_span(kt);
#pragma unroll
    for (int i = 0; i < C::kALoads; ++i) load_a(d, i, st);
  };
  auto issue_b = [&](int kt, unsigned char* st) {
    const DenseSpan d = b_span(kt);
#pragma unroll
    for (int i = 0; i < C::kBLoads; ++i) load_b(d, i, st);
  };

  f32x4 acc[C::kMB][C::kNB];
#pragma unroll
  for (int mb = 0; mb < C::kMB; ++mb)
#pragma unroll
    for (int nb = 0; nb < C::kNB; ++nb) acc[mb][nb] = f32x4{0.f, 0.f, 0.f, 0.f};

  // Slots hold A(0) B(0) A(1) B(1) A(2) | B(2) A(3) ...: A(s) sits in slot
  // 2 s mod 5, B(s) in the next.
  issue_a(0, smem);
  issue_b(0, smem + C::kSlot);
  issue_a(1, smem + 2 * C::kSlot);
  issue_b(1, smem + 3 * C::kSlot);
  issue_a(2, smem + 4 * C::kSlot);
  wait_vmcnt<0>();
  lds_barrier();
  typedef DenseFrags<C> Frags;
  Frags f0, f1;
  auto mfmas = [&](const Frags& f) {
#pragma unroll
    for (int mb = 0; mb < C::kMB; ++mb)
#pragma unroll
      for (int nb = 0; nb < C::kNB; ++nb) acc[mb][nb] = dmfma(f.b[nb], f.a[mb], acc[mb][nb]);
  };
  dense_read<C, ACOL, BCOL, PAIRED>(smem, smem + C::kSlot, 0, wm, wn, lane, f0);
  dense_read<C, ACOL, BCOL, PAIRED>(smem, smem + C::kSlot, 1, wm, wn, lane, f1);
  mfmas(f0);
  // One slice: every fragment of slice s - 1 is in registers; wait for slice s
  // (the newest loads, A(s + 1), may stay in flight), then read on and refill the
  // two slots of slice s - 1 under the MFMAs.  The loads are spread over the
  // MFMAs: issued together after the barrier, the 64 of a workgroup queue for the
  // CU's one address path, and every wave's MFMAs queue behind its last load.
  // The slots written and the slots read never coincide: __restrict__ tells the
  // compiler, which otherwise waits for every load in flight before each LDS
  // read.
  auto slice = [&](int s, unsigned char* __restrict__ wa, unsigned char* __restrict__ wb,
                   const unsigned char* __restrict__ ra, const unsigned char* __restrict__ rb)
                   __attribute__((always_inline)) {
    const DenseSpan bd = b_span(s + 1);
    const DenseSpan ad = a_span(s + 2);
    __builtin_amdgcn_sched_barrier(0);
    wait_vmcnt<C::kALoads>();
    lds_barrier();
    dense_substep<C, C::kBLoads>(
        f1, acc, [&](int i) { dense_read1<C, ACOL, BCOL, PAIRED>(ra, rb, 0, i, wm, wn, lane, f0); },
        [&](int i) { load_b(bd, i, wa); });
    dense_substep<C, C::kALoads>(
        f0, acc, [&](int i) { dense_read1<C, ACOL, BCOL, PAIRED>(ra, rb, 1, i, wm, wn, lane, f1); },
        [&](int i) { load_a(ad, i, wb); });
  };
  int sa = 0, sb = 1;   // slots of slice s - 1
  for (int s = 1; s < nk; ++s) {
    const int ra = sa >= 3 ? sa - 3 : sa + 2, rb = sb >= 3 ? sb - 3 : sb + 2;
    slice(s, smem + sa * C::kSlot, smem + sb * C::kSlot, smem + ra * C::kSlot, smem + rb * C::kSlot);
    sa = ra;
    sb = rb;
  }
  // The tile goes through the ring a wave's 32 x 64 piece at a time (paired: 32
  // gate and 32 up columns); a lane then holds 8 consecutive columns of kJ rows.
  // A piece's epilogue inputs are loaded together, before the piece goes through
  // LDS; loading them a piece ahead measured the same.
  constexpr int kPieces = C::kMB / 2 * (C::kNB / 4), kJ = PAIRED ? 2 : 4;
  const bool fused = p.partial == nullptr;
  const int64_t ps = (int64_t)p.M * (PAIRED ? 2 * p.N : p.N);
  auto piece_row = [&](int mc, int j) {
    return m0 + wm * (C::BM / C::WM) + 32 * (mc / (C::kNB / 4)) + (PAIRED ? 16 * j + (lane >> 2) : 8 * j + (lane >> 3));
  };
  auto piece_col = [&](int mc) {
    return PAIRED ? n0 + wn * (C::BN / 2 / C::WN) + 32 * (mc % (C::kNB / 4)) + 8 * (lane & 3)
                  : n0 + wn * (C::BN / C::WN) + 64 * (mc % (C::kNB / 4)) + 8 * (lane & 7);
  };
  typedef EpiIn<bf16_t, EPI> In;
  auto load_piece = [&](int mc, In (&x)[kJ]) {
    if constexpr (In::N > 0) {
      if (!fused) return;
      const int n = piece_col(mc);
#pragma unroll
      for (int j = 0; j < kJ; ++j) {
        const int row = piece_row(mc, j);
        if (row < p.M && n < p.N) epi_load<bf16_t, EPI>(p.e, row, n, p.N, x[j]);
      }
    }
  };
  // The loop's last loads are zeros for slices past the end, but they still write
  // the ring: they land before any wave passes the barrier.
  wait_vmcnt<0>();
  mfmas(f1);
  lds_barrier();  // every wave has read its last fragments: the ring is free

  if constexpr (C::KW > 1) {
    // groups 1, 2, ... leave their sums in their rings; group 0 adds them in order
    if (kw > 0) {
#pragma unroll
      for (int mb = 0; mb < C::kMB; ++mb)
#pragma unroll
        for (int nb = 0; nb < C::kNB; ++nb)
          ((f32x4*)smem)[((wave * C::kMB + mb) * C::kNB + nb) * kWave + lane] = acc[mb][nb];
    }
    lds_barrier();
    if (kw > 0) return;
#pragma unroll
    for (int g = 1; g < C::KW; ++g)
#pragma unroll
      for (int mb = 0; mb < C::kMB; ++mb)
#pragma unroll
        for (int nb = 0; nb < C::kNB; ++nb)
          acc[mb][nb] += ((const f32x4*)(smem0 + g * C::kRing))[((wave * C::kMB + mb) * C::kNB + nb) * kWave + lane];
  }

  // Swapped 16x16 layout: row = lane % 16, column = 4 (lane / 16) + i.
  unsigned char* buf = smem + wave * 8192;   // 32 rows of 64 columns fp32, chunks XORed by the row
#pragma unroll
  for (int mc = 0; mc < kPieces; ++mc) {
    const int mp = mc / (C::kNB / 4), c = mc % (C::kNB / 4);
    In in[kJ];
    load_piece(mc, in);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int nb = 0; nb < 4; ++nb) {
        const int r = 16 * h + (lane & 15);
        *(f32x4*)(buf + r * 256 + (((4 * nb + (lane >> 4)) ^ (r & 15)) * 16)) = acc[2 * mp + h][4 * c + nb];
      }
    wave_lds_fence();
    auto get = [&](int row, int col8, float (&v)[8]) {
      const f32x4 a = *(const f32x4*)(buf + row * 256 + (((2 * col8) ^ (row & 15)) * 16));
      const f32x4 b = *(const f32x4*)(buf + row * 256 + (((2 * col8 + 1) ^ (row & 15)) * 16));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = a[i];
        v[4 + i] = b[i];
      }
    };
    const int n = piece_col(mc);
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
      const int row = piece_row(mc, j), rr = PAIRED ? 16 * j + (lane >> 2) : 8 * j + (lane >> 3);
      float v[8], u[8];
      if constexpr (PAIRED) {
        get(rr, lane & 3, v);
        get(rr, 4 + (lane & 3), u);
      } else {
        get(rr, lane & 7, v);
      }
      if (row < p.M && n < p.N) {
        if (fused) {
          epi8<bf16_t, EPI>(p.e, row, n, p.N, v, PAIRED ? u : v, in[j]);
        } else {
          float* o = p.partial + t.split * ps + (int64_t)row * (PAIRED ? 2 * p.N : p.N) + n;
          store8(o, v);
          if constexpr (PAIRED) store8(o + p.N, u);
        }
      }
    }
    wave_lds_fence();
  }
}

// ------------------------------------------------------------------------------------------
// float32: 32 x 32 tiles, 64-deep slices, fp32 FMAs
// ------------------------------------------------------------------------------------------
// The float32 path serves small layers, where a product is as long as one
// workgroup's chain of slices: small tiles, two halves of the workgroup on
// alternate halves of a slice (added at the end), and the next slice's loads in
// flight while one is worked on.  A thread holds eight columns of one row.
template <bool ACOL, bool BCOL, int EPI>
__device__ __forceinline__ void dense_f32_tile(const DenseProblem& p, int unit, float* smem) {
  constexpr bool PAIRED = dense_paired<EPI>();
  constexpr int KB = 64, NB = PAIRED ? 2 : 1;
  float(*sA)[36] = (float(*)[36])smem;                       // [KB][32 + 4]
  float(*sB)[36] = (float(*)[36])(smem + KB * 36);           // [NB * KB][32 + 4]
  const int tid = threadIdx.x;
  const int split = unit / (p.m_tiles * p.n_tiles), tile = unit % (p.m_tiles * p.n_tiles);
  const int m0 = (tile % p.m_tiles) * 32, n0 = (tile / p.m_tiles) * 32;
  const int k_lo = split * p.k_split, k_hi = min(k_lo + p.k_split, p.K);
  const float* A = (const float*)p.a;
  const float* B = (const float*)p.b;
  // A thread loads two float4 of each operand slice: along k ("row") or along the
  // other index ("col"); sizes are multiples of 8 along the contiguous one.
  auto load = [&](const float* src, bool col, int ld, int o0, int limit, int64_t shift, int k0, int i) {
    const int v = tid + 256 * i;
    const int k = col ? v / 8 : 4 * (v % 16), o = col ? 4 * (v % 8) : v / 16;
    const bool ok = o0 + o < limit && k0 + k < k_hi;
    const int64_t at = col ? (int64_t)(k0 + k) * ld + shift + o0 + o : (shift + o0 + o) * (int64_t)ld + k0 + k;
    return ok ? *(const f32x4*)(src + at) : f32x4{0.f, 0.f, 0.f, 0.f};
  };
  auto put = [&](float (*dst)[36], bool col, int i, const f32x4& x) {
    const int v = tid + 256 * i;
    if (col) {
      *(f32x4*)&dst[v / 8][4 * (v % 8)] = x;
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) dst[4 * (v % 16) + q][v / 16] = x[q];
    }
  };
  const int half = tid >> 7, r = (tid & 127) >> 2, c8 = tid & 3;
  float acc[NB][8];
#pragma unroll
  for (int h = 0; h < NB; ++h)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[h][j] = 0.f;
  f32x4 ra[2], rb[NB][2];
  auto fetch = [&](int k0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      ra[i] = load(A, ACOL, p.lda, m0, p.M, 0, k0, i);
#pragma unroll
      for (int h = 0; h < NB; ++h) rb[h][i] = load(B, BCOL, p.ldb, n0, p.N, h ? p.N : 0, k0, i);
    }
  };
  fetch(k_lo);
  for (int k0 = k_lo; k0 < k_hi; k0 += KB) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      put(sA, ACOL, i, ra[i]);
#pragma unroll
      for (int h = 0; h < NB; ++h) put(sB + h * KB, BCOL, i, rb[h][i]);
    }
    __syncthreads();
    if (k0 + KB < k_hi) fetch(k0 + KB);
#pragma unroll 8
    for (int q = 0; q < KB / 2; ++q) {
      const int k = half * (KB / 2) + q;
      const float a = sA[k][r];
#pragma unroll
      for (int h = 0; h < NB; ++h) {
        float b[8];
        load8(&sB[h * KB + k][8 * c8], b);
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[h][j] = fmaf(a, b[j], acc[h][j]);
      }
    }
  }
  // the upper half's sums are added to the lower half's
  __syncthreads();
  float* red = smem + (tid & 127) * 8 * NB;
  if (half) {
#pragma unroll
    for (int h = 0; h < NB; ++h) store8(red + 8 * h, acc[h]);
  }
  __syncthreads();
  const int m = m0 + r, n = n0 + 8 * c8;
  if (half || m >= p.M || n >= p.N) return;
#pragma unroll
  for (int h = 0; h < NB; ++h) {
    float b[8];
    load8(red + 8 * h, b);
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[h][j] += b[j];
  }
  if (p.partial) {
    float* o = p.partial + ((int64_t)split * p.M + m) * (PAIRED ? 2 * p.N : p.N) + n;
    store8(o, acc[0]);
    if constexpr (PAIRED) store8(o + p.N, acc[1]);
    return;
  }
  epi8_now<float, EPI>(p.e, m, n, p.N, acc[0], acc[NB - 1]);
}

template <int EPI>
constexpr int dense_f32_lds() { return (dense_paired<EPI>() ? 3 : 2) * 64 * 36; }

template <class C>
constexpr int dense_min_waves() { return C::kWgsPerCu * C::kWaves / 4 < 1 ? 1 : C::kWgsPerCu * C::kWaves / 4; }

typedef DenseCfg<128, 128, 2, 2> DenseM;   // 4 waves of 64 x 64, two workgroups per CU
typedef DenseCfg<128, 64, 4, 1> DenseN;    // 4 waves of 32 x 64, two per CU

}  // namespace
}  // namespace moe
