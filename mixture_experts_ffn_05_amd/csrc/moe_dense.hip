// Dense GEMMs of the shared expert in training: both forward halves and the
// input and weight gradients of both, with their elementwise work fused in.
//
// PLENA_Compiler PR #69, section "Group C -- shared experts": the shared expert
// is a dense FFN over every token.  Its training passes are the chain rule of
//
//   h = x Ws1 = [g | u],   a = silu(g) u,   ys = a Ws2,   y (+)= gate ys
//
// so they need five products: x Ws1 (SwiGLU epilogue, h and a stored), a Ws2
// (gate epilogue), D Ws2^T (SwiGLU' epilogue), d_h Ws1^T (gate gradient added),
// and the two weight gradients A^T D.  Every product is
//
//   C[m, n] = sum_k A(m, k) B(k, n)
//
// where an operand is stored either with k contiguous ("row": A [M, K],
// B [N, K]) or with its other index contiguous ("col": A [K, M], B [K, N]).
//
// bf16 kernel:
//   * One workgroup per output tile (BM x BN) and reduction range; slices of 64
//     along k travel HBM -> LDS with buffer_load ... lds into a ring of five
//     slots of one operand slice each (two whole slices and the next A: what 160
//     KiB hold of a 256 x 256 tile), so half of a slice's loads are issued two
//     slices ahead and half one slice ahead.  Rows, columns and k past an operand's end are out of the buffer
//     descriptor's range (or given an out-of-range offset), which the hardware
//     turns into zeros in LDS, so no size has a special path.
//   * "row" operands sit in LDS as 128-byte rows whose 16-byte chunks are XORed
//     with (row >> 1) & 7: an MFMA fragment is one ds_read_b128.  "col" operands
//     sit as k rows with chunks XORed by the k row; a fragment is two
//     ds_read_b64_tr_b16 transpose reads.
//   * v_mfma_f32_16x16x32_bf16: on random data the chip is bound by power, and a
//     register-only loop of it sustains 1985 TFLOP/s against 1750 of 32x32x16,
//     which moves four times the accumulators per instruction.
//   * Each wave alternates between two fragment sets: the next 32-deep
//     substep's LDS reads run under the current substep's MFMAs, across slice
//     boundaries too.
//   * The product is taken swapped (B's fragment as the MFMA's first operand),
//     so a lane holds four consecutive columns of one row; the tile goes through
//     the idle ring, a wave's 32 x 64 piece at a time, and the epilogue works on
//     eight consecutive columns per lane with 16-byte loads and stores.
//   * A reduction can be split over workgroups when the output has too few
//     tiles to fill the chip: partial sums go to the workspace in fp32 and
//     dense_finish adds them in split order and runs the same epilogue, so
//     results do not depend on timing.
// f32 kernel: 32 x 64 tiles, one row and eight columns per thread.
#include "moe_common.h"

#include <type_traits>

namespace moe {
namespace {

constexpr int kDBK = 64;        // reduction slice
constexpr int kSlots = 5;         // ring slots, one operand slice each
constexpr int kDXcds = 8;
constexpr int kOob = 0x7ffffff0;  // byte offset past every descriptor's range

// Epilogues.  v holds eight consecutive output columns of one row (for the
// paired one: g and u columns of the same outputs).
// kEPartial: partial sums only (the caller adds them).
enum DenseEpi { kESwigluSave = 0, kEGateAdd = 1, kESwigluBwd = 2, kEInputGrad = 3, kEStore = 4, kEPartial = 5 };

struct DenseEpiArgs {
  void* out;
  void* out2;
  const void* aux;
  const float* row;   // per-row factor, or null
  const void* col;    // per-column factor (kEInputGrad), or null
  int accumulate;
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
// the output is added to.  Loaded apart from its use, so that a tile's loads
// can be in flight while the tile before them is worked on.
template <typename T, int EPI>
struct EpiIn {
  static constexpr int N = EPI == kESwigluBwd ? (sizeof(T) == 2 ? 2 : 4) : (EPI == kEGateAdd || EPI == kEInputGrad) ? 2 : 0;
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
    store8(h, v);
    store8(h + N, v2);
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
    // dg = da u s (1 + g (1 - s)), du = da g s, s = sigmoid(g)
    float g[8], u[8];
    unpack8(in.v, g, T{});
    unpack8(in.v + EpiIn<T, EPI>::N / 2, u, T{});
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float s = epi_sigmoid<T>(g[i]);
      o[i] = v[i] * u[i] * s * (1.0f + g[i] * (1.0f - s));
      p[i] = v[i] * g[i] * s;
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
template <int BM_, int BN_, int WM_, int WN_>
struct DenseCfg {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;
  static constexpr int kWaves = WM * WN, NT = kWaves * kWave;
  static constexpr int kMB = BM / WM / 16, kNB = BN / WN / 16;   // 16 x 16 MFMA blocks of a wave
  static constexpr int kABytes = BM * kDBK * 2, kBBytes = BN * kDBK * 2;   // one operand slice
  static constexpr int kALoads = kABytes / 1024 / kWaves, kBLoads = kBBytes / 1024 / kWaves;
  static constexpr int kSlot = kABytes > kBBytes ? kABytes : kBBytes;
  static constexpr int kLds = kSlots * kSlot;
  static constexpr int kFit = (160 * 1024) / kLds;
  static constexpr int kWgs0 = kFit < 1 ? 1 : kFit;
  // waves per SIMD that the registers allow: 128-accumulator waves fit two
  static constexpr int kWgsPerCu = kWgs0 * kWaves > 8 ? (8 / kWaves < 1 ? 1 : 8 / kWaves) : kWgs0;
  static_assert(kABytes % (1024 * kWaves) == 0 && kBBytes % (1024 * kWaves) == 0, "slices split into 1 KiB loads");
  static_assert(kMB % 2 == 0 && kNB % 4 == 0, "a wave holds pairs of 16-row blocks and 64-column pieces");
  static_assert(kWaves * 8192 <= kLds, "epilogue: 8 KiB of the ring per wave");
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
__device__ __forceinline__ void dense_tile(const DenseProblem& p, int unit, unsigned char* __restrict__ smem) {
  constexpr bool PAIRED = dense_paired<EPI>();
  constexpr int OUT = PAIRED ? C::BN / 2 : C::BN;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / C::WN, wn = wave % C::WN;
  const DenseUnit t = dense_unit(p, unit);
  const int m0 = t.mt * C::BM, n0 = t.nt * OUT;
  const int k_lo = t.split * p.k_split, k_hi = min(k_lo + p.k_split, p.K);
  const int nk = (k_hi - k_lo + kDBK - 1) / kDBK;
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
    const int k0 = k_lo + kt * kDBK, kv = min(kDBK, k_hi - k0);
    return DenseSpan{ACOL ? A + (int64_t)k0 * p.lda + m0 : A + (int64_t)m0 * p.lda + k0,
                     kv > 0 ? 2 * (ACOL ? (kv - 1) * p.lda + a_rows : (a_rows - 1) * p.lda + kv) : 0, kv};
  };
  auto b_span = [&](int kt) {
    const int k0 = k_lo + kt * kDBK, kv = min(kDBK, k_hi - k0);
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
  // The next piece's epilogue inputs are loaded while this one is worked on.
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
  In in[2][kJ];
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
  load_piece(0, in[0]);
  mfmas(f1);
  lds_barrier();  // every wave has read its last fragments: the ring is free

  // Swapped 16x16 layout: row = lane % 16, column = 4 (lane / 16) + i.
  unsigned char* buf = smem + wave * 8192;   // 32 rows of 64 columns fp32, chunks XORed by the row
#pragma unroll
  for (int mc = 0; mc < kPieces; ++mc) {
    const int mp = mc / (C::kNB / 4), c = mc % (C::kNB / 4);
    if (mc + 1 < kPieces) load_piece(mc + 1, in[(mc + 1) & 1]);
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
          epi8<bf16_t, EPI>(p.e, row, n, p.N, v, PAIRED ? u : v, in[mc & 1][j]);
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

template <class C>
constexpr int dense_min_waves() { return C::kWgsPerCu * C::kWaves / 4 < 1 ? 1 : C::kWgsPerCu * C::kWaves / 4; }

template <class C, bool ACOL, bool BCOL, int EPI>
__global__ __launch_bounds__(C::NT, dense_min_waves<C>()) void dense_bf16(DenseProblem p) {
  extern __shared__ __attribute__((aligned(1024))) unsigned char smem[];
  dense_tile<C, ACOL, BCOL, EPI>(p, blockIdx.x, smem);
}

// The two products of a half's backward in one launch: the input gradient (d)
// and the weight gradient (w).  Their tiles have different reduction lengths;
// the host puts the longer ones first (n_first units of them), so the
// dispatcher fills the CUs that finish early with the shorter ones, and the
// epilogues of the two kinds do not run at the same time on every CU.
template <class CD, class CW, bool BCOL, int EPI>
__global__ __launch_bounds__(CD::NT, dense_min_waves<CW>()) void dense_pair_bf16(DenseProblem d, DenseProblem w,
                                                                                 int n_first, int w_first) {
  static_assert(CD::NT == CW::NT, "one workgroup size");
  extern __shared__ __attribute__((aligned(1024))) unsigned char smem[];
  const int u = blockIdx.x;
  if ((u < n_first) != (w_first != 0))
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
  float v[8] = {0, 0, 0, 0, 0, 0, 0, 0}, w[8] = {0, 0, 0, 0, 0, 0, 0, 0}, x[8];
  for (int z = 0; z < p.splits; ++z) {
    load8(s + z * ps, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += x[j];
    if constexpr (PAIRED) {
      load8(s + z * ps + p.N, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] += x[j];
    }
  }
  epi8_now<T, EPI>(p.e, m, n, p.N, v, w);
}

// ------------------------------------------------------------------------------------------
// float32: 32 x 64 tiles, 16-deep slices in LDS, fp32 FMAs
// ------------------------------------------------------------------------------------------
template <bool ACOL, bool BCOL, int EPI>
__global__ __launch_bounds__(256) void dense_f32(DenseProblem p) {
  constexpr bool PAIRED = dense_paired<EPI>();
  constexpr int KB = 16;
  __shared__ float sA[KB][33];
  __shared__ __attribute__((aligned(16))) float sB[PAIRED ? 2 : 1][KB][64];
  const int tid = threadIdx.x;
  const int split = blockIdx.x / (p.m_tiles * p.n_tiles), tile = blockIdx.x % (p.m_tiles * p.n_tiles);
  const int m0 = (tile % p.m_tiles) * 32, n0 = (tile / p.m_tiles) * 64;
  const int k_lo = split * p.k_split, k_hi = min(k_lo + p.k_split, p.K);
  const float* A = (const float*)p.a;
  const float* B = (const float*)p.b;
  const int r = tid >> 3, c8 = tid & 7;
  float v[8] = {0, 0, 0, 0, 0, 0, 0, 0}, w[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  for (int k0 = k_lo; k0 < k_hi; k0 += KB) {
    for (int i = tid; i < 32 * KB; i += 256) {
      const int m = ACOL ? i % 32 : i / KB, k = ACOL ? i / 32 : i % KB;
      const bool ok = m0 + m < p.M && k0 + k < k_hi;
      sA[k][m] = ok ? A[ACOL ? (int64_t)(k0 + k) * p.lda + m0 + m : (int64_t)(m0 + m) * p.lda + k0 + k] : 0.f;
    }
#pragma unroll
    for (int h = 0; h < (PAIRED ? 2 : 1); ++h)
      for (int i = tid; i < 64 * KB; i += 256) {
        const int n = BCOL ? i % 64 : i / KB, k = BCOL ? i / 64 : i % KB;
        const bool ok = n0 + n < p.N && k0 + k < k_hi;
        const int64_t nn = n0 + n + (h ? p.N : 0);
        sB[h][k][n] = ok ? B[BCOL ? (int64_t)(k0 + k) * p.ldb + nn : nn * p.ldb + k0 + k] : 0.f;
      }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < KB; ++k) {
      const float a = sA[k][r];
      float b[8];
      load8(&sB[0][k][8 * c8], b);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = fmaf(a, b[j], v[j]);
      if constexpr (PAIRED) {
        load8(&sB[1][k][8 * c8], b);
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = fmaf(a, b[j], w[j]);
      }
    }
    __syncthreads();
  }
  const int m = m0 + r, n = n0 + 8 * c8;
  if (m >= p.M || n >= p.N) return;
  if (p.partial) {
    float* o = p.partial + ((int64_t)split * p.M + m) * (PAIRED ? 2 * p.N : p.N) + n;
    store8(o, v);
    if constexpr (PAIRED) store8(o + p.N, w);
    return;
  }
  epi8_now<float, EPI>(p.e, m, n, p.N, v, w);
}

// ------------------------------------------------------------------------------------------
// Elementwise and reduction steps
// ------------------------------------------------------------------------------------------
// One wave per token.  gate[t] = sigmoid(x[t] . w_gate), fp32.
template <typename T>
__global__ __launch_bounds__(256) void dense_gate(const T* __restrict__ x, const T* __restrict__ wg, int Tn, int H,
                                                  float* __restrict__ gate) {
  const int lane = threadIdx.x & 63;
  const int t = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= Tn) return;
  float s = 0.f;
  for (int h = 8 * lane; h < H; h += 512) {
    float a[8], b[8];
    load8(x + (int64_t)t * H + h, a);
    load8(wg + h, b);
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fmaf(a[i], b[i], s);
  }
  s = wave_sum(s);
  if (lane == 0) gate[t] = sigmoidf_(s);
}

// One wave per token: d_rows[t] = gate[t] * dy[t] in the element type (null: not
// wanted), and the gate logit's gradient gate (1 - gate) (dy[t] . ys[t]).
template <typename T>
__global__ __launch_bounds__(256) void dense_dy(const float* __restrict__ dy, const float* __restrict__ ys,
                                                const float* __restrict__ gate, int Tn, int H, T* __restrict__ d_rows,
                                                float* __restrict__ d_z) {
  const int lane = threadIdx.x & 63;
  const int t = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= Tn) return;
  const float g = gate ? gate[t] : 1.0f;
  const int64_t base = (int64_t)t * H;
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
  if (!gate) return;
  s = wave_sum(s);
  if (lane == 0) d_z[t] = g * (1.0f - g) * s;
}

// part[c][h] = sum over the rows of chunk c of d_z[t] x[t, h]; 512 columns and
// kGateRows rows per workgroup, the four waves' sums added in wave order.
constexpr int kGateRows = 64;
template <typename T>
__global__ __launch_bounds__(256) void dense_gate_grad(const float* __restrict__ d_z, const T* __restrict__ x, int Tn,
                                                       int H, float* __restrict__ part) {
  __shared__ __attribute__((aligned(16))) float s_part[4][512];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int h = blockIdx.y * 512 + 8 * lane;
  const int64_t t0 = (int64_t)blockIdx.x * kGateRows, t1 = min(t0 + kGateRows, (int64_t)Tn);
  float s[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (h < H)
    for (int64_t t = t0 + wave; t < t1; t += 4) {
      float a[8];
      load8(x + t * H + h, a);
      const float z = d_z[t];
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = fmaf(z, a[i], s[i]);
    }
  store8(&s_part[wave][8 * lane], s);
  __syncthreads();
  for (int c = threadIdx.x; c < 512; c += 256) {
    const int col = blockIdx.y * 512 + c;
    if (col < H)
      part[(int64_t)blockIdx.x * H + col] = ((s_part[0][c] + s_part[1][c]) + s_part[2][c]) + s_part[3][c];
  }
}

// One workgroup per 64 columns: four waves each add a quarter of the chunks in
// order, and the quarters are added in order.
template <typename T>
__global__ __launch_bounds__(256) void dense_gate_grad_sum(const float* __restrict__ part, int chunks, int H,
                                                           T* __restrict__ d_wg) {
  __shared__ float s_q[4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int h = blockIdx.x * 64 + lane;
  const int per = (chunks + 3) / 4, c0 = wave * per, n = max(min(per, chunks - c0), 0);
  s_q[wave][lane] = h < H ? sum_slices(part + (int64_t)c0 * H + h, H, n) : 0.f;
  __syncthreads();
  if (wave == 0 && h < H)
    store_from_f32(d_wg, h, ((s_q[0][lane] + s_q[1][lane]) + s_q[2][lane]) + s_q[3][lane]);
}

// ------------------------------------------------------------------------------------------
// Host: configurations and their choice
// ------------------------------------------------------------------------------------------
typedef DenseCfg<256, 256, 2, 2> DenseL;   // 4 waves of 128 x 128, one workgroup per CU
typedef DenseCfg<256, 256, 2, 4> DenseL8;  // 8 waves of 128 x 64
typedef DenseCfg<128, 128, 2, 2> DenseM;   // 4 waves of 64 x 64, two per CU
typedef DenseCfg<64, 128, 2, 2> DenseS;    // 4 waves of 32 x 64, two per CU

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

// The 256 x 256 tile has four waves, whose 128 x 128 pieces read a third less
// LDS than eight waves' 128 x 64 (measured, Scout-shaped fc2 forward at 2048
// tokens 165 against 178 us; fc1 backward at 4096 tokens 330 against 336), except
// with SwiGLU's gradient as the epilogue, whose loads and arithmetic want two
// waves per SIMD (fc2 backward at 4096 tokens 207 against 241 us).
template <int EPI>
using DenseLarge = std::conditional_t<EPI == kESwigluBwd, DenseL8, DenseL>;

// A configuration's tile, its workgroups per CU, and measured microseconds: per
// 64-deep slice with one workgroup on a CU and with every slot taken, and per
// tile besides its slices.
struct DenseShape {
  int bm, bn, slots;
  double alone, full, fixed;
};
constexpr DenseShape kShapeL{256, 256, 1, 1.2, 1.5, 6.0}, kShapeM{128, 128, 2, 0.53, 0.95, 3.0},
    kShapeS{64, 128, 2, 0.46, 0.58, 3.0};
// Choices for one product, or for the input and the weight gradient of a pair
// (the two 4-wave tiles of 256 threads can share a launch).
struct DenseChoice {
  DenseShape d, w;
};
constexpr DenseChoice kChoices[4] = {{kShapeL, kShapeL}, {kShapeM, kShapeM}, {kShapeS, kShapeS}, {kShapeS, kShapeM}};
// A split product's second launch, and its partial sums' trip through memory.
constexpr double kFinishUs = 4.0, kFinishUsPerMb = 0.38;

// One product's tiles: M x Ns outputs (Ns counts the staged columns: both halves
// of a paired product), K reduced.
struct DenseWork {
  int M, Ns, K;
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
  for (int c = 0; c < (products == 2 ? 4 : 3); ++c) {
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
          if (sp[q] > 1) extra += kFinishUs + kFinishUsPerMb * sp[q] * ((double)w[q].M * w[q].Ns * 4e-6);
        }
        if (!ok) continue;
        // average share of the slots at work while the longest tile runs
        double work = 0, chain = 0;
        for (int q = 0; q < products; ++q) {
          const double one = per[q] * sh[q]->full;
          work += one * units[q];
          chain = one > chain ? one : chain;
        }
        double occ = work / (chain * slots);
        occ = occ < 1.0 ? occ : 1.0;
        const double shared = (occ * slots - cu_count) / (slots - cu_count + 1e-9);
        const double busy = sh[0]->slots == 1 ? occ : shared > 0 ? shared : 0.0;
        for (int q = 0; q < products; ++q)
          len[q] = per[q] * (sh[q]->alone + busy * (sh[q]->full - sh[q]->alone)) + sh[q]->fixed;
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
  static const hipError_t attr = hipFuncSetAttribute(reinterpret_cast<const void*>(&dense_bf16<C, ACOL, BCOL, EPI>),
                                                     hipFuncAttributeMaxDynamicSharedMemorySize, C::kLds);
  if (attr != hipSuccess) return attr;
  set_tiles<C, dense_paired<EPI>()>(p);
  hipLaunchKernelGGL((dense_bf16<C, ACOL, BCOL, EPI>), dim3(p.m_tiles * p.n_tiles * p.splits), dim3(C::NT), C::kLds, s,
                     p);
  return hipGetLastError();
}

template <class CD, class CW, bool BCOL, int EPI>
hipError_t launch_pair_cfg(DenseProblem d, DenseProblem w, bool w_first, hipStream_t s) {
  constexpr int lds = CD::kLds > CW::kLds ? CD::kLds : CW::kLds;
  static const hipError_t attr =
      hipFuncSetAttribute(reinterpret_cast<const void*>(&dense_pair_bf16<CD, CW, BCOL, EPI>),
                          hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (attr != hipSuccess) return attr;
  set_tiles<CD, false>(d);
  set_tiles<CW, false>(w);
  const int nd = d.m_tiles * d.n_tiles * d.splits, nw = w.m_tiles * w.n_tiles * w.splits;
  hipLaunchKernelGGL((dense_pair_bf16<CD, CW, BCOL, EPI>), dim3(nd + nw), dim3(CD::NT), lds, s, d, w,
                     w_first ? nw : nd, w_first ? 1 : 0);
  return hipGetLastError();
}

template <bool ACOL, bool BCOL, int EPI>
hipError_t launch_f32(DenseProblem p, hipStream_t s) {
  p.m_tiles = (p.M + 31) / 32;
  p.n_tiles = (p.N + 63) / 64;
  hipLaunchKernelGGL((dense_f32<ACOL, BCOL, EPI>), dim3(p.m_tiles * p.n_tiles * p.splits), dim3(256), 0, s, p);
  return hipGetLastError();
}

void whole_reduction(DenseProblem& p) {
  p.splits = 1;
  p.k_split = (p.K + kDBK - 1) / kDBK * kDBK;
}

template <int EPI>
DenseWork work_of(const DenseProblem& p) {
  return DenseWork{p.M, dense_paired<EPI>() ? 2 * p.N : p.N, p.K};
}

// One product; B is the weight (b_col: stored [K, N], else [N, K]).
template <int EPI>
hipError_t launch_forward(int dt, bool b_col, DenseProblem p, float* partial, size_t cap, int cu_count, hipStream_t s) {
  whole_reduction(p);
  if (dt != 1) return b_col ? launch_f32<false, true, EPI>(p, s) : launch_f32<false, false, EPI>(p, s);
  const DenseWork w[2] = {work_of<EPI>(p), {0, 0, 0}};
  const DensePlan plan = dense_plan(w, cap, cu_count);
  p.splits = plan.splits[0];
  p.k_split = plan.k_split[0];
  p.partial = p.splits > 1 ? partial : nullptr;
  auto go = [&](auto c) {
    typedef decltype(c) C;
    return b_col ? launch_dense_cfg<C, false, true, EPI>(p, s) : launch_dense_cfg<C, false, false, EPI>(p, s);
  };
  const hipError_t err = plan.choice == 0 ? go(DenseLarge<EPI>{}) : plan.choice == 1 ? go(DenseM{}) : go(DenseS{});
  if (err != hipSuccess || !p.partial) return err;
  return launch_finish<bf16_t, EPI>(p, s);
}

// The two products of a half's backward: d (epilogue EPI, B the weight) and w (the weight's gradient).
template <int EPI>
hipError_t launch_backward(int dt, bool b_col, DenseProblem d, DenseProblem w, float* partial, size_t cap,
                           int cu_count, hipStream_t s) {
  whole_reduction(d);
  whole_reduction(w);
  if (dt != 1) {
    const hipError_t err = b_col ? launch_f32<false, true, EPI>(d, s) : launch_f32<false, false, EPI>(d, s);
    return err != hipSuccess ? err : launch_f32<true, true, kEStore>(w, s);
  }
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
    return b_col ? launch_pair_cfg<CD, CW, true, EPI>(d, w, plan.w_first, s)
                 : launch_pair_cfg<CD, CW, false, EPI>(d, w, plan.w_first, s);
  };
  typedef DenseLarge<EPI> Large;
  hipError_t err = plan.choice == 0   ? go(Large{}, Large{})
                   : plan.choice == 1 ? go(DenseM{}, DenseM{})
                   : plan.choice == 2 ? go(DenseS{}, DenseS{})
                                      : go(DenseS{}, DenseM{});
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
    const dim3 grid((T + 3) / 4);
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
  const dim3 grid((T + 3) / 4);
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
  return launch_backward<kESwigluBwd>(dt, wl == 1, d, w, shared_partials(ws, dt, T, H), partial_cap(T, H, I_s), cu_count,
                                      s);
}

hipError_t shared_fc1_backward(int dt, int wl, const void* d_h, const void* x, const void* ws1, const float* d_z,
                               const void* w_gate, int T, int H, int I_s, int accumulate, float* d_x, void* d_ws1,
                               void* d_w_gate, void* ws, int cu_count, hipStream_t s) {
  using namespace moe;
  // d_x = d_h Ws1^T: reduction 2 I_s, outputs H; Ws1 [H, 2 I_s] is the "row" form here
  DenseProblem d{d_h, ws1, T, H, 2 * I_s, 2 * I_s, wl ? H : 2 * I_s};
  d.e = DenseEpiArgs{d_x, nullptr, nullptr, w_gate ? d_z : nullptr, w_gate, accumulate};
  DenseProblem w = wl ? DenseProblem{d_h, x, 2 * I_s, H, T, 2 * I_s, H} : DenseProblem{x, d_h, H, 2 * I_s, T, H, 2 * I_s};
  w.e = DenseEpiArgs{d_ws1, nullptr, nullptr, nullptr, nullptr, 0};
  const hipError_t err = launch_backward<kEInputGrad>(dt, wl == 1, d, w, shared_partials(ws, dt, T, H),
                                                      partial_cap(T, H, I_s), cu_count, s);
  if (err != hipSuccess || !w_gate) return err;
  const int chunks = (T + kGateRows - 1) / kGateRows;
  const dim3 g1(chunks, (H + 511) / 512), g2((H + 63) / 64);
  float* part = (float*)ws;
  if (dt == 1) {
    hipLaunchKernelGGL(dense_gate_grad<bf16_t>, g1, dim3(256), 0, s, d_z, (const bf16_t*)x, T, H, part);
    hipLaunchKernelGGL(dense_gate_grad_sum<bf16_t>, g2, dim3(256), 0, s, part, chunks, H, (bf16_t*)d_w_gate);
  } else {
    hipLaunchKernelGGL(dense_gate_grad<float>, g1, dim3(256), 0, s, d_z, (const float*)x, T, H, part);
    hipLaunchKernelGGL(dense_gate_grad_sum<float>, g2, dim3(256), 0, s, part, chunks, H, (float*)d_w_gate);
  }
  return hipGetLastError();
}

// d_w partial sums of the router: part[z][h][e] = sum over tokens of range z of x[t, h] d_logits[t, e], x [T, H] and
// d_logits [T, Ep] in the element type, Ep a multiple of 8.
hipError_t router_wgrad_partials(int dt, const void* x, const void* d_logits, int T, int H, int Ep, int splits,
                                 int k_split, float* part, hipStream_t s) {
  using namespace moe;
  DenseProblem p{x, d_logits, H, Ep, T, H, Ep, splits, k_split};
  p.partial = part;
  return dt == 1 ? launch_dense_cfg<DenseM, true, true, kEPartial>(p, s) : launch_f32<true, true, kEPartial>(p, s);
}

}  // namespace moe_launch
