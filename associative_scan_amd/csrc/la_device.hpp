// Building blocks of the linear attention kernels: tiles in LDS, matrix-core
// fragments, the split of fp32 values into 16-bit pieces, and the per-chunk
// decays.
//
// One recurrence, S_t = e^{g_t} S_{t-1} + y_t z_t^T, out_t = S_t^T x_t, is run
// in chunks of C steps. With b the inclusive cumulative sum of g in a chunk and
// S the state before it,
//   out_r = e^{b_r} x_r S + sum_{c <= r} e^{b_r - b_c} (x_r . y_c) z_c
//   S'    = e^{b_C} S + sum_c y_c (e^{b_C - b_c} z_c)^T
// and, run from the last step to the first (the adjoint, whose decay enters
// after a step instead of before it),
//   out_r = e^{b_C - b_r} x_r S + sum_{c >= r} e^{b_c - b_r} (x_r . y_c) z_c
//   S'    = e^{b_C} S + sum_c y_c (e^{b_c} z_c)^T.
// The forward pass is (x, y, z) = (q, k, v); with Lam the reverse state of
// (q, do), dq is (do, v, k), and in reverse dv is (k, q, do), dk is (v, do, q).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "la_launch.hpp"

namespace mscan {
namespace la {

typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf4 __attribute__((ext_vector_type(4)));
typedef short s4v __attribute__((ext_vector_type(4)));
typedef float f4v __attribute__((ext_vector_type(4)));
typedef float f8v __attribute__((ext_vector_type(8)));
typedef float f16v __attribute__((ext_vector_type(16)));
typedef uint32_t u4v __attribute__((ext_vector_type(4)));
typedef uint32_t u2v __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ int lane_id() { return (int)(threadIdx.x & 63); }
// The lane as a value of its own: what is computed from it stays inside the
// phase of a chunk that asks for it, instead of in registers over the whole
// loop over chunks.
__device__ __forceinline__ int fresh_lane() {
  int l = lane_id();
  asm volatile("" : "+v"(l));
  return l;
}
// Keeps the reads of later steps of a phase from being moved ahead, which
// would hold their results in registers too.
__device__ __forceinline__ void step_fence() { __builtin_amdgcn_sched_barrier(0); }

// ---------------------------------------------------------------------------
// matrix-core fragments
//
// A fragment holds 8 values per lane of an operand's contraction axis. Lanes l
// and l + 32 (32-wide tiles) take the axis entries {4h + j, 8 + 4h + j}, j < 4,
// h = l / 32, of a 16-step: the entries that an accumulator of the previous
// product holds in 8 consecutive registers, so a state kept in accumulators is
// an operand without a move between lanes. Both operands use the same order, so
// the product does not depend on it. fp32 math issues eight products of one
// value per lane in place of one 16-bit product of eight.
// ---------------------------------------------------------------------------
template <class TM>
struct Math;

template <>
struct Math<__bf16> {
  typedef bf8 Frag;
  typedef bf4 Unit;  // 4 consecutive elements of a tile row
  static __device__ __forceinline__ f16v mma32(Frag a, Frag b, f16v c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ f4v mma16(Frag a, Frag b, f4v c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ Frag join(Unit a, Unit b) {
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  }
  static __device__ __forceinline__ f8v widen(Frag f) { return __builtin_convertvector(f, f8v); }
};

template <>
struct Math<float> {
  typedef f8v Frag;
  typedef f4v Unit;
  static __device__ __forceinline__ f16v mma32(Frag a, Frag b, f16v c) {
#pragma unroll
    for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[e], b[e], c, 0, 0, 0);
    return c;
  }
  static __device__ __forceinline__ f4v mma16(Frag a, Frag b, f4v c) {
#pragma unroll
    for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
    return c;
  }
  static __device__ __forceinline__ Frag join(Unit a, Unit b) {
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  }
  static __device__ __forceinline__ f8v widen(Frag f) { return f; }
};

// x as a sum of N fragments: bf16 pieces of 8 bits each, every piece the
// rounding of what the ones before it left (N = 2: off by 2^-18 of x at most,
// N = 3: exact but for fp32's own last bits); fp32 math takes x whole.
template <class TM, int N>
__device__ __forceinline__ void split8(f8v x, typename Math<TM>::Frag (&out)[N]) {
  if constexpr (sizeof(TM) == 4) {
    out[0] = x;
  } else {
#pragma unroll
    for (int p = 0; p < N; ++p) {
      out[p] = __builtin_convertvector(x, bf8);
      if (p + 1 < N) x -= __builtin_convertvector(out[p], f8v);
    }
  }
}
template <class TM, int N>
__device__ __forceinline__ void split4(f4v x, typename Math<TM>::Unit (&out)[N]) {
  if constexpr (sizeof(TM) == 4) {
    out[0] = x;
  } else {
#pragma unroll
    for (int p = 0; p < N; ++p) {
      out[p] = __builtin_convertvector(x, bf4);
      if (p + 1 < N) x -= __builtin_convertvector(out[p], f4v);
    }
  }
}

// ---------------------------------------------------------------------------
// tiles in LDS: [rows][D] in units of 4 elements, the unit index of a row
// XORed with a function of the row. 8-byte units (16-bit elements): 32 rows at
// one unit index, and 4 rows at 8 consecutive ones, each cover all 64 banks.
// 16-byte units (fp32): 16 rows at one unit index do.
// ---------------------------------------------------------------------------
template <class TM, int D>
__device__ __forceinline__ int swizzle(int row) {
  constexpr int U = D / 4;
  static_assert(U == 8 || U == 16 || U == 32, "tile width");
  if constexpr (sizeof(TM) == 2) {
    constexpr int drop = U >= 32 ? 0 : (U == 16 ? 1 : 2);
    return (((row & 3) >> drop) << 3) | ((row >> 2) & 7);
  } else {
    return U >= 16 ? (row & 15) : ((row >> 1) & 7);
  }
}
template <class TM, int D>
__device__ __forceinline__ int unit_at(int row, int unit) {  // element offset of a unit
  return row * D + ((unit ^ swizzle<TM, D>(row)) << 2);
}

// rows row0 + (l & 31), contraction axis along the row at k0 (32-wide tiles)
template <class TM, int D>
__device__ __forceinline__ typename Math<TM>::Frag row_frag32(const TM* tile, int row0, int k0, int l) {
  typedef typename Math<TM>::Unit Unit;
  const int row = row0 + (l & 31), u = (k0 >> 2) + (l >> 5);
  const Unit a = *(const Unit*)(tile + unit_at<TM, D>(row, u));
  const Unit b = *(const Unit*)(tile + unit_at<TM, D>(row, u + 2));
  return Math<TM>::join(a, b);
}
// rows row0 + (l & 15), 32 axis entries from k0 (16-wide tiles); the four lane
// groups take units {0,2}, {4,6}, {1,3}, {5,7}, which keeps a read of 32 lanes
// on distinct banks
template <class TM, int D>
__device__ __forceinline__ typename Math<TM>::Frag row_frag16(const TM* tile, int row0, int k0, int l) {
  typedef typename Math<TM>::Unit Unit;
  const int row = row0 + (l & 15), q = l >> 4;
  const int u = (k0 >> 2) + ((q & 1) << 2) + (q >> 1);
  const Unit a = *(const Unit*)(tile + unit_at<TM, D>(row, u));
  const Unit b = *(const Unit*)(tile + unit_at<TM, D>(row, u + 2));
  return Math<TM>::join(a, b);
}
// columns col0 + (l & 31), contraction axis down the rows from row0 (a 16-step)
template <class TM, int D>
__device__ __forceinline__ typename Math<TM>::Frag col_frag32(const TM* tile, int row0, int col0, int l) {
  const int h = l >> 5;
  if constexpr (sizeof(TM) == 2) {
    // a transposing read: each 16 lanes read 4 rows x 16 columns, lane i of
    // them 8 bytes of row i / 4, and get column i of the four rows
    typedef __attribute__((address_space(3))) s4v* lds4;
    const int row = row0 + 4 * h + ((l & 15) >> 2);
    const int u = (col0 >> 2) + ((l >> 4) & 1) * 4 + (l & 3);
    const s4v a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(tile + unit_at<TM, D>(row, u)));
    const s4v b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(tile + unit_at<TM, D>(row + 8, u)));
    return Math<TM>::join(__builtin_bit_cast(bf4, a), __builtin_bit_cast(bf4, b));
  } else {
    const int c = col0 + (l & 31);
    f8v f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int row = row0 + 4 * h + (e & 3) + ((e >> 2) << 3);
      f[e] = tile[unit_at<TM, D>(row, c >> 2) + (c & 3)];
    }
    return f;
  }
}

// ---------------------------------------------------------------------------
// global memory -> registers -> LDS, 8 elements per thread and step. Rows at or
// past nrows and columns at or past d (a multiple of 8) become zeros.
// ---------------------------------------------------------------------------
template <class TIn>
struct Raw {
  u4v w[sizeof(TIn) == 4 ? 2 : 1];
};

template <class TIn, int C, int D, int NT>
struct TileRegs {
  static constexpr int N = C * (D / 8) / NT;
  static_assert(C * (D / 8) % NT == 0, "tile split");
  Raw<TIn> r[N];

  __device__ __forceinline__ void load(const TIn* base, int64_t st, int d, int nrows, int tid) {
    asm volatile("" : "+v"(tid));  // addresses are built anew for every chunk
    constexpr int STEP = NT / (D / 8);  // rows between a thread's loads
    static_assert(NT % (D / 8) == 0, "rows per pass");
    const int row0 = tid / (D / 8), c = (tid % (D / 8)) * 8;
    const TIn* p = base + (int64_t)row0 * st + c;
    const int n = c < d ? nrows : 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      r[i].w[0] = u4v{0, 0, 0, 0};
      if constexpr (sizeof(TIn) == 4) r[i].w[1] = u4v{0, 0, 0, 0};
      if (row0 + i * STEP < n) {
        r[i].w[0] = *(const u4v*)p;
        if constexpr (sizeof(TIn) == 4) r[i].w[1] = *(const u4v*)(p + 4);
      }
      p += STEP * st;
    }
  }
  template <class TM>
  __device__ __forceinline__ void store(TM* tile, int tid) const {
    asm volatile("" : "+v"(tid));
    typedef typename Math<TM>::Unit Unit;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = tid + i * NT, row = e / (D / 8), u = (e % (D / 8)) * 2;
      Unit a, b;
      if constexpr (sizeof(TIn) == 4) {
        a = __builtin_bit_cast(f4v, r[i].w[0]);
        b = __builtin_bit_cast(f4v, r[i].w[1]);
      } else if constexpr (sizeof(TM) == 4) {  // 16-bit input, fp32 math: widened exactly
        const f8v f = __builtin_convertvector(__builtin_bit_cast(h8, r[i].w[0]), f8v);
        a = __builtin_shufflevector(f, f, 0, 1, 2, 3);
        b = __builtin_shufflevector(f, f, 4, 5, 6, 7);
      } else {
        const bf8 f = __builtin_bit_cast(bf8, r[i].w[0]);
        a = __builtin_shufflevector(f, f, 0, 1, 2, 3);
        b = __builtin_shufflevector(f, f, 4, 5, 6, 7);
      }
      *(Unit*)(tile + unit_at<TM, D>(row, u)) = a;
      *(Unit*)(tile + unit_at<TM, D>(row, u + 1)) = b;
    }
  }
};

// ---------------------------------------------------------------------------
// decays of a chunk
// ---------------------------------------------------------------------------
// Cumulative log decays in base 2 and 64 bits: differences of nearby steps keep
// their digits next to strong decays, and a reset (g = -inf, taken as -1e5, a
// factor of zero in fp32) leaves no inf - inf.
template <int C>
struct Decays {
  double b[C];   // inclusive cumulative sum
  float up[C];   // e^{b_t}
  float dn[C];   // e^{b_C - b_t}
  float all;     // e^{b_C}
  float pad[3];
};

template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_add(double x) {
  const int2 w = __builtin_bit_cast(int2, x);
  int2 o;
  o.x = __builtin_amdgcn_update_dpp(0, w.x, CTRL, ROWS, 0xf, false);
  o.y = __builtin_amdgcn_update_dpp(0, w.y, CTRL, ROWS, 0xf, false);
  return x + __builtin_bit_cast(double, o);
}
// inclusive sum over the lanes of a wave
__device__ __forceinline__ double wave_cumsum(double x) {
  x = dpp_add<0x111, 0xf>(x);  // row_shr:1
  x = dpp_add<0x112, 0xf>(x);
  x = dpp_add<0x114, 0xf>(x);
  x = dpp_add<0x118, 0xf>(x);
  x = dpp_add<0x142, 0xa>(x);  // row_bcast:15
  x = dpp_add<0x143, 0xc>(x);  // row_bcast:31
  return x;
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

__device__ __forceinline__ double log2_decay(float g) {
  return (double)(g < -1e5f ? -1e5f : g) * 1.4426950408889634074;
}

// by one wave: lane t holds g of step t (0 past the chunk's last step)
template <int C>
__device__ __forceinline__ double write_decays(Decays<C>& dst, float g) {
  const int l = lane_id();
  const double b = wave_cumsum(l < C ? log2_decay(g) : 0.0);
  const double all = __shfl(b, C - 1);
  if (l < C) {
    dst.b[l] = b;
    dst.up[l] = exp2_fast((float)b);
    dst.dn[l] = exp2_fast((float)(all - b));
    if (l == 0) dst.all = exp2_fast((float)all);
  }
  return all;
}

// ---------------------------------------------------------------------------
// which steps a workgroup runs
// ---------------------------------------------------------------------------
// Sequences are cut into spans of a.span steps. With B equal sequences, span c
// of sequence s is slot s * spans + c. Packed, it is slot cu[s] / span + s + c:
// ceil(len / span) <= (cu[s] + len) / span - cu[s] / span + 1, so no two spans
// share a slot, and the sequence of a slot is the last s whose first slot is
// not behind it. Steps behind the last sequence form one more "sequence" nseg.
struct Span {
  int32_t seq;       // sequence; nseg for the steps behind the last one
  int32_t first;     // first span of the sequence / the span is the last one
  int64_t t0;        // first step, counted from the row of the sequence's batch entry
  int64_t batch;     // batch entry
  int32_t n;         // steps (0: nothing to run)
  bool is_first, is_last;
};

__device__ __forceinline__ int64_t clamp_cu(const LaProblem& a, int i) {
  const int64_t v = a.cu[i];
  return v < 0 ? 0 : (v > a.T ? a.T : v);
}

__device__ __forceinline__ Span find_span(const LaProblem& a, int slot) {
  Span s;
  if (!a.cu) {
    s.seq = slot / a.spans;
    const int c = slot - s.seq * a.spans;
    s.batch = s.seq;
    s.t0 = (int64_t)c * a.span;
    const int64_t left = a.T - s.t0;
    s.n = (int)(left < a.span ? left : a.span);
    s.is_first = c == 0;
    s.is_last = c == a.spans - 1;
    s.first = slot - c;
    return s;
  }
  int lo = 0, hi = a.nseg;  // the last i in [0, nseg] with cu[i] / span + i <= slot
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (clamp_cu(a, mid) / a.span + mid <= slot) lo = mid; else hi = mid - 1;
  }
  const int64_t start = clamp_cu(a, lo), end = lo < a.nseg ? clamp_cu(a, lo + 1) : a.T;
  s.first = (int)(start / a.span) + lo;
  const int64_t c = slot - s.first;
  s.seq = lo;
  s.batch = 0;
  s.t0 = start + c * a.span;
  int64_t left = end - s.t0;
  if (c < 0 || left < 0) left = 0;
  s.n = (int)(left < a.span ? left : a.span);
  s.is_first = c == 0;
  s.is_last = (c + 1) * a.span >= end - start && (s.n > 0 || c == 0);
  return s;
}

}  // namespace la
}  // namespace mscan
