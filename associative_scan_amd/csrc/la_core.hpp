// One chunk of linear attention on one workgroup (see la_device.hpp for the
// form), and the passes that both directions share: the states between spans.
#pragma once

#include "la_device.hpp"

namespace mscan {
namespace la {

// Chunk sizes: 64 steps for 16-bit math; 32 for fp32 math, whose tiles are
// twice as wide and whose products within a chunk cost sixteen times as much.
template <class TM>
constexpr int kChunk = sizeof(TM) == 2 ? 64 : 32;
// Pieces of the masked scores: bf16 alone would be as coarse as a bf16 output.
template <class TM>
constexpr int kPiecesP = sizeof(TM) == 2 ? 2 : 1;
// Pieces of the injected values and of the state as an operand. Three keep
// fp32 states and gate gradients to fp32; two are enough for 16-bit outputs.
template <class TM>
constexpr int kPiecesZ = sizeof(TM) == 2 ? 3 : 1;
template <class TM>
constexpr int kPiecesX = sizeof(TM) == 2 ? 2 : 1;
template <class TM>
constexpr int kPiecesXExact = sizeof(TM) == 2 ? 3 : 1;

__device__ __forceinline__ int acc_row(int r) { return ((r >> 2) << 3) + ((lane_id() >> 5) << 2) + (r & 3); }

// One 16 x 16 tile of the scores x_r . y_c, transposed: rows ct*16 + 4 (l / 16)
// + i, i < 4, are steps c, column rt*16 + (l & 15) is step r.
template <class TM, int DX>
__device__ __forceinline__ f4v score_tile(const TM* X, const TM* Y, int rt, int ct, int l) {
  f4v acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int k0 = 0; k0 < DX; k0 += 32)
    acc = Math<TM>::mma16(row_frag16<TM, DX>(Y, ct * 16, k0, l), row_frag16<TM, DX>(X, rt * 16, k0, l), acc);
  return acc;
}
// The decays of such a tile: e^{b_r - b_c} for c <= r (REV: e^{b_c - b_r} for
// c >= r), zero elsewhere.
template <int C, bool REV>
__device__ __forceinline__ f4v decay_tile(const Decays<C>& d, int rt, int ct, int l) {
  const int r = rt * 16 + (l & 15), c0 = ct * 16 + ((l >> 4) << 2);
  const double br = d.b[r];
  f4v o;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = c0 + i;
    const double bc = d.b[c];
    const float e = exp2_fast((float)(REV ? bc - br : br - bc));
    o[i] = (REV ? c >= r : c <= r) ? e : 0.f;
  }
  return o;
}
// Masked scores into P [NP][C][C] (row r, column c).
template <class TM, int C, int NP>
__device__ __forceinline__ void put_tile(TM* P, f4v val, int rt, int ct, int l) {
  const int r = rt * 16 + (l & 15), u = ct * 4 + (l >> 4);
  typename Math<TM>::Unit piece[NP];
  split4<TM, NP>(val, piece);
#pragma unroll
  for (int p = 0; p < NP; ++p) *(typename Math<TM>::Unit*)(P + p * C * C + unit_at<TM, C>(r, u)) = piece[p];
}
// The 16 x 16 tiles that a product over P reads: for every 32 rows, the columns
// up to their end (REV: from their start). Tile i of kTiles<C>.
template <int C>
constexpr int kTiles = C == 64 ? 12 : 4;
template <int C, bool REV>
__device__ __forceinline__ void tile_of(int i, int& rt, int& ct) {
  if constexpr (C == 32) {
    rt = i >> 1;
    ct = i & 1;
  } else {
    // rows 0-31 (REV: 32-63) have 2 tiles a row, the others 4
    const bool small = i < 4;
    rt = small ? i >> 1 : 2 + ((i - 4) >> 2);
    ct = small ? i & 1 : (i - 4) & 3;
    if (REV) {
      rt = 3 - rt;
      ct = 3 - ct;
    }
  }
}
template <class TM, int C, int DX, int NP, bool REV>
__device__ __forceinline__ void scores(const TM* X, const TM* Y, TM* P, const Decays<C>& d, float scale, int wave,
                                       int nwaves) {
  const int l = fresh_lane();
  for (int i = wave; i < kTiles<C>; i += nwaves) {
    int rt, ct;
    tile_of<C, REV>(i, rt, ct);
    const f4v dec = decay_tile<C, REV>(d, rt, ct, l);
    f4v acc = score_tile<TM, DX>(X, Y, rt, ct, l);
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] = dec[e] != 0.f ? acc[e] * (dec[e] * scale) : 0.f;
    put_tile<TM, C, NP>(P, acc, rt, ct, l);
  }
}

// Registers 8 s .. 8 s + 7 of the state's tiles are rows 16 s .. 16 s + 15, as
// an operand's contraction axis wants them.
template <int NT>
__device__ __forceinline__ f8v state8(const f16v (&S)[NT], int s) {
  const f16v& t = S[s >> 1];
  return (s & 1) ? __builtin_shufflevector(t, t, 8, 9, 10, 11, 12, 13, 14, 15)
                 : __builtin_shufflevector(t, t, 0, 1, 2, 3, 4, 5, 6, 7);
}

// acc[rt] = rows of X times the state
template <class TM, int C, int DX, int NS>
__device__ __forceinline__ void from_state(const TM* X, const f16v (&S)[DX / 32], f16v (&acc)[C / 32]) {
#pragma unroll
  for (int rt = 0; rt < C / 32; ++rt)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[rt][r] = 0.f;
  const int l = fresh_lane();
#pragma unroll
  for (int s = 0; s < DX / 16; ++s) {
    step_fence();
    typename Math<TM>::Frag piece[NS];
    split8<TM, NS>(state8<DX / 32>(S, s), piece);
#pragma unroll
    for (int rt = 0; rt < C / 32; ++rt) {
      const typename Math<TM>::Frag x = row_frag32<TM, DX>(X, rt * 32, s * 16, l);
#pragma unroll
      for (int p = 0; p < NS; ++p) acc[rt] = Math<TM>::mma32(x, piece[p], acc[rt]);
    }
  }
}
// rows of acc times f[row] * s
template <int C>
__device__ __forceinline__ void scale_rows(f16v (&acc)[C / 32], const float* f, float s) {
  const int h4 = (fresh_lane() >> 5) << 2;
#pragma unroll
  for (int rt = 0; rt < C / 32; ++rt)
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const f4v w = *(const f4v*)(f + rt * 32 + a * 8 + h4);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[rt][a * 4 + i] *= w[i] * s;
    }
}
template <int NT>
__device__ __forceinline__ void scale_state(f16v (&S)[NT], float f) {
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int r = 0; r < 16; ++r) S[t][r] *= f;
}
// S += Y^T (f z) for one 16-step js; z: the wave's 32 columns of those steps
template <class TM, int DX, int NS>
__device__ __forceinline__ void into_state(const TM* Y, typename Math<TM>::Frag z, const float* f, float s, int js,
                                           int l, f16v (&S)[DX / 32]) {
  const int h = l >> 5;
  const f4v fa = *(const f4v*)(f + js * 16 + 4 * h), fb = *(const f4v*)(f + js * 16 + 8 + 4 * h);
  f8v w = Math<TM>::widen(z);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[i] *= fa[i] * s;
    w[4 + i] *= fb[i] * s;
  }
  typename Math<TM>::Frag piece[NS];
  split8<TM, NS>(w, piece);
#pragma unroll
  for (int t = 0; t < DX / 32; ++t) {
    const typename Math<TM>::Frag y = col_frag32<TM, DX>(Y, js * 16, t * 32, l);
#pragma unroll
    for (int p = 0; p < NS; ++p) S[t] = Math<TM>::mma32(y, piece[p], S[t]);
  }
}
// acc += P Z, and S = e^{b_C} S + Y^T (f Z), sharing the reads of Z
template <class TM, int C, int DX, int DZ, int NP, int NS, bool REV>
__device__ __forceinline__ void within_chunk(const TM* Y, const TM* Z, const TM* P, const Decays<C>& d, float sz,
                                             int z0, f16v (&S)[DX / 32], f16v (&acc)[C / 32]) {
  scale_state<DX / 32>(S, d.all);
  const int l = fresh_lane();
#pragma unroll
  for (int js = 0; js < C / 16; ++js) {
    step_fence();
    const typename Math<TM>::Frag z = col_frag32<TM, DZ>(Z, js * 16, z0, l);
#pragma unroll
    for (int rt = 0; rt < C / 32; ++rt) {
      if (REV ? js * 16 < rt * 32 : js * 16 >= rt * 32 + 32) continue;
#pragma unroll
      for (int p = 0; p < NP; ++p)
        acc[rt] = Math<TM>::mma32(row_frag32<TM, C>(P + p * C * C, rt * 32, js * 16, l), z, acc[rt]);
    }
    into_state<TM, DX, NS>(Y, z, REV ? d.up : d.dn, sz, js, l, S);
  }
}

// The wave's 32 columns of a state in memory: element (x, z) of the wave's
// view is at x * ldx + z * ldz, x < dx, z < dz (dx, dz multiples of 8).
template <int DX>
__device__ __forceinline__ void load_state(f16v (&S)[DX / 32], const float* p, int ldx, int ldz, int dx, int dz,
                                           int z0) {
  const int l = fresh_lane(), z = z0 + (l & 31), r0 = (l >> 5) << 2;
  const int n = p && z < dz ? dx : 0;
  p += (int64_t)r0 * ldx + (int64_t)z * ldz;
#pragma unroll
  for (int t = 0; t < DX / 32; ++t)
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const bool in = t * 32 + a * 8 < n;
#pragma unroll
      for (int i = 0; i < 4; ++i) S[t][a * 4 + i] = in ? p[(int64_t)(t * 32 + a * 8 + i) * ldx] : 0.f;
    }
}
template <int DX>
__device__ __forceinline__ void store_state(const f16v (&S)[DX / 32], float* p, int ldx, int ldz, int dx, int dz,
                                            int z0) {
  const int l = fresh_lane(), z = z0 + (l & 31), r0 = (l >> 5) << 2;
  const int n = z < dz ? dx : 0;
  p += (int64_t)r0 * ldx + (int64_t)z * ldz;
#pragma unroll
  for (int t = 0; t < DX / 32; ++t)
#pragma unroll
    for (int a = 0; a < 4; ++a)
      if (t * 32 + a * 8 < n) {
#pragma unroll
        for (int i = 0; i < 4; ++i) p[(int64_t)(t * 32 + a * 8 + i) * ldx] = S[t][a * 4 + i];
      }
}

// The same for ldx = 1: the wave's view is the transpose of the memory's rows.
template <int DX>
__device__ __forceinline__ void load_state_t(f16v (&S)[DX / 32], const float* p, int ldz, int dx, int dz, int z0) {
  const int l = fresh_lane(), z = z0 + (l & 31), r0 = (l >> 5) << 2;
  const int n = p && z < dz ? dx : 0;
  p += r0 + (int64_t)z * ldz;
#pragma unroll
  for (int t = 0; t < DX / 32; ++t)
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      f4v v = {0.f, 0.f, 0.f, 0.f};
      if (t * 32 + a * 8 < n) v = *(const f4v*)(p + t * 32 + a * 8);
#pragma unroll
      for (int i = 0; i < 4; ++i) S[t][a * 4 + i] = v[i];
    }
}

template <int CTRL>
__device__ __forceinline__ float ror_add(float x) {
  return x + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xf, 0xf, false));
}
__device__ __forceinline__ float sum16(float x) {  // over the 16 lanes of a DPP row, to all of them
  return ror_add<0x121>(ror_add<0x122>(ror_add<0x124>(ror_add<0x128>(x))));
}
// Sums over the wave's 32 columns of acc times the rows of a tile, to dst[C].
template <class TM, int C, int D>
__device__ __forceinline__ void row_dots(const f16v (&acc)[C / 32], const TM* tile, int z0, float* dst) {
  const int l = fresh_lane(), z = z0 + (l & 31), h4 = (l >> 5) << 2;
  constexpr int N = C / 4;  // values of a lane, halved by the exchange between DPP rows
  float w[C / 2];
#pragma unroll
  for (int i = 0; i < C / 2; ++i) {
    const int row = (i >> 4) * 32 + (((i & 15) >> 2) << 3) + h4 + (i & 3);
    w[i] = acc[i >> 4][i & 15] * (float)tile[unit_at<TM, D>(row, z >> 2) + (z & 3)];
  }
  float mine = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    // the first DPP row of a pair sums value i, the second value i + N
    const auto x = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, w[i]),
                                                    __builtin_bit_cast(uint32_t, w[i + N]), false, false);
    const float v = sum16(__builtin_bit_cast(float, (uint32_t)x[0]) + __builtin_bit_cast(float, (uint32_t)x[1]));
    mine = (l & 15) == i ? v : mine;
  }
  const int i = (l & 15) + ((l >> 4) & 1) * N;
  if ((l & 15) < N) dst[(i >> 4) * 32 + (((i & 15) >> 2) << 3) + h4 + (i & 3)] = mine;
}

// Rows of an output, [n][H][d] from out (stride st), the wave's 32 columns.
template <class TOut, int C>
__device__ __forceinline__ void store_rows(const f16v (&acc)[C / 32], TOut* out, int64_t st, int n, int d, int z0) {
  const int l = fresh_lane(), z = z0 + (l & 31), r0 = (l >> 5) << 2;
  if (z >= d) return;
  TOut* p = out + r0 * st + z;
#pragma unroll
  for (int rt = 0; rt < C / 32; ++rt)
#pragma unroll
    for (int a = 0; a < 4; ++a) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (rt * 32 + a * 8 + i + r0 < n) *p = (TOut)acc[rt][a * 4 + i];
        p += st;
      }
      p += 4 * st;
    }
}

template <class TIn>
__device__ __forceinline__ const TIn* head_base(const Heads& x, int64_t batch, int64_t t, int h) {
  return (const TIn*)x.p + batch * x.sb + t * x.st + (int64_t)(h / x.share) * x.sh;
}
__device__ __forceinline__ const float* gate_base(const LaProblem& p, int64_t batch, int64_t t, int h) {
  return p.g + batch * p.gsb + t * p.gst + (int64_t)h * p.gsh;
}
// g of step t0 + l of n, 0 past the end
__device__ __forceinline__ float load_gate(const float* g, int64_t st, int t0, int n) {
  const int t = t0 + lane_id();
  return t < n ? g[(int64_t)t * st] : 0.f;
}

// Decay over a span and the state it adds, from a zero state: REV runs the
// adjoint's recurrence. Not needed for the span that ends a sequence (REV: that
// starts it), whose state nothing reads.
template <class TIn, class TM, int DX, int NW, bool REV>
__global__ __launch_bounds__(NW * 64, 2) void k_span_states(const LaProblem pr, const Heads y, const Heads z, float sz,
                                                         float* states, float* totals) {
  constexpr int C = kChunk<TM>, DZ = NW * 32, NT = NW * 64;
  __shared__ __align__(16) TM Y[C * DX];
  __shared__ __align__(16) TM Z[C * DZ];
  __shared__ __align__(16) Decays<C> dec;
  const int tid = threadIdx.x, wave = tid >> 6, z0 = wave * 32;
  const int h = blockIdx.x % pr.H, slot = blockIdx.x / pr.H;
  const Span sp = find_span(pr, slot);
  if (sp.seq >= (pr.cu ? pr.nseg : (int)pr.B) || sp.n == 0 || (REV ? sp.is_first : sp.is_last)) return;
  const TIn* yp = head_base<TIn>(y, sp.batch, sp.t0, h);
  const TIn* zp = head_base<TIn>(z, sp.batch, sp.t0, h);
  const float* gp = gate_base(pr, sp.batch, sp.t0, h);
  f16v S[DX / 32];
#pragma unroll
  for (int t = 0; t < DX / 32; ++t)
#pragma unroll
    for (int r = 0; r < 16; ++r) S[t][r] = 0.f;
  const int nc = (sp.n + C - 1) / C;
  TileRegs<TIn, C, DX, NT> ry;
  TileRegs<TIn, C, DZ, NT> rz;
  float rg = 0.f;
  double total = 0.0;
  auto fetch = [&](int i) {
    const int c = REV ? nc - 1 - i : i, t = c * C;
    ry.load(yp + (int64_t)t * y.st, y.st, y.d, sp.n - t, tid);
    rz.load(zp + (int64_t)t * z.st, z.st, z.d, sp.n - t, tid);
    if (wave == 0) rg = load_gate(gp, pr.gst, t, sp.n);
  };
  fetch(0);
  for (int i = 0; i < nc; ++i) {
    ry.store(Y, tid);
    rz.store(Z, tid);
    if (wave == 0) total += write_decays<C>(dec, rg);
    __syncthreads();
    if (i + 1 < nc) fetch(i + 1);
    scale_state<DX / 32>(S, dec.all);
    const int l = fresh_lane();
#pragma unroll
    for (int js = 0; js < C / 16; ++js) {
      step_fence();
      into_state<TM, DX, kPiecesZ<TM>>(Y, col_frag32<TM, DZ>(Z, js * 16, z0, l), REV ? dec.up : dec.dn, sz, js, l, S);
    }
    __syncthreads();
  }
  store_state<DX>(S, states + ((int64_t)slot * pr.H + h) * pr.Dk * pr.Dv, pr.Dv, 1, pr.Dk, pr.Dv, z0);
  if (tid == 0) totals[(int64_t)slot * pr.H + h] = exp2_fast((float)total);
}

}  // namespace la
}  // namespace mscan
