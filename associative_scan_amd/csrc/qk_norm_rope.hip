// RMS norm of queries and keys for each head, with the position rotation.
//
//   n = x w / sqrt(mean(x^2) + eps)  over the D entries of a head, then the first
//   `rot` entries of n are rotated in pairs by (cos, sin) of the token's position.
//
// Every element is read once and written once: the kernels are bound by HBM. A
// row (one head of one token) is spread over L = 8, 16 or 32 lanes of 8 elements,
// two units of 4. A rotated lane holds both halves of its four pairs, (4 c + i,
// rot / 2 + 4 c + i), so the rotation needs nothing from other lanes and a pair
// shares its angle. A lane's 16 bytes of a 16-bit type are one access: of the
// first half by even lanes, of the second by odd ones, and two neighbours then
// exchange a unit. A lane group takes several heads of a token and reads the
// token's angles once. Loads and stores are streaming: they pass the caches by for
// inputs that come back.
// Measured in bf16, D = 128: forward, 32767 tokens of 16 + 4 heads 61 us (5.6 TB/s;
// with two accesses of 8 bytes 76), forward and backward, 32768 tokens of 12 + 12
// heads 189 us (5.5 TB/s; a copy reaches 5.35); a decoding step of 7 tokens 4.4 us,
// its three dependent trips to memory.
#include "la_device.hpp"
#include "qk_norm_rope.hpp"

namespace mscan {
namespace la {

template <class T>
struct Four {
  typedef T type __attribute__((ext_vector_type(4)));
};
template <class T>
__device__ __forceinline__ f4v wide(T v) {
  return __builtin_convertvector(v, f4v);
}
__device__ __forceinline__ f4v load_weight(const void* w, int dtype, int at) {
  f4v v = {1.f, 1.f, 1.f, 1.f};
  if (!w) return v;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = dtype == 0 ? ((const float*)w)[at + i]
                      : dtype == 1 ? (float)((const __bf16*)w)[at + i] : (float)((const _Float16*)w)[at + i];
  return v;
}

template <int CTRL>
__device__ __forceinline__ float dpp_plus(float x) {
  return x + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xf, 0xf, false));
}
// sum over the L lanes of a row, to all of them
template <int L>
__device__ __forceinline__ float row_sum(float x) {
  x = dpp_plus<0xb1>(x);   // quad_perm 1,0,3,2
  x = dpp_plus<0x4e>(x);   // quad_perm 2,3,0,1
  x = dpp_plus<0x141>(x);  // row_half_mirror: the other quad of 8
  if constexpr (L >= 16) x = dpp_plus<0x140>(x);  // row_mirror: the other half of 16
  if constexpr (L >= 32) {
    const uint32_t w = __builtin_bit_cast(uint32_t, x);
    const auto y = __builtin_amdgcn_permlane16_swap(w, w, false, false);
    x = __builtin_bit_cast(float, (uint32_t)y[0]) + __builtin_bit_cast(float, (uint32_t)y[1]);
  }
  return x;
}
__device__ __forceinline__ float dot4(f4v a, f4v b) { return (a[0] * b[0] + a[1] * b[1]) + (a[2] * b[2] + a[3] * b[3]); }

// A lane's two units of a row, and the angles of its pairs (1 and 0 where it has
// none). Interleaved pairs lie inside a unit.
struct Place {
  int a, b;
  int at;         // the 8 elements that the lane itself reads and writes, of a 16-bit type
  bool even, odd; // place in a pair of lanes that exchange a unit
  bool in, rotated;
};
template <bool PAIRS>
__device__ __forceinline__ Place place_of(const NormProblem& p, int lane) {
  Place q;
  q.in = lane * 8 < p.D;
  q.rotated = lane * 8 < p.rot;
  q.a = q.rotated && !PAIRS ? lane * 4 : lane * 8;
  q.b = q.rotated && !PAIRS ? p.rot / 2 + lane * 4 : lane * 8 + 4;
  q.even = q.rotated && !PAIRS && !(lane & 1);
  q.odd = q.rotated && !PAIRS && (lane & 1);
  q.at = q.odd ? p.rot / 2 + (lane - 1) * 4 : q.a;
  return q;
}
// An even lane's second unit and the next one's first change places.
__device__ __forceinline__ u4v exchange(u4v x, const Place& at) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t mine = at.odd ? x[i] : x[2 + i];
    const uint32_t other = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)mine, 0xb1, 0xf, 0xf, false);  // lane ^ 1
    x[i] = at.odd ? other : x[i];
    x[2 + i] = at.even ? other : x[2 + i];
  }
  return x;
}
struct Angles {
  f4v c, s;
};
__device__ __forceinline__ int64_t position_of(const NormProblem& p, int64_t b, int64_t t) {
  if (!p.positions) return t;
  const int64_t at = p.per_batch ? b * p.T + t : t;
  return p.positions64 ? ((const int64_t*)p.positions)[at] : (int64_t)((const int32_t*)p.positions)[at];
}
__device__ __forceinline__ Angles load_angles(const NormProblem& p, int64_t pos, int lane) {
  pos = pos < 0 ? 0 : (pos >= p.table ? p.table - 1 : pos);
  const int64_t at = pos * (p.rot / 2) + lane * 4;
  return Angles{*(const f4v*)(p.cos + at), *(const f4v*)(p.sin + at)};
}
// (a, b) turned by the angles (sign -1: back)
template <bool PAIRS>
__device__ __forceinline__ void rotate(f4v& a, f4v& b, const Angles& x, float sign) {
  const f4v s = x.s * sign;
  if constexpr (PAIRS) {
    const f4v u = a, v = b;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      a[2 * i] = u[2 * i] * x.c[i] - u[2 * i + 1] * s[i];
      a[2 * i + 1] = u[2 * i + 1] * x.c[i] + u[2 * i] * s[i];
      b[2 * i] = v[2 * i] * x.c[2 + i] - v[2 * i + 1] * s[2 + i];
      b[2 * i + 1] = v[2 * i + 1] * x.c[2 + i] + v[2 * i] * s[2 + i];
    }
  } else {
    const f4v u = a;
    a = u * x.c - b * s;
    b = b * x.c + u * s;
  }
}

// Which rows a lane group runs: HP heads of one token at a time.
template <int L, int HP>
struct Rows {
  int64_t b, t;
  int h0, nh;  // first head; heads, 0 past the end
  __device__ __forceinline__ Rows(const NormProblem& p, int heads, uint32_t group) {  // at most 2^27 groups
    const uint32_t per = (uint32_t)(heads + HP - 1) / HP, token = group / per, batch = token / (uint32_t)p.T;
    h0 = (int)(group - token * per) * HP;
    b = batch;
    t = token - batch * (uint32_t)p.T;
    nh = b < p.B ? (heads - h0 < HP ? heads - h0 : HP) : 0;
  }
};

// A lane's part of HP heads, as it lies in memory.
template <class TIn, int HP>
struct Heads4 {
  typedef typename Four<TIn>::type t4;
  static constexpr int W = sizeof(TIn) == 4 ? 2 : 1;  // 16-byte accesses
  u4v w[HP][W];
  __device__ __forceinline__ void load(const Heads& x, int64_t b, int64_t t, int h0, int nh, const Place& at) {
    const TIn* p = (const TIn*)x.p + b * x.sb + t * x.st + h0 * x.sh;
#pragma unroll
    for (int j = 0; j < HP; ++j) {
#pragma unroll
      for (int i = 0; i < W; ++i) w[j][i] = u4v{0, 0, 0, 0};
      if (at.in && j < nh) {
        w[j][0] = __builtin_nontemporal_load((const u4v*)(p + j * x.sh + (W == 2 ? at.a : at.at)));
        if constexpr (W == 2) w[j][1] = __builtin_nontemporal_load((const u4v*)(p + j * x.sh + at.b));
      }
    }
  }
  // the units at at.a and at.b; by all lanes of a wave
  __device__ __forceinline__ void get(int j, const Place& at, f4v& u, f4v& v) const {
    if constexpr (W == 2) {
      u = __builtin_bit_cast(f4v, w[j][0]);
      v = __builtin_bit_cast(f4v, w[j][1]);
    } else {
      const u4v x = exchange(w[j][0], at);
      u = wide(__builtin_bit_cast(t4, u2v{x[0], x[1]}));
      v = wide(__builtin_bit_cast(t4, u2v{x[2], x[3]}));
    }
  }
  static __device__ __forceinline__ void put(TIn* p, const Place& at, bool live, f4v a, f4v b) {
    if constexpr (W == 2) {
      if (!live) return;
      __builtin_nontemporal_store(a, (f4v*)(p + at.a));
      __builtin_nontemporal_store(b, (f4v*)(p + at.b));
    } else {
      const u2v x = __builtin_bit_cast(u2v, __builtin_convertvector(a, t4));
      const u2v y = __builtin_bit_cast(u2v, __builtin_convertvector(b, t4));
      const u4v z = exchange(u4v{x[0], x[1], y[0], y[1]}, at);
      if (live) __builtin_nontemporal_store(z, (u4v*)(p + at.at));
    }
  }
};

// A workgroup goes over its share of the rows, the next rows and their angles on
// their way while it works on the last ones: a position, its angles and the rows
// are three trips to memory, of which a workgroup that ran one set of rows would
// overlap none.
template <class TIn, int L, int HP, bool PAIRS>
__global__ __launch_bounds__(256) void k_norm_fwd(const NormProblem p, const NormSide q, const NormSide k,
                                                  unsigned qblocks) {
  constexpr int G = 256 / L;
  const bool isq = blockIdx.x < qblocks;
  const NormSide& x = isq ? q : k;
  const unsigned blk = isq ? blockIdx.x : blockIdx.x - qblocks, nblk = isq ? qblocks : gridDim.x - qblocks;
  const int lane = threadIdx.x % L;
  const Place at = place_of<PAIRS>(p, lane);
  const f4v zero = {0.f, 0.f, 0.f, 0.f}, one = {1.f, 1.f, 1.f, 1.f};
  const uint32_t groups = (uint32_t)(p.B * p.T * ((x.heads + HP - 1) / HP));
  const uint32_t first = blk * G + threadIdx.x / L, step = nblk * G;
  const f4v wu = at.in ? load_weight(x.w, p.wtype, at.a) : zero, wv = at.in ? load_weight(x.w, p.wtype, at.b) : zero;
  const float inv = 1.f / (float)p.D;
  const auto rows_of = [&](uint32_t g) { return Rows<L, HP>(p, x.heads, g < groups ? g : groups - 1); };
  Rows<L, HP> r = rows_of(first);
  Heads4<TIn, HP> in;
  Angles ang{one, zero};
  in.load(x.x, r.b, r.t, r.h0, r.nh, at);
  int64_t pos = 0;
  if (at.rotated) {
    ang = load_angles(p, position_of(p, r.b, r.t), lane);
    const Rows<L, HP> n = rows_of(first + step);
    pos = position_of(p, n.b, n.t);
  }
  for (uint32_t g = first; g < groups; g += step) {
    const Rows<L, HP> next = rows_of(g + step);
    const Heads4<TIn, HP> now = in;
    const Angles turn = ang;
    if (g + step < groups) {
      in.load(x.x, next.b, next.t, next.h0, next.nh, at);
      if (at.rotated) {
        ang = load_angles(p, pos, lane);
        const Rows<L, HP> n = rows_of(g + 2 * step);
        pos = position_of(p, n.b, n.t);
      }
    }
    TIn* yp = (TIn*)x.y + ((r.b * p.T + r.t) * x.heads + r.h0) * p.D;
#pragma unroll
    for (int j = 0; j < HP; ++j) {
      f4v u, v;
      now.get(j, at, u, v);
      const float rs = rsqrtf(row_sum<L>(dot4(u, u) + dot4(v, v)) * inv + p.eps);
      f4v a = u * rs * wu, b = v * rs * wv;
      rotate<PAIRS>(a, b, turn, 1.f);
      Heads4<TIn, HP>::put(yp + (int64_t)j * p.D, at, at.in && j < r.nh, a, b);
    }
    r = next;
  }
}

// dn = R^T dy, dw = sum dn x_hat, dx = r (dn w - x_hat mean(dn w x_hat)) with
// x_hat = x r, r = 1 / sqrt(mean(x^2) + eps). A workgroup adds dw up over all
// its rows in registers and writes one partial sum, in a fixed order.
template <class TIn, int L, int HP, bool PAIRS>
__global__ __launch_bounds__(256) void k_norm_bwd(const NormProblem p, const NormSide q, const NormSide k,
                                                  unsigned qblocks, float* partial) {
  constexpr int G = 256 / L;
  __shared__ float sums[G][L * 8 + 1];
  const bool isq = blockIdx.x < qblocks;
  const NormSide& x = isq ? q : k;
  const unsigned blk = isq ? blockIdx.x : blockIdx.x - qblocks, nblk = isq ? qblocks : gridDim.x - qblocks;
  const int lane = threadIdx.x % L;
  const Place at = place_of<PAIRS>(p, lane);
  const f4v zero = {0.f, 0.f, 0.f, 0.f}, one = {1.f, 1.f, 1.f, 1.f};
  const f4v wu = at.in ? load_weight(x.w, p.wtype, at.a) : zero, wv = at.in ? load_weight(x.w, p.wtype, at.b) : zero;
  const float inv = 1.f / (float)p.D;
  const uint32_t groups = (uint32_t)(p.B * p.T * ((x.heads + HP - 1) / HP));
  const uint32_t first = blk * G + threadIdx.x / L, step = nblk * G;
  const auto rows_of = [&](uint32_t g) { return Rows<L, HP>(p, x.heads, g < groups ? g : groups - 1); };
  Rows<L, HP> r = rows_of(first);
  Heads4<TIn, HP> in, din;
  Angles ang{one, zero};
  in.load(x.x, r.b, r.t, r.h0, r.nh, at);
  din.load(x.dy, r.b, r.t, r.h0, r.nh, at);
  int64_t pos = 0;
  if (at.rotated) {
    ang = load_angles(p, position_of(p, r.b, r.t), lane);
    const Rows<L, HP> n = rows_of(first + step);
    pos = position_of(p, n.b, n.t);
  }
  f4v du = zero, dv = zero;
  for (uint32_t g = first; g < groups; g += step) {
    const Rows<L, HP> next = rows_of(g + step);
    const Heads4<TIn, HP> now = in, dnow = din;
    const Angles turn = ang;
    if (g + step < groups) {
      in.load(x.x, next.b, next.t, next.h0, next.nh, at);
      din.load(x.dy, next.b, next.t, next.h0, next.nh, at);
      if (at.rotated) {
        ang = load_angles(p, pos, lane);
        const Rows<L, HP> n = rows_of(g + 2 * step);
        pos = position_of(p, n.b, n.t);
      }
    }
    TIn* yp = (TIn*)x.y + ((r.b * p.T + r.t) * x.heads + r.h0) * p.D;
#pragma unroll
    for (int j = 0; j < HP; ++j) {
      f4v a, b, u, v;
      dnow.get(j, at, a, b);
      rotate<PAIRS>(a, b, turn, -1.f);
      now.get(j, at, u, v);
      const float rs = rsqrtf(row_sum<L>(dot4(u, u) + dot4(v, v)) * inv + p.eps);
      const f4v hu = u * rs, hv = v * rs, tu = a * wu, tv = b * wv;
      const float m = row_sum<L>(dot4(tu, hu) + dot4(tv, hv)) * inv;
      if (j < r.nh) {
        du += a * hu;
        dv += b * hv;
      }
      Heads4<TIn, HP>::put(yp + (int64_t)j * p.D, at, at.in && j < r.nh, (tu - hu * m) * rs, (tv - hv * m) * rs);
    }
    r = next;
  }
  if (at.in) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      sums[threadIdx.x / L][at.a + i] = du[i];
      sums[threadIdx.x / L][at.b + i] = dv[i];
    }
  }
  __syncthreads();
  if ((int)threadIdx.x < p.D) {
    float s = 0.f;
#pragma unroll
    for (int g = 0; g < G; ++g) s += sums[g][threadIdx.x];
    partial[(int64_t)blockIdx.x * p.D + threadIdx.x] = s;
  }
}

// The partial sums of dw: q's blocks, then k's.
__global__ __launch_bounds__(256) void k_norm_weights(const float* partial, int D, unsigned qblocks, unsigned kblocks,
                                                      float* dwq, float* dwk) {
  __shared__ float sums[32][9];
  const int parts = D / 8;
  const bool isq = (int)blockIdx.x < parts;
  float* out = isq ? dwq : dwk;
  if (!out) return;
  const int c = threadIdx.x & 7, r = threadIdx.x >> 3, col = (int)(blockIdx.x % parts) * 8 + c;
  const unsigned first = isq ? 0 : qblocks, n = isq ? qblocks : kblocks;
  float s = 0.f;
#pragma unroll 8
  for (unsigned i = r; i < n; i += 32) s += partial[(int64_t)(first + i) * D + col];
  sums[r][c] = s;
  __syncthreads();
  if (threadIdx.x < 8) {
    float t = 0.f;
    for (int i = 0; i < 32; ++i) t += sums[i][threadIdx.x];
    out[col] = t;
  }
}

static int norm_lanes(int D) { return D <= 64 ? 8 : D <= 128 ? 16 : 32; }

// Workgroups for q's and k's rows: all that there are, or `most` shared out by
// their number.
static void norm_blocks(const NormProblem& p, int Hq, int Hk, int hp, int64_t most, unsigned& qb, unsigned& kb) {
  const int L = norm_lanes(p.D);
  const int64_t nq = (p.B * p.T * ((Hq + hp - 1) / hp) * L + 255) / 256;
  const int64_t nk = (p.B * p.T * ((Hk + hp - 1) / hp) * L + 255) / 256;
  if (nq + nk <= most) {
    qb = (unsigned)nq;
    kb = (unsigned)nk;
    return;
  }
  const int64_t n = most * nq / (nq + nk);
  qb = (unsigned)(n < 1 ? 1 : n > most - 1 ? most - 1 : n);
  kb = (unsigned)(most - qb);
}
constexpr int kBwdHeads = 2;
// The backward's partial sums of dw are one row per workgroup: few enough to stay
// small, enough to fill the card.
void norm_bwd_blocks(const NormProblem& p, int Hq, int Hk, unsigned& qb, unsigned& kb) {
  norm_blocks(p, Hq, Hk, kBwdHeads, 2048, qb, kb);
}

template <class TIn, int L, int HP, bool PAIRS>
static hipError_t fwd_heads(const NormProblem& p, const NormSide& q, const NormSide& k, hipStream_t st) {
  unsigned qb, kb;
  norm_blocks(p, q.heads, k.heads, HP, 4096, qb, kb);
  hipLaunchKernelGGL((k_norm_fwd<TIn, L, HP, PAIRS>), dim3(qb + kb), dim3(256), 0, st, p, q, k, qb);
  return hipGetLastError();
}
template <class TIn, int L, bool PAIRS>
static hipError_t fwd_lanes(const NormProblem& p, const NormSide& q, const NormSide& k, hipStream_t st) {
  // four heads per lane group once there is a wave for every SIMD of the card
  // (32767 tokens of 16 + 4 heads: 62 us, with two 67 us; below, one gives the most waves)
  return p.B * p.T * (q.heads + k.heads) * L >= (int64_t)1024 * 64 * 4 ? fwd_heads<TIn, L, 4, PAIRS>(p, q, k, st)
                                                                       : fwd_heads<TIn, L, 1, PAIRS>(p, q, k, st);
}

template <class TIn, int L, bool PAIRS>
static hipError_t bwd_lanes(const NormProblem& p, const NormSide& q, const NormSide& k, float* dwq, float* dwk,
                            float* partial, hipStream_t st) {
  unsigned qb, kb;
  norm_bwd_blocks(p, q.heads, k.heads, qb, kb);
  hipLaunchKernelGGL((k_norm_bwd<TIn, L, kBwdHeads, PAIRS>), dim3(qb + kb), dim3(256), 0, st, p, q, k, qb, partial);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || (!dwq && !dwk)) return e;
  hipLaunchKernelGGL(k_norm_weights, dim3(2 * p.D / 8), dim3(256), 0, st, partial, p.D, qb, kb, dwq, dwk);
  return hipGetLastError();
}

template <class TIn, bool PAIRS>
static hipError_t norm_pairs(const NormProblem& p, const NormSide& q, const NormSide& k, bool bwd, float* dwq,
                             float* dwk, float* partial, hipStream_t st) {
  const int L = norm_lanes(p.D);
  if (!bwd)
    return L == 8 ? fwd_lanes<TIn, 8, PAIRS>(p, q, k, st)
                  : L == 16 ? fwd_lanes<TIn, 16, PAIRS>(p, q, k, st) : fwd_lanes<TIn, 32, PAIRS>(p, q, k, st);
  return L == 8 ? bwd_lanes<TIn, 8, PAIRS>(p, q, k, dwq, dwk, partial, st)
                : L == 16 ? bwd_lanes<TIn, 16, PAIRS>(p, q, k, dwq, dwk, partial, st)
                          : bwd_lanes<TIn, 32, PAIRS>(p, q, k, dwq, dwk, partial, st);
}

template <class TIn>
static hipError_t norm_type(const NormProblem& p, const NormSide& q, const NormSide& k, bool bwd, float* dwq,
                            float* dwk, float* partial, hipStream_t st) {
  return p.interleaved ? norm_pairs<TIn, true>(p, q, k, bwd, dwq, dwk, partial, st)
                       : norm_pairs<TIn, false>(p, q, k, bwd, dwq, dwk, partial, st);
}

hipError_t launch_norm(const NormProblem& p, const NormSide& q, const NormSide& k, int dtype, bool bwd, float* dwq,
                       float* dwk, float* partial, hipStream_t st) {
  if (dtype == 0) return norm_type<float>(p, q, k, bwd, dwq, dwk, partial, st);
  if (dtype == 1) return norm_type<__bf16>(p, q, k, bwd, dwq, dwk, partial, st);
  return norm_type<_Float16>(p, q, k, bwd, dwq, dwk, partial, st);
}

}  // namespace la
}  // namespace mscan
