// RMS norm of queries and keys for each head, with the position rotation.
//
//   n = x w / sqrt(mean(x^2) + eps)  over the D entries of a head, then the first
//   `rot` entries of n are rotated in pairs by (cos, sin) of the token's position.
//
// Every element is read once and written once: the kernels are bound by HBM. A
// row (one head of one token) is spread over L = 8, 16 or 32 lanes of 8 elements,
// so a wave reads whole rows as 16-byte units; the pair of an element lies in
// another lane's unit (or, interleaved, in its own). A lane group takes several
// heads of a token and reads the token's angles once.
#include "la_device.hpp"
#include "qk_norm_rope.hpp"

namespace mscan {
namespace la {

template <class T>
__device__ __forceinline__ f8v load8(const T* p) {
  if constexpr (sizeof(T) == 4) {
    const f4v a = __builtin_nontemporal_load((const f4v*)p), b = __builtin_nontemporal_load((const f4v*)(p + 4));
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  } else {
    typedef T t8 __attribute__((ext_vector_type(8)));
    return __builtin_convertvector(__builtin_nontemporal_load((const t8*)p), f8v);
  }
}
template <class T>
__device__ __forceinline__ void store8(T* p, f8v v) {
  if constexpr (sizeof(T) == 4) {
    __builtin_nontemporal_store(__builtin_shufflevector(v, v, 0, 1, 2, 3), (f4v*)p);
    __builtin_nontemporal_store(__builtin_shufflevector(v, v, 4, 5, 6, 7), (f4v*)(p + 4));
  } else {
    typedef T t8 __attribute__((ext_vector_type(8)));
    __builtin_nontemporal_store(__builtin_convertvector(v, t8), (t8*)p);
  }
}
__device__ __forceinline__ f8v load_weight(const void* w, int dtype, int at) {
  f8v v = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
  if (!w) return v;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    v[i] = dtype == 0 ? ((const float*)w)[at + i]
                      : dtype == 1 ? (float)((const __bf16*)w)[at + i] : (float)((const _Float16*)w)[at + i];
  return v;
}

// sum over the L lanes of a row
template <int L>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int m = 1; m < L; m <<= 1) x += __shfl_xor(x, m);
  return x;
}
__device__ __forceinline__ float dot8(f8v a, f8v b) {
  return ((a[0] * b[0] + a[1] * b[1]) + (a[2] * b[2] + a[3] * b[3])) +
         ((a[4] * b[4] + a[5] * b[5]) + (a[6] * b[6] + a[7] * b[7]));
}

// The angles that a lane's 8 elements need: c[i], and s[i] with the sign that
// its pair's value enters with (the transposed rotation flips it).
struct Angles {
  f8v c, s;
};
template <bool PAIRS>
__device__ __forceinline__ Angles load_angles(const NormProblem& p, int64_t b, int64_t t, int unit) {
  Angles a;
  a.c = f8v{1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
  a.s = f8v{0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (unit * 8 >= p.rot) return a;
  int64_t pos = t;
  if (p.positions) {
    const int64_t at = p.per_batch ? b * p.T + t : t;
    pos = p.positions64 ? ((const int64_t*)p.positions)[at] : (int64_t)((const int32_t*)p.positions)[at];
  }
  pos = pos < 0 ? 0 : (pos >= p.table ? p.table - 1 : pos);
  const int half = p.rot / 2;
  if constexpr (PAIRS) {
    const f4v c = *(const f4v*)(p.cos + pos * half + unit * 4), s = *(const f4v*)(p.sin + pos * half + unit * 4);
    a.c = __builtin_shufflevector(c, c, 0, 0, 1, 1, 2, 2, 3, 3);
    a.s = __builtin_shufflevector(s, s, 0, 0, 1, 1, 2, 2, 3, 3);
    a.s[0] = -a.s[0];
    a.s[2] = -a.s[2];
    a.s[4] = -a.s[4];
    a.s[6] = -a.s[6];
  } else {
    const bool low = unit * 8 < half;
    const int at = low ? unit * 8 : unit * 8 - half;
    const f4v* c = (const f4v*)(p.cos + pos * half + at);  // shared by the token's heads: not streamed
    const f4v* s = (const f4v*)(p.sin + pos * half + at);
    a.c = __builtin_shufflevector(c[0], c[1], 0, 1, 2, 3, 4, 5, 6, 7);
    a.s = __builtin_shufflevector(s[0], s[1], 0, 1, 2, 3, 4, 5, 6, 7);
    if (low) a.s = -a.s;
  }
  return a;
}
// v c + pair(v) s; `other`: the lane that holds the pairs
template <bool PAIRS>
__device__ __forceinline__ f8v rotate(f8v v, const Angles& a, float sign, int other) {
  f8v w;
  if constexpr (PAIRS) {
    w = __builtin_shufflevector(v, v, 1, 0, 3, 2, 5, 4, 7, 6);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = __shfl(v[i], other);
  }
  return v * a.c + w * (a.s * sign);
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

template <class TIn, int L, int HP, bool PAIRS>
__global__ __launch_bounds__(256) void k_norm_fwd(const NormProblem p, const NormSide q, const NormSide k,
                                                  unsigned qblocks) {
  const bool isq = blockIdx.x < qblocks;
  const NormSide& x = isq ? q : k;
  const unsigned blk = isq ? blockIdx.x : blockIdx.x - qblocks;
  const int lane = threadIdx.x % L;
  const Rows<L, HP> r(p, x.heads, blk * (256 / L) + threadIdx.x / L);
  const bool in = lane * 8 < p.D;
  const TIn* xp = (const TIn*)x.x.p + r.b * x.x.sb + r.t * x.x.st + r.h0 * x.x.sh + lane * 8;
  f8v v[HP];
#pragma unroll
  for (int j = 0; j < HP; ++j) {
    v[j] = f8v{0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (in && j < r.nh) v[j] = load8<TIn>(xp + j * x.x.sh);
  }
  f8v w = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  Angles a{w, w};
  if (in && r.nh) {
    a = load_angles<PAIRS>(p, r.b, r.t, lane);
    w = load_weight(x.w, p.wtype, lane * 8);
  }
  const int half = p.rot / 16, other = (threadIdx.x & 63) + (lane < half ? half : lane < 2 * half ? -half : 0);
  TIn* yp = (TIn*)x.y + ((r.b * p.T + r.t) * x.heads + r.h0) * p.D + lane * 8;
  const float inv = 1.f / (float)p.D;
#pragma unroll
  for (int j = 0; j < HP; ++j) {
    const float rs = 1.f / sqrtf(row_sum<L>(dot8(v[j], v[j])) * inv + p.eps);
    const f8v y = rotate<PAIRS>(v[j] * rs * w, a, 1.f, other);
    if (in && j < r.nh) store8<TIn>(yp + (int64_t)j * p.D, y);
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
  const bool in = lane * 8 < p.D;
  const f8v zero = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  const f8v w = in ? load_weight(x.w, p.wtype, lane * 8) : zero;
  const int half = p.rot / 16, other = (threadIdx.x & 63) + (lane < half ? half : lane < 2 * half ? -half : 0);
  const float inv = 1.f / (float)p.D;
  const int64_t groups = p.B * p.T * ((x.heads + HP - 1) / HP);
  f8v dw = zero;
  for (int64_t g0 = (int64_t)blk * G; g0 < groups; g0 += (int64_t)nblk * G) {
    const Rows<L, HP> r(p, x.heads, (uint32_t)g0 + threadIdx.x / L);
    const TIn* xp = (const TIn*)x.x.p + r.b * x.x.sb + r.t * x.x.st + r.h0 * x.x.sh + lane * 8;
    const TIn* dp = (const TIn*)x.dy.p + r.b * x.dy.sb + r.t * x.dy.st + r.h0 * x.dy.sh + lane * 8;
    f8v v[HP], d[HP];
#pragma unroll
    for (int j = 0; j < HP; ++j) {
      v[j] = zero;
      d[j] = zero;
      if (in && j < r.nh) {
        v[j] = load8<TIn>(xp + j * x.x.sh);
        d[j] = load8<TIn>(dp + j * x.dy.sh);
      }
    }
    Angles a{zero, zero};
    if (in && r.nh) a = load_angles<PAIRS>(p, r.b, r.t, lane);
    TIn* yp = (TIn*)x.y + ((r.b * p.T + r.t) * x.heads + r.h0) * p.D + lane * 8;
#pragma unroll
    for (int j = 0; j < HP; ++j) {
      const f8v dn = rotate<PAIRS>(d[j], a, -1.f, other);
      const float rs = 1.f / sqrtf(row_sum<L>(dot8(v[j], v[j])) * inv + p.eps);
      const f8v hat = v[j] * rs, t = dn * w;
      const float m = row_sum<L>(dot8(t, hat)) * inv;
      if (j < r.nh) dw += dn * hat;
      if (in && j < r.nh) store8<TIn>(yp + (int64_t)j * p.D, (t - hat * m) * rs);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) sums[threadIdx.x / L][lane * 8 + i] = dw[i];
  __syncthreads();
  if ((int)threadIdx.x < p.D) {
    float s = 0.f;
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

template <int HP>
static int64_t norm_groups(const NormProblem& p, int heads) {
  return p.B * p.T * ((heads + HP - 1) / HP);
}

template <class TIn, int L, bool PAIRS>
static hipError_t fwd_lanes(const NormProblem& p, const NormSide& q, const NormSide& k, hipStream_t st) {
  // several heads per lane group once there is a wave for every SIMD of the card
  constexpr int HP = 4;
  if (p.B * p.T * (q.heads + k.heads) * L >= (int64_t)1024 * 64 * HP) {
    const unsigned qb = (unsigned)((norm_groups<HP>(p, q.heads) * L + 255) / 256);
    const unsigned kb = (unsigned)((norm_groups<HP>(p, k.heads) * L + 255) / 256);
    hipLaunchKernelGGL((k_norm_fwd<TIn, L, HP, PAIRS>), dim3(qb + kb), dim3(256), 0, st, p, q, k, qb);
  } else {
    const unsigned qb = (unsigned)((norm_groups<1>(p, q.heads) * L + 255) / 256);
    const unsigned kb = (unsigned)((norm_groups<1>(p, k.heads) * L + 255) / 256);
    hipLaunchKernelGGL((k_norm_fwd<TIn, L, 1, PAIRS>), dim3(qb + kb), dim3(256), 0, st, p, q, k, qb);
  }
  return hipGetLastError();
}

// Workgroups of the backward pass, q's and k's: enough to fill the card, few
// enough that the partial sums of dw stay small.
void norm_bwd_blocks(const NormProblem& p, int Hq, int Hk, unsigned& qb, unsigned& kb) {
  const int L = norm_lanes(p.D);
  const int64_t nq = (norm_groups<2>(p, Hq) * L + 255) / 256, nk = (norm_groups<2>(p, Hk) * L + 255) / 256;
  const int64_t most = 2048;
  if (nq + nk <= most) {
    qb = (unsigned)nq;
    kb = (unsigned)nk;
    return;
  }
  qb = (unsigned)(most * nq / (nq + nk));
  if (qb < 1) qb = 1;
  if (qb > most - 1) qb = (unsigned)(most - 1);
  kb = (unsigned)(most - qb);
}

template <class TIn, int L, bool PAIRS>
static hipError_t bwd_lanes(const NormProblem& p, const NormSide& q, const NormSide& k, float* dwq, float* dwk,
                            float* partial, hipStream_t st) {
  unsigned qb, kb;
  norm_bwd_blocks(p, q.heads, k.heads, qb, kb);
  hipLaunchKernelGGL((k_norm_bwd<TIn, L, 2, PAIRS>), dim3(qb + kb), dim3(256), 0, st, p, q, k, qb, partial);
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
