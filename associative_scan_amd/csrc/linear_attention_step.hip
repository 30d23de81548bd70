// Linear attention, one step of each sequence against a pool of states.
//
// S = e^g S + k v^T in place and o = scale S^T q. The state is read and written
// once (8 Dk Dv bytes per head) and everything else is small, so the step is
// bound by HBM; one workgroup per head and COLS columns of its state, every
// thread holding its part in registers between the read and the write. A row of
// COLS fp32 columns is read as whole 16-byte units, 128 bytes at a time, past the
// caches: a pool of states is larger than they are. 251 sequences of 12 heads,
// 128 x 128: 395 MB in 79 us, 5.0 TB/s (a copy reaches 5.35). One sequence: 4.4 us,
// the latency of a launch and of two trips to memory.
#include "la_device.hpp"

namespace mscan {
namespace la {

template <class TIn>
__device__ __forceinline__ float widen(TIn x) {
  return (float)x;
}

// Sequence of batch row b whose state slot it owns: -1 when the slot is out of
// range, or when an earlier row of the batch has the same slot (that row then
// runs this one's step after its own, in the order of the batch).
__device__ __forceinline__ bool slot_taken_before(const int32_t* slots, int b, int32_t slot) {
  bool hit = false;
  for (int i = (int)threadIdx.x; i < b; i += (int)blockDim.x) hit |= slots[i] == slot;
  return __syncthreads_or(hit);
}
// The next row after b with the same slot, or n.
__device__ __forceinline__ int next_with(const int32_t* slots, int b, int n, int32_t slot, int* lds) {
  __syncthreads();
  if (threadIdx.x == 0) *lds = n;
  __syncthreads();
  int first = n;
  for (int i = b + 1 + (int)threadIdx.x; i < n; i += (int)blockDim.x)
    if (slots[i] == slot) {
      first = i;
      break;
    }
  if (first < n) atomicMin(lds, first);
  __syncthreads();
  return *lds;
}

// COLS columns by DK rows on 256 threads: 16-byte units of a row by rows.
template <class TIn, int DK, int COLS>
__global__ __launch_bounds__(256) void k_attn_step(const StepArgs a) {
  constexpr int UN = COLS / 4;       // units of a row
  constexpr int RW = 256 / UN;       // rows at a time
  constexpr int N = DK / RW;         // rows of a thread
  static_assert(DK % RW == 0, "rows");
  __shared__ float qs[DK], ks[DK];
  __shared__ __align__(16) f4v part[4][UN];
  __shared__ int next;
  const int tid = threadIdx.x, u = tid % UN, r0 = tid / UN;
  const int parts = (a.Dv + COLS - 1) / COLS;
  const int part_i = blockIdx.x % parts, h = blockIdx.x / parts % a.H, b0 = blockIdx.x / parts / a.H;
  const int col = part_i * COLS + u * 4;
  const bool in = col < a.Dv;
  const int32_t slot = a.slots ? a.slots[b0] : b0;
  const bool live = slot >= 0 && slot < a.pool;
  // a row's own inputs, one entry of q and k to a thread
  float qv, kv, gv;
  f4v v;
  const auto fetch = [&](int b) {
    const TIn* qp = (const TIn*)a.q.p + (int64_t)b * a.q.sb + (int64_t)(h / a.q.share) * a.q.sh;
    const TIn* kp = (const TIn*)a.k.p + (int64_t)b * a.k.sb + (int64_t)(h / a.k.share) * a.k.sh;
    const TIn* vp = (const TIn*)a.v.p + (int64_t)b * a.v.sb + (int64_t)h * a.v.sh;
    qv = tid < a.Dk ? widen<TIn>(qp[tid]) * a.scale : 0.f;
    kv = tid < a.Dk ? widen<TIn>(kp[tid]) : 0.f;
    gv = a.g[(int64_t)b * a.gsb + (int64_t)h * a.gsh];
    v = f4v{0.f, 0.f, 0.f, 0.f};
    if (in)
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = widen<TIn>(vp[col + j]);
  };
  fetch(b0);
  float* sp = a.state + ((int64_t)(live ? slot : 0) * a.H + h) * a.Dk * a.Dv + col;
  f4v S[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int row = r0 + i * RW;
    S[i] = f4v{0.f, 0.f, 0.f, 0.f};
    if (live && in && row < a.Dk) S[i] = __builtin_nontemporal_load((const f4v*)(sp + (int64_t)row * a.Dv));
  }
  // the loads above are in flight; what is read of a state another row owns is dropped
  if (a.slots && live && slot_taken_before(a.slots, b0, slot)) return;
  for (int b = b0; b < a.B;) {
    TIn* op = (TIn*)a.o + ((int64_t)b * a.H + h) * a.Dv;
    if (!live) {  // no state: a zero output
      if (r0 == 0 && in)
        for (int j = 0; j < 4; ++j) op[col + j] = (TIn)0.f;
      return;
    }
    if (tid < DK) {
      qs[tid] = qv;
      ks[tid] = kv;
    }
    const float decay = exp2_fast((float)log2_decay(gv));
    __syncthreads();
    f4v o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int row = r0 + i * RW;
      S[i] = S[i] * decay + v * ks[row];
      o += S[i] * qs[row];
    }
    // rows of a wave, then waves
#pragma unroll
    for (int m = UN; m < 64; m <<= 1)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] += __shfl_xor(o[j], m);
    if ((tid & 63) < UN) part[tid >> 6][u] = o;
    __syncthreads();
    if (tid < UN && in) {
      o = part[0][u] + part[1][u] + part[2][u] + part[3][u];
#pragma unroll
      for (int j = 0; j < 4; ++j) op[col + j] = (TIn)o[j];
    }
    b = a.slots ? next_with(a.slots, b, a.B, slot, &next) : a.B;
    if (b < a.B) fetch(b);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int row = r0 + i * RW;
    if (in && row < a.Dk) __builtin_nontemporal_store(S[i], (f4v*)(sp + (int64_t)row * a.Dv));
  }
}

template <class TIn>
static hipError_t step_type(const StepArgs& a, hipStream_t st) {
  const unsigned heads = (unsigned)((int64_t)a.B * a.H);
  if (a.Dk <= 64)
    hipLaunchKernelGGL((k_attn_step<TIn, 64, 32>), dim3(heads * ((a.Dv + 31) / 32)), dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL((k_attn_step<TIn, 128, 32>), dim3(heads * ((a.Dv + 31) / 32)), dim3(256), 0, st, a);
  return hipGetLastError();
}

hipError_t launch_step(const StepArgs& a, int dtype, hipStream_t st) {
  if (dtype == 0) return step_type<float>(a, st);
  if (dtype == 1) return step_type<__bf16>(a, st);
  return step_type<_Float16>(a, st);
}

}  // namespace la
}  // namespace mscan
