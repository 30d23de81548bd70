// C ABI of the linear attention operators: host-side validation, workspace
// sizing and dispatch. Every check runs before any HIP call.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "la_launch.hpp"
#include "mscan.h"
#include "mscan_launch.hpp"

namespace {

using mscan::la::Heads;
using mscan::la::LaProblem;

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
mscan_status hip_status(hipError_t e) { return (mscan_status)mscan::status_of_hip(e); }

constexpr int64_t kMaxHeadDim = 128;
// A launch counts its work-items in 32 bits, and a workgroup has up to 512.
constexpr int64_t kMaxBlocks = (int64_t)1 << 22;

mscan_status check(const mscan_attention* p) {
  if (!p) return MSCAN_ERR_INVALID;
  if (p->B < 1 || p->T < 1 || p->T > (int64_t)INT32_MAX || p->H < 1 || p->Hk < 1 || p->H % p->Hk) return MSCAN_ERR_INVALID;
  if (p->nseg < 1) return MSCAN_ERR_INVALID;
  if (p->cu_seqlens ? (p->B != 1 || ((uintptr_t)p->cu_seqlens & 3u)) : (p->nseg != p->B)) return MSCAN_ERR_INVALID;
  if (p->Dk < 1 || p->Dv < 1) return MSCAN_ERR_INVALID;
  if (p->Dk % 8 || p->Dv % 8 || p->Dk > kMaxHeadDim || p->Dv > kMaxHeadDim) return MSCAN_ERR_UNSUPPORTED;
  if (p->B > kMaxBlocks || p->H > kMaxBlocks || p->nseg > kMaxBlocks) return MSCAN_ERR_UNSUPPORTED;
  return MSCAN_OK;
}

LaProblem problem(const mscan_attention* p, const float* g, bool backward) {
  LaProblem r{};
  r.B = p->B;
  r.T = p->T;
  r.H = p->H;
  r.Hk = p->Hk;
  r.Dk = p->Dk;
  r.Dv = p->Dv;
  r.cu = p->cu_seqlens;
  r.nseg = p->nseg;
  r.scale = p->scale;
  r.g = g;
  r.gsb = p->g_strides[0];
  r.gst = p->g_strides[1];
  r.gsh = p->g_strides[2];
  mscan::la::plan(r, backward);
  return r;
}

mscan_status check_blocks(const LaProblem& r) {
  // workgroups of the main passes and of k_join
  const int64_t joins = ((int64_t)r.Dk * r.Dv / 4 + 255) / 256 * r.H * r.nseg;
  return r.slots * (int64_t)r.H > kMaxBlocks || joins > kMaxBlocks * 2 ? MSCAN_ERR_UNSUPPORTED : MSCAN_OK;
}

// The array's strides in the kernels' form; heads of it are shared by `share`.
mscan_status heads(const mscan_heads* x, int dtype, int share, int d, Heads& out) {
  if (!x || !x->p || !aligned16(x->p)) return MSCAN_ERR_INVALID;
  const int64_t unit = dtype == MSCAN_F32 ? 4 : 8;
  for (int i = 0; i < 3; ++i)
    if (x->strides[i] < 0 || x->strides[i] % unit) return MSCAN_ERR_INVALID;
  out = Heads{x->p, x->strides[0], x->strides[1], x->strides[2], share, d};
  return MSCAN_OK;
}

size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

struct FwdSpace {
  size_t states = 0, totals = 0, bytes = 0;
};
FwdSpace fwd_space(const LaProblem& r) {
  FwdSpace w;
  if (r.T <= r.span) return w;
  w.states = 0;
  w.totals = up256((size_t)r.slots * r.H * r.Dk * r.Dv * 4);
  w.bytes = w.totals + up256((size_t)r.slots * r.H * 4);
  return w;
}

}  // namespace

extern "C" {

size_t linear_attention_workspace_bytes(const mscan_attention* prob, int backward) {
  if (check(prob) != MSCAN_OK || backward < 0 || backward > 1) return 0;
  const LaProblem r = problem(prob, nullptr, backward == 1);
  if (check_blocks(r) != MSCAN_OK) return 0;
  return fwd_space(r).bytes + 256;
}

mscan_status linear_attention_fwd(const mscan_attention* prob, int dtype, const mscan_heads* q, const mscan_heads* k,
                                  const mscan_heads* v, const float* g, const float* h0, void* o, float* ht, void* ws,
                                  size_t ws_bytes, void* stream) {
  mscan_status s = check(prob);
  if (s != MSCAN_OK) return s;
  if (dtype != MSCAN_F32 && dtype != MSCAN_BF16 && dtype != MSCAN_F16) return MSCAN_ERR_UNSUPPORTED;
  mscan::la::FwdArgs a{};
  a.pr = problem(prob, g, false);
  const int share = prob->H / prob->Hk;
  if ((s = heads(q, dtype, share, prob->Dk, a.q)) != MSCAN_OK) return s;
  if ((s = heads(k, dtype, share, prob->Dk, a.k)) != MSCAN_OK) return s;
  if ((s = heads(v, dtype, 1, prob->Dv, a.v)) != MSCAN_OK) return s;
  if (!g || ((uintptr_t)g & 3u) || !o || !aligned16(o)) return MSCAN_ERR_INVALID;
  if (!aligned16(h0) || !aligned16(ht)) return MSCAN_ERR_INVALID;
  if ((s = check_blocks(a.pr)) != MSCAN_OK) return s;
  const FwdSpace w = fwd_space(a.pr);
  if (w.bytes && (!ws || !aligned16(ws) || ws_bytes < w.bytes)) return MSCAN_ERR_WORKSPACE;
  a.o = o;
  a.h0 = h0;
  a.ht = ht;
  a.states = w.bytes ? (float*)((char*)ws + w.states) : nullptr;
  a.totals = w.bytes ? (float*)((char*)ws + w.totals) : nullptr;
  return hip_status(mscan::la::launch_fwd(a, dtype, (hipStream_t)stream));
}

}  // extern "C"
