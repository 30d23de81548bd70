"""Python binding of the linear attention operators (see include/mscan.h).

    linear_attention_fwd(q, k, v, g, h0=None, cu_seqlens=None, scale=None, need_ht=True) -> (o, ht)
    linear_attention_bwd(q, k, v, g, do, h0=None, dht=None, ...) -> (dq, dk, dv, dg, dh0)
    linear_attention_step(q, k, v, g, state, slots=None, scale=None) -> o        (state updated in place)
    qk_norm_rope_fwd(q, k, q_weight, k_weight, cos, sin, positions=None, eps=1e-6, interleaved=False) -> (q', k')
    qk_norm_rope_bwd(q, k, q_weight, k_weight, cos, sin, dq', dk', ...) -> (dq, dk, dq_weight, dk_weight)

q, k: [B, T, Hk, Dk]; v: [B, T, H, Dv], H a multiple of Hk; bf16, fp16 or fp32,
any strides with a contiguous last axis and 16-byte aligned rows. g: fp32 log
decays, [B, T, H] or [H]. h0, ht: fp32 [N, H, Dk, Dv] with N the number of
sequences (B, or those of cu_seqlens, which needs B = 1). scale defaults to
Dk ** -0.5. The step takes one token of each sequence: q, k [B, Hk, Dk],
v [B, H, Dv], g [B, H] or [H], against state, fp32 [pool, H, Dk, Dv].
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import MscanError, _check, _in_dtype, _ptr, _segments, _stream_handle, lib


class Attention(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int64), ("T", ctypes.c_int64), ("H", ctypes.c_int32), ("Hk", ctypes.c_int32),
        ("Dk", ctypes.c_int32), ("Dv", ctypes.c_int32), ("cu_seqlens", ctypes.c_void_p), ("nseg", ctypes.c_int32),
        ("scale", ctypes.c_float), ("g_strides", ctypes.c_int64 * 3),
    ]


class NormRope(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int64), ("T", ctypes.c_int64), ("Hq", ctypes.c_int32), ("Hk", ctypes.c_int32),
        ("D", ctypes.c_int32), ("rot", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("eps", ctypes.c_float),
        ("cos", ctypes.c_void_p), ("sin", ctypes.c_void_p), ("table", ctypes.c_int64), ("positions", ctypes.c_void_p),
        ("positions_int64", ctypes.c_int32), ("positions_per_batch", ctypes.c_int32), ("w_dtype", ctypes.c_int32),
    ]


class HeadsArray(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("strides", ctypes.c_int64 * 3)]


def _on(device):
    """Make the tensors' device the current one for a call's launches."""
    if device.index is None or device.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(device)


def _same_device(dev, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != dev:
            raise ValueError(f"{name} is on {t.device}, the queries on {dev}")


def _heads(t, name):
    if t.stride(3) != 1 and t.shape[3] != 1:
        raise ValueError(f"{name}: the last axis must be contiguous")
    unit = 16 // t.element_size()
    # the stride of an axis of one entry is never used
    st = [0 if t.shape[i] == 1 else t.stride(i) for i in range(3)]
    if t.data_ptr() % 16 or st[0] % unit or st[1] % unit or st[2] % unit:
        raise ValueError(f"{name}: rows must be 16-byte aligned (a storage offset and strides of whole 16 bytes)")
    return HeadsArray(t.data_ptr(), (ctypes.c_int64 * 3)(*st))


def _attention(q, k, v, g, cu_seqlens, scale):
    """(problem, dtype, cu_seqlens, number of sequences) of a call, checked."""
    if not q.is_cuda:
        raise ValueError("q must be a GPU tensor")
    dev = q.device
    if q.dim() != 4 or v.dim() != 4 or k.shape != q.shape or v.shape[:2] != q.shape[:2]:
        raise ValueError("q and k must be [B, T, Hk, Dk] and v [B, T, H, Dv]")
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k and v must have the same dtype")
    dt = _in_dtype(q, "q")
    B, T, Hk, Dk = (int(x) for x in q.shape)
    H, Dv = int(v.shape[2]), int(v.shape[3])
    if Hk == 0 or H == 0 or H % Hk:
        raise ValueError(f"the number of value heads ({H}) must be a multiple of the number of key heads ({Hk})")
    for d, n in ((Dk, "Dk"), (Dv, "Dv")):
        if d % 8 or not 8 <= d <= 128:
            raise ValueError(f"{n} must be a multiple of 8 up to 128, got {d}")
    if g.dtype != torch.float32:
        raise ValueError("g (log decays) must be float32")
    if tuple(g.shape) == (H,):
        gs = (0, 0, g.stride(0))
    elif tuple(g.shape) == (B, T, H):
        gs = g.stride()
    else:
        raise ValueError(f"g must be [B, T, H] = {(B, T, H)} or [H], got {tuple(g.shape)}")
    _same_device(dev, k=k, v=v, g=g)
    cu, nseg = _segments(cu_seqlens, dev, T)
    if cu is None:
        nseg = B
    elif B != 1:
        raise ValueError("cu_seqlens needs B = 1 (packed sequences)")
    else:
        _same_device(dev, cu_seqlens=cu)
    prob = Attention(B, T, H, Hk, Dk, Dv, None if cu is None else cu.data_ptr(), nseg,
                     float(Dk ** -0.5 if scale is None else scale), (ctypes.c_int64 * 3)(*gs))
    return prob, dt, cu, nseg


def _states(t, shape, name, dev):
    if t is None:
        return None
    if t.dtype != torch.float32 or t.device != dev or not t.is_contiguous() or t.data_ptr() % 16:
        raise ValueError(f"{name} must be a contiguous, 16-byte aligned fp32 tensor on {dev}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must be [N, H, Dk, Dv] = {shape}, got {tuple(t.shape)}")
    return t


def _space(prob, backward, dev):
    """A workspace of the call's own: torch's allocator keeps it in the stream's
    order, and in a captured graph's own pool."""
    need = lib.linear_attention_workspace_bytes(ctypes.byref(prob), backward)
    if need <= 256:
        return None, 0
    return torch.empty(need, dtype=torch.uint8, device=dev), need


def linear_attention_fwd(q, k, v, g, h0=None, cu_seqlens=None, scale=None, need_ht=True):
    """S_t = e^{g_t} S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t: (o, ht), ht the
    state after each sequence (None without need_ht)."""
    prob, dt, cu, nseg = _attention(q, k, v, g, cu_seqlens, scale)
    dev = q.device
    shape = (nseg, prob.H, prob.Dk, prob.Dv)
    h0 = _states(h0, shape, "h0", dev)
    qh, kh, vh = _heads(q, "q"), _heads(k, "k"), _heads(v, "v")
    o = torch.empty(v.shape, dtype=v.dtype, device=dev)
    ht = torch.empty(shape, dtype=torch.float32, device=dev) if need_ht else None
    if prob.B == 0 or prob.T == 0 or nseg == 0:
        if need_ht:
            ht.zero_() if h0 is None else ht.copy_(h0)
        return o, ht
    with _on(dev):
        ws, n = _space(prob, 0, dev)
        _check("linear_attention_fwd", lib.linear_attention_fwd(
            ctypes.byref(prob), dt, ctypes.byref(qh), ctypes.byref(kh), ctypes.byref(vh), _ptr(g), _ptr(h0), _ptr(o),
            _ptr(ht), _ptr(ws), n, _stream_handle(dev)))
    return o, ht


def linear_attention_bwd(q, k, v, g, do, h0=None, dht=None, cu_seqlens=None, scale=None, need_dg=True, need_dh0=True):
    """Adjoint of linear_attention_fwd for the gradients do of o and dht of ht
    (None: zero): (dq, dk, dv, dg, dh0), dg of g's shape and dh0 in fp32 (None
    when not needed)."""
    prob, dt, cu, nseg = _attention(q, k, v, g, cu_seqlens, scale)
    dev = q.device
    shape = (nseg, prob.H, prob.Dk, prob.Dv)
    h0, dht = _states(h0, shape, "h0", dev), _states(dht, shape, "dht", dev)
    if do.shape != v.shape or do.dtype != v.dtype or do.device != dev:
        raise ValueError("do must have the shape, dtype and device of v")
    qh, kh, vh, oh = _heads(q, "q"), _heads(k, "k"), _heads(v, "v"), _heads(do, "do")
    dq, dk, dv = (torch.empty(x.shape, dtype=x.dtype, device=dev) for x in (q, k, v))
    dg = torch.empty(g.shape, dtype=torch.float32, device=dev) if need_dg else None
    dh0 = torch.empty(shape, dtype=torch.float32, device=dev) if need_dh0 else None
    if prob.B == 0 or prob.T == 0 or nseg == 0:
        if need_dg:
            dg.zero_()
        if need_dh0:
            dh0.zero_() if dht is None else dh0.copy_(dht)
        return dq, dk, dv, dg, dh0
    with _on(dev):
        ws, n = _space(prob, 1, dev)
        _check("linear_attention_bwd", lib.linear_attention_bwd(
            ctypes.byref(prob), dt, ctypes.byref(qh), ctypes.byref(kh), ctypes.byref(vh), _ptr(g), ctypes.byref(oh),
            _ptr(h0), _ptr(dht), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dg), int(g.dim() == 1), _ptr(dh0), _ptr(ws), n,
            _stream_handle(dev)))
    return dq, dk, dv, dg, dh0


def linear_attention_step(q, k, v, g, state, slots=None, scale=None):
    """One step of every sequence, in place on a pool of states: with
    S = state[slots[b]], S = e^{g_b} S + k_b v_b^T and o_b = scale S^T q_b.

    slots: int32 [B] on the GPU, or None (row b has state b). A slot outside
    [0, pool) marks a row of padding, with an output of zero. Rows that share a
    slot are consecutive steps of that sequence, in the order of the batch."""
    if q.dim() != 3 or k.dim() != 3 or v.dim() != 3 or g.dim() not in (1, 2):
        raise ValueError("q and k must be [B, Hk, Dk], v [B, H, Dv] and g [B, H] or [H]")
    prob, dt, _, _ = _attention(q[:, None], k[:, None], v[:, None], g[:, None] if g.dim() == 2 else g, None, scale)
    dev, B = q.device, prob.B
    if state.dim() != 4 or tuple(state.shape[1:]) != (prob.H, prob.Dk, prob.Dv):
        raise ValueError(f"state must be [pool, H, Dk, Dv] with {(prob.H, prob.Dk, prob.Dv)}, got {tuple(state.shape)}")
    pool = int(state.shape[0])
    _states(state, tuple(state.shape), "state", dev)
    if slots is None:
        if B > pool:
            raise ValueError(f"{B} rows without slots need as many states, got {pool}")
    elif slots.dtype != torch.int32 or slots.device != dev or tuple(slots.shape) != (B,) or not slots.is_contiguous():
        raise ValueError(f"slots must be a contiguous int32 tensor [B] on {dev}")
    qh, kh, vh = _heads(q[:, None], "q"), _heads(k[:, None], "k"), _heads(v[:, None], "v")
    o = torch.empty(v.shape, dtype=v.dtype, device=dev)
    if B == 0:
        return o
    if pool == 0:
        return o.zero_()  # every row is padding
    with _on(dev):
        _check("linear_attention_step", lib.linear_attention_step(
            ctypes.byref(prob), dt, ctypes.byref(qh), ctypes.byref(kh), ctypes.byref(vh), _ptr(g), _ptr(slots), pool,
            _ptr(state), _ptr(o), _stream_handle(dev)))
    return o


def _norm_rope(q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved):
    """(problem, dtype) of a norm call, checked."""
    if not q.is_cuda:
        raise ValueError("q must be a GPU tensor")
    dev = q.device
    if q.dim() != 4 or k.dim() != 4 or q.shape[:2] != k.shape[:2] or q.shape[3] != k.shape[3]:
        raise ValueError("q must be [B, T, Hq, D] and k [B, T, Hk, D]")
    if k.dtype != q.dtype:
        raise ValueError("q and k must have the same dtype")
    dt = _in_dtype(q, "q")
    B, T, Hq, D = (int(x) for x in q.shape)
    Hk = int(k.shape[2])
    if D % 8 or not 8 <= D <= 256:
        raise ValueError(f"the head size must be a multiple of 8 up to 256, got {D}")
    wt = 0
    if (q_weight is None) != (k_weight is None):
        raise ValueError("give both weights or neither")
    if q_weight is not None:
        if q_weight.dtype != k_weight.dtype:
            raise ValueError("q_weight and k_weight must have the same dtype")
        wt = _in_dtype(q_weight, "q_weight")
        for w, n in ((q_weight, "q_weight"), (k_weight, "k_weight")):
            if tuple(w.shape) != (D,) or not w.is_contiguous():
                raise ValueError(f"{n} must be a contiguous tensor [D] = {(D,)}, got {tuple(w.shape)}")
    rot, table = 0, 0
    if (cos is None) != (sin is None):
        raise ValueError("give both cos and sin or neither")
    if cos is not None:
        for x, n in ((cos, "cos"), (sin, "sin")):
            if x.dtype != torch.float32 or x.dim() != 2 or not x.is_contiguous() or x.data_ptr() % 16:
                raise ValueError(f"{n} must be a contiguous, 16-byte aligned fp32 tensor [positions, rot / 2]")
        if cos.shape != sin.shape or cos.shape[0] < 1:
            raise ValueError("cos and sin must have one shape, with at least one position")
        table, rot = int(cos.shape[0]), 2 * int(cos.shape[1])
        if rot % 16 or rot > D:
            raise ValueError(f"the rotated entries must be a multiple of 16 up to the head size, got {rot}")
    per_batch = i64 = 0
    if positions is not None:
        if positions.dtype not in (torch.int32, torch.int64) or not positions.is_contiguous():
            raise ValueError("positions must be a contiguous int32 or int64 tensor")
        if tuple(positions.shape) not in ((T,), (B, T)):
            raise ValueError(f"positions must be [T] or [B, T], got {tuple(positions.shape)}")
        per_batch, i64 = int(positions.dim() == 2), int(positions.dtype == torch.int64)
    _same_device(dev, k=k, q_weight=q_weight, k_weight=k_weight, cos=cos, sin=sin, positions=positions)
    return NormRope(B, T, Hq, Hk, D, rot, int(bool(interleaved)), float(eps), _ptr(cos), _ptr(sin), table,
                    _ptr(positions), i64, per_batch, wt), dt


def qk_norm_rope_fwd(q, k, q_weight=None, k_weight=None, cos=None, sin=None, positions=None, eps=1e-6,
                     interleaved=False):
    """RMS norm of every head of q [B, T, Hq, D] and k [B, T, Hk, D], times the
    weights [D], then the rotation of its first 2 * cos.shape[1] entries by the
    row of cos, sin (fp32 [positions, rot / 2]) at the token's position
    (positions: [T] or [B, T], default 0, 1, ..). Pairs are entries (i, i + rot /
    2), or (2i, 2i + 1) when interleaved. No weights: ones; no cos, sin: no
    rotation."""
    prob, dt = _norm_rope(q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved)
    dev = q.device
    qh, kh = _heads(q, "q"), _heads(k, "k")
    yq, yk = torch.empty(q.shape, dtype=q.dtype, device=dev), torch.empty(k.shape, dtype=k.dtype, device=dev)
    if prob.B * prob.T * prob.Hq * prob.Hk == 0:
        if q.numel() or k.numel():
            raise ValueError("q and k both need heads")
        return yq, yk
    with _on(dev):
        _check("qk_norm_rope_fwd", lib.qk_norm_rope_fwd(
            ctypes.byref(prob), dt, ctypes.byref(qh), ctypes.byref(kh), _ptr(q_weight), _ptr(k_weight), _ptr(yq),
            _ptr(yk), _stream_handle(dev)))
    return yq, yk


def qk_norm_rope_bwd(q, k, q_weight, k_weight, cos, sin, dyq, dyk, positions=None, eps=1e-6, interleaved=False,
                     need_dw=True):
    """Adjoint of qk_norm_rope_fwd: (dq, dk, dq_weight, dk_weight), the weights'
    gradients in fp32 (None without weights or need_dw)."""
    prob, dt = _norm_rope(q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved)
    dev = q.device
    for x, d, n in ((q, dyq, "dyq"), (k, dyk, "dyk")):
        if d.shape != x.shape or d.dtype != x.dtype or d.device != dev:
            raise ValueError(f"{n} must have the shape, dtype and device of what it is a gradient of")
    qh, kh, dqh, dkh = _heads(q, "q"), _heads(k, "k"), _heads(dyq, "dyq"), _heads(dyk, "dyk")
    dq, dk = torch.empty(q.shape, dtype=q.dtype, device=dev), torch.empty(k.shape, dtype=k.dtype, device=dev)
    dwq = dwk = None
    if q_weight is not None and need_dw:
        dwq = torch.empty(prob.D, dtype=torch.float32, device=dev)
        dwk = torch.empty(prob.D, dtype=torch.float32, device=dev)
    if prob.B * prob.T * prob.Hq * prob.Hk == 0:
        if q.numel() or k.numel():
            raise ValueError("q and k both need heads")
        return dq, dk, (None if dwq is None else dwq.zero_()), (None if dwk is None else dwk.zero_())
    with _on(dev):
        need = lib.qk_norm_rope_workspace_bytes(ctypes.byref(prob))
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
        _check("qk_norm_rope_bwd", lib.qk_norm_rope_bwd(
            ctypes.byref(prob), dt, ctypes.byref(qh), ctypes.byref(kh), _ptr(q_weight), _ptr(k_weight),
            ctypes.byref(dqh), ctypes.byref(dkh), _ptr(dq), _ptr(dk), _ptr(dwq), _ptr(dwk), _ptr(ws), need,
            _stream_handle(dev)))
    return dq, dk, dwq, dwk
