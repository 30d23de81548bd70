"""Python binding of the linear attention operators (see include/mscan.h).

    linear_attention_fwd(q, k, v, g, h0=None, cu_seqlens=None, scale=None, need_ht=True) -> (o, ht)

q, k: [B, T, Hk, Dk]; v: [B, T, H, Dv], H a multiple of Hk; bf16, fp16 or fp32,
any strides with a contiguous last axis and 16-byte aligned rows. g: fp32 log
decays, [B, T, H] or [H]. h0, ht: fp32 [N, H, Dk, Dv] with N the number of
sequences (B, or those of cu_seqlens, which needs B = 1). scale defaults to
Dk ** -0.5.
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
