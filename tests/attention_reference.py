"""Linear attention in 64 bits, step by step on the CPU, with the magnitudes that
its rounding errors go by: every result comes with the same sum over absolute
values, so a bound on an error is a factor times that magnitude."""
import numpy as np


def _segments(B, T, cu):
    """(batch entry, first step, end) of every sequence."""
    if cu is None:
        return [(b, 0, T) for b in range(B)]
    return [(0, int(a), int(e)) for a, e in zip(cu[:-1], cu[1:])]


def forward(q, k, v, g, h0=None, cu=None, scale=1.0):
    """o, ht and their magnitudes. q, k [B, T, Hk, Dk], v [B, T, H, Dv], g [B, T, H] or [H]."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    B, T, H = v.shape[:3]
    r = H // q.shape[2]
    q, k = np.repeat(q, r, 2), np.repeat(k, r, 2)
    a = np.exp(np.broadcast_to(np.asarray(g, np.float64), (B, T, H)))
    segs = _segments(B, T, cu)
    o, om = np.zeros(v.shape), np.zeros(v.shape)
    shape = (len(segs), H, q.shape[3], v.shape[3])
    ht = np.zeros(shape) if h0 is None else np.asarray(h0, np.float64).copy()
    hm = np.abs(ht)
    for n, (b, s, e) in enumerate(segs):
        for t in range(s, e):
            d = a[b, t][:, None, None]
            kv = k[b, t][:, :, None] * v[b, t][:, None, :]
            ht[n] = d * ht[n] + kv
            hm[n] = d * hm[n] + np.abs(kv)
            o[b, t] = scale * np.einsum("hk,hkv->hv", q[b, t], ht[n])
            om[b, t] = scale * np.einsum("hk,hkv->hv", np.abs(q[b, t]), hm[n])
    return (o, om), (ht, hm)


def backward(q, k, v, g, do, h0=None, dht=None, cu=None, scale=1.0):
    """((dq, its magnitude), (dk, ..), (dv, ..), (dg, ..), (dh0, ..)); dg is [B, T, H]
    whatever g's shape."""
    q, k, v, do = (np.asarray(x, np.float64) for x in (q, k, v, do))
    B, T, H = v.shape[:3]
    Hk = q.shape[2]
    r = H // Hk
    q, k = np.repeat(q, r, 2), np.repeat(k, r, 2)
    a = np.exp(np.broadcast_to(np.asarray(g, np.float64), (B, T, H)))
    segs = _segments(B, T, cu)
    shape = (len(segs), H, q.shape[3], v.shape[3])
    out = {n: [np.zeros(x), np.zeros(x)] for n, x in
           (("dq", q.shape), ("dk", k.shape), ("dv", v.shape), ("dg", (B, T, H)), ("dh0", shape))}
    for n, (b, s, e) in enumerate(segs):
        S = np.zeros(shape[1:]) if h0 is None else np.asarray(h0[n], np.float64).copy()
        Sm = np.abs(S)
        before = []
        for t in range(s, e):
            before.append((S, Sm))
            d = a[b, t][:, None, None]
            kv = k[b, t][:, :, None] * v[b, t][:, None, :]
            S, Sm = d * S + kv, d * Sm + np.abs(kv)
            out["dq"][0][b, t] = scale * np.einsum("hkv,hv->hk", S, do[b, t])
            out["dq"][1][b, t] = scale * np.einsum("hkv,hv->hk", Sm, np.abs(do[b, t]))
        L = np.zeros(shape[1:]) if dht is None else np.asarray(dht[n], np.float64).copy()
        Lm = np.abs(L)
        for t in range(e - 1, s - 1, -1):
            x = scale * q[b, t][:, :, None] * do[b, t][:, None, :]
            L, Lm = L + x, Lm + np.abs(x)
            out["dk"][0][b, t] = np.einsum("hkv,hv->hk", L, v[b, t])
            out["dk"][1][b, t] = np.einsum("hkv,hv->hk", Lm, np.abs(v[b, t]))
            out["dv"][0][b, t] = np.einsum("hkv,hk->hv", L, k[b, t])
            out["dv"][1][b, t] = np.einsum("hkv,hk->hv", Lm, np.abs(k[b, t]))
            d = a[b, t][:, None, None]
            S, Sm = before.pop()
            out["dg"][0][b, t] = (L * d * S).sum((1, 2))
            out["dg"][1][b, t] = (Lm * d * Sm).sum((1, 2))
            L, Lm = d * L, d * Lm
        out["dh0"][0][n], out["dh0"][1][n] = L, Lm
    for x in ("dq", "dk"):
        out[x] = [y.reshape(B, T, Hk, r, -1).sum(3) for y in out[x]]
    return tuple(tuple(out[x]) for x in ("dq", "dk", "dv", "dg", "dh0"))
