"""The linear attention and query/key norm operators: the calls that are measured,
and the same results from elementary torch operations.

Operators (``op`` of a case):
    prompt  linear attention over whole sequences: outputs and final states
    train   the same with its backward pass: outputs and all gradients
    step    one token per sequence against a pool of states, updated in place
    norm    per-head RMS norm of queries and keys with the position rotation
    norm_train  the same with its backward pass
"""
import math

import torch

own = False

CHUNK = 64  # steps per block of the plain chunked form


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    attn = dict(Hk=0, packed=0, gate="token")
    return [
        # a first short turn of one conversation: latency
        dict(attn, name="prompt short", op="prompt", B=1, T=37, H=8, Dk=64, Dv=64, dtype="bf16"),
        # prompts of a served batch
        dict(attn, name="prompt batch", op="prompt", B=8, T=4096, H=12, Dk=128, Dv=128, dtype="bf16"),
        # one very long document, few heads, a fixed decay per head: the time axis has to be split
        dict(attn, name="prompt long", op="prompt", B=1, T=65536, H=12, Dk=128, Dv=128, dtype="bf16", gate="head"),
        # packed prompts of ragged lengths
        dict(attn, name="prompt packed", op="prompt", B=1, T=16381, H=16, Dk=128, Dv=128, dtype="bf16", packed=23),
        # a training step's layer
        dict(attn, name="train batch", op="train", B=8, T=4096, H=12, Dk=128, Dv=128, dtype="bf16"),
        # a training layer whose queries and keys are shared by all heads, packed documents, half precision
        dict(attn, name="train shared packed", op="train", B=1, T=8191, H=16, Hk=2, Dk=128, Dv=64, dtype="fp16",
             packed=9),
        # a small model in full precision, odd sizes
        dict(attn, name="train fp32 odd", op="train", B=3, T=333, H=5, Dk=48, Dv=80, dtype="fp32"),
        # decoding for one user, and for a full server
        dict(name="step one", op="step", B=1, slots=4, H=12, Hk=0, Dk=128, Dv=128, dtype="bf16", gate="token"),
        dict(name="step server", op="step", B=251, slots=300, H=12, Hk=0, Dk=128, Dv=128, dtype="bf16", gate="token"),
        # queries and keys of a few decoded tokens, of a long prompt, and of a training step
        dict(name="norm decode", op="norm", B=7, T=1, H=12, Hk=12, D=128, rot=128, far=65536, dtype="bf16"),
        dict(name="norm prompt", op="norm", B=1, T=32767, H=16, Hk=4, D=128, rot=64, far=65536, dtype="bf16"),
        dict(name="norm train", op="norm_train", B=8, T=4096, H=12, Hk=12, D=128, rot=128, far=65536, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "train", "train", "step", "norm", "norm_train"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp16", "fp32"])
    if op in ("norm", "norm_train"):
        D = rng.choice([64, 80, 128, 128, 192, 256])
        B, T = rng.choice([1, 2, 5]), _log(rng, 1, 6000)
        return dict(op=op, B=B, T=T, H=rng.choice([5, 8, 12, 16]), Hk=rng.choice([1, 2, 4, 8]), D=D,
                    rot=rng.choice([d for d in (16, 32, 64, 128, D) if d <= D and d % 16 == 0]), far=65536, dtype=dtype)
    Dk, Dv = rng.choice([(128, 128), (128, 128), (64, 64), (128, 64), (64, 128), (96, 112), (40, 72)])
    H = rng.choice([3, 8, 12, 16])
    Hk = rng.choice([0, 0, 0, 1])
    gate = rng.choice(["token", "token", "head"])
    if op == "step":
        B = _log(rng, 1, 200)
        return dict(op=op, B=B, slots=B + rng.randrange(1, 20), H=H, Hk=Hk, Dk=Dk, Dv=Dv, dtype=dtype, gate=gate)
    B, T, packed = rng.choice([1, 1, 2, 4]), _log(rng, 1, 6000), 0
    if B == 1 and T > 40 and rng.random() < 0.5:
        packed = rng.randrange(2, 20)
    return dict(op=op, B=B, T=T, H=H, Hk=Hk, Dk=Dk, Dv=Dv, dtype=dtype, packed=packed, gate=gate)


def _type(case):
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[case["dtype"]]


def _lengths(case, seed):
    """Lengths of packed sequences, ragged, one of them a single step, one empty."""
    g = torch.Generator()
    g.manual_seed(seed)
    n, T = case["packed"], case["T"]
    cuts = torch.sort(torch.randint(1, T, (n - 2,), generator=g)).values.tolist()
    cu = sorted([0, 0] + cuts + [T])  # the first sequence is empty
    return cu


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = _type(case)

    def normal(*shape, dtype=dt):
        return torch.randn(shape, device=dev, generator=g).to(dtype)

    s = dict(case=case)
    B, H = case["B"], case["H"]
    Hk = case["Hk"] or H
    if case["op"] in ("norm", "norm_train"):
        T, D, R = case["T"], case["D"], case["rot"]
        qkv = normal(B, T, H + 2 * Hk, D)  # the projection's output: q and k are views of it
        s["q"], s["k"] = qkv[:, :, :H], qkv[:, :, H:H + Hk]
        s["qw"] = (1 + 0.2 * normal(D, dtype=torch.float32)).to(dt)
        s["kw"] = (1 + 0.2 * normal(D, dtype=torch.float32)).to(dt)
        pos = torch.arange(case["far"], device=dev, dtype=torch.float64)
        inv = 10000.0 ** (-torch.arange(0, R, 2, device=dev, dtype=torch.float64) / R)
        s["cos"], s["sin"] = torch.cos(pos[:, None] * inv).float(), torch.sin(pos[:, None] * inv).float()
        first = torch.randint(0, case["far"] - T + 1, (B, 1), device=dev, generator=g)
        s["pos"] = (first + torch.arange(T, device=dev)).to(torch.int32)
        if case["op"] == "norm_train":
            s["dq"], s["dk"] = normal(B, T, H, D), normal(B, T, Hk, D)
        return s
    Dk, Dv = case["Dk"], case["Dv"]
    s["scale"] = Dk ** -0.5
    lead = (B,) if case["op"] == "step" else (B, case["T"])
    s["q"], s["k"], s["v"] = normal(*lead, Hk, Dk), normal(*lead, Hk, Dk), normal(*lead, H, Dv)
    # memories from a few steps to a few thousand over the heads
    far = torch.linspace(1.0, 8.0, H, device=dev)
    z = normal(*lead, H, dtype=torch.float32) + far if case["gate"] == "token" else far
    s["g"] = torch.nn.functional.logsigmoid(z)
    if case["op"] == "step":
        s["state"] = normal(case["slots"], H, Dk, Dv, dtype=torch.float32)
        s["slots"] = torch.randperm(case["slots"], device=dev, generator=g)[:B].to(torch.int32)
        return s
    s["cu"], n = None, B
    if case["packed"]:
        s["cu"] = torch.tensor(_lengths(case, seed), dtype=torch.int32, device=dev)
        n = case["packed"]
    s["h0"] = normal(n, H, Dk, Dv, dtype=torch.float32)
    if case["op"] == "train":
        s["do"] = normal(*lead, H, Dv)
        s["dht"] = normal(n, H, Dk, Dv, dtype=torch.float32)
    return s


def run(s):
    op = s["case"]["op"]
    if own:
        return _OWN[op](s)
    return _PLAIN[op](s)


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------
def _own_prompt(s):
    import associative_scan_amd as m
    return m.linear_attention_fwd(s["q"], s["k"], s["v"], s["g"], h0=s["h0"], cu_seqlens=s["cu"], scale=s["scale"])


def _own_train(s):
    import associative_scan_amd as m
    o, ht = m.linear_attention_fwd(s["q"], s["k"], s["v"], s["g"], h0=s["h0"], cu_seqlens=s["cu"], scale=s["scale"])
    grads = m.linear_attention_bwd(s["q"], s["k"], s["v"], s["g"], s["do"], h0=s["h0"], dht=s["dht"],
                                   cu_seqlens=s["cu"], scale=s["scale"])
    return (o, ht) + tuple(grads)


def _own_step(s):
    import associative_scan_amd as m
    o = m.linear_attention_step(s["q"], s["k"], s["v"], s["g"], s["state"], slots=s["slots"], scale=s["scale"])
    return o, s["state"]


def _own_norm(s):
    import associative_scan_amd as m
    return m.qk_norm_rope_fwd(s["q"], s["k"], s["qw"], s["kw"], s["cos"], s["sin"], positions=s["pos"])


def _own_norm_train(s):
    import associative_scan_amd as m
    y = m.qk_norm_rope_fwd(s["q"], s["k"], s["qw"], s["kw"], s["cos"], s["sin"], positions=s["pos"])
    grads = m.qk_norm_rope_bwd(s["q"], s["k"], s["qw"], s["kw"], s["cos"], s["sin"], s["dq"], s["dk"],
                               positions=s["pos"])
    return tuple(y) + tuple(grads)


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _padded(cu, T):
    """(index [n, L] into the packed axis, valid [n, L]) of packed sequences."""
    cu = cu.long()
    L = int((cu[1:] - cu[:-1]).max())
    at = cu[:-1, None] + torch.arange(L, device=cu.device)
    valid = at < cu[1:, None]
    return at.clamp(max=T - 1), valid


def _chunked(q, k, v, g, h0, scale):
    """q, k [n, L, H, Dk], v [n, L, H, Dv], g [n, L, H], h0 [n, H, Dk, Dv], all fp32 -> (o, ht)."""
    n, L, H, Dk = q.shape
    Dv, C = v.shape[-1], CHUNK
    N = -(-L // C)
    pad = N * C - L
    if pad:  # steps of no effect: no injection, a decay of one
        q, k, v = (torch.nn.functional.pad(x, (0, 0, 0, 0, 0, pad)) for x in (q, k, v))
        g = torch.nn.functional.pad(g, (0, 0, 0, pad))
    q, k, v = (x.reshape(n, N, C, H, -1).permute(0, 3, 1, 2, 4).contiguous() for x in (q, k, v))  # [n, H, N, C, D]
    g = g.reshape(n, N, C, H).permute(0, 3, 1, 2).double()
    b = g.cumsum(-1)
    tri = torch.ones(C, C, device=q.device, dtype=torch.bool).tril()
    decay = torch.where(tri, b[..., :, None] - b[..., None, :], -math.inf).float().exp()
    o = (q @ k.transpose(-1, -2)) * decay @ v
    local = (k * (b[..., -1:] - b).float().exp()[..., None]).transpose(-1, -2) @ v  # [n, H, N, Dk, Dv]
    # states before each chunk and after the last: decays between chunks as one (N + 1) x (N + 1) matrix
    e = torch.nn.functional.pad(b[..., -1].cumsum(-1), (1, 0))  # [n, H, N + 1]
    tri = torch.ones(N + 1, N + 1, device=q.device, dtype=torch.bool).tril()
    between = torch.where(tri, e[..., :, None] - e[..., None, :], -math.inf).float().exp()
    sources = torch.cat([h0[:, :, None], local], 2).reshape(n, H, N + 1, Dk * Dv)
    states = (between @ sources).reshape(n, H, N + 1, Dk, Dv)
    o = o + (q * b.float().exp()[..., None]) @ states[:, :, :-1]
    o = (o * scale).permute(0, 2, 3, 1, 4).reshape(n, N * C, H, Dv)[:, :L]
    return o, states[:, :, -1]


def _plain_attention(q, k, v, g, h0, cu, scale):
    """Linear attention of fp32 tensors in the operators' layouts."""
    H, Hk, T = v.shape[2], q.shape[2], q.shape[1]
    q, k = (x.repeat_interleave(H // Hk, 2) for x in (q, k))
    g = g.expand(*v.shape[:3])
    if cu is None:
        return _chunked(q, k, v, g, h0, scale)
    at, valid = _padded(cu, T)
    w = valid[..., None]
    q, k, v = (torch.where(w[..., None], x[0][at], 0.0) for x in (q, k, v))
    o, ht = _chunked(q, k, v, torch.where(w, g[0][at], 0.0), h0, scale)
    return o[valid][None], ht


def _plain_prompt(s):
    o, ht = _plain_attention(s["q"].float(), s["k"].float(), s["v"].float(), s["g"], s["h0"], s["cu"], s["scale"])
    return o.to(s["v"].dtype), ht


def _plain_train(s):
    leaves = [x.float().requires_grad_() for x in (s["q"], s["k"], s["v"])]
    leaves += [s["g"].detach().clone().requires_grad_(), s["h0"].detach().clone().requires_grad_()]
    with torch.enable_grad():
        o, ht = _plain_attention(*leaves, s["cu"], s["scale"])
    dq, dk, dv, dg, dh0 = torch.autograd.grad([o, ht], leaves, [s["do"].float(), s["dht"]])
    dt = s["v"].dtype
    return o.detach().to(dt), ht.detach(), dq.to(dt), dk.to(dt), dv.to(dt), dg, dh0


def _plain_step(s):
    H, Hk = s["v"].shape[1], s["q"].shape[1]
    q, k = (s[x].float().repeat_interleave(H // Hk, 1) for x in ("q", "k"))
    v, at = s["v"].float(), s["slots"].long()
    S = s["state"][at] * s["g"].expand(*v.shape[:2]).exp()[..., None, None] + k[..., :, None] * v[..., None, :]
    s["state"][at] = S
    o = (q[..., :, None] * S).sum(-2) * s["scale"]
    return o.to(s["v"].dtype), s["state"]


def _rotate(n, cos, sin):
    """The first 2 * cos.shape[-1] entries of each head as pairs (i, i + half)."""
    r = cos.shape[-1]
    a, b, rest = n[..., :r], n[..., r:2 * r], n[..., 2 * r:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)


def _plain_heads(x, w, cos, sin):
    x = x.float()
    return _rotate(x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.float(), cos, sin)


def _plain_norm(s):
    at = s["pos"].long()
    cos, sin = s["cos"][at][:, :, None], s["sin"][at][:, :, None]
    return tuple(_plain_heads(s[x], s[w], cos, sin).to(s[x].dtype) for x, w in (("q", "qw"), ("k", "kw")))


def _plain_norm_train(s):
    at = s["pos"].long()
    cos, sin = s["cos"][at][:, :, None], s["sin"][at][:, :, None]
    ys, dxs, dws = [], [], []
    for x, w, dy in (("q", "qw", "dq"), ("k", "kw", "dk")):
        ys.append(_plain_heads(s[x], s[w], cos, sin).to(s[x].dtype))
        f, wf = s[x].float(), s[w].float()
        r = torch.rsqrt((f * f).mean(-1, keepdim=True) + 1e-6)
        dn = _rotate(s[dy].float(), cos, -sin)
        hat = f * r
        t = dn * wf
        dxs.append((r * (t - hat * (t * hat).mean(-1, keepdim=True))).to(s[x].dtype))
        dws.append((dn * hat).sum((0, 1, 2)))
    return tuple(ys + dxs + dws)


_OWN = dict(prompt=_own_prompt, train=_own_train, step=_own_step, norm=_own_norm, norm_train=_own_norm_train)
_PLAIN = dict(prompt=_plain_prompt, train=_plain_train, step=_plain_step, norm=_plain_norm, norm_train=_plain_norm_train)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    e = 4 if case["dtype"] == "fp32" else 2
    B, H = case["B"], case["H"]
    Hk = case["Hk"] or H
    if case["op"] in ("norm", "norm_train"):
        rows, D, R = B * case["T"], case["D"], case["rot"]
        x = rows * (H + Hk) * D
        table = min(rows, case["far"]) * R * 4 + rows * 4
        if case["op"] == "norm":
            return dict(bytes=2 * x * e + table + 2 * D * e, flops=8 * x)
        # forward: x, y; backward: x, dy, dx
        return dict(bytes=5 * x * e + 2 * table + 2 * D * (2 * e + 4), flops=26 * x)
    Dk, Dv = case["Dk"], case["Dv"]
    tokens = B * case.get("T", 1)
    gates = tokens * H * 4 if case["gate"] == "token" else H * 4
    qk, vo = tokens * Hk * Dk * e, tokens * H * Dv * e
    cell = tokens * H * Dk * Dv
    if case["op"] == "step":
        return dict(bytes=2 * qk + 2 * vo + gates + 8 * cell, flops=5 * cell)
    states = (case["packed"] or B) * H * Dk * Dv * 4
    fwd = 2 * qk + 2 * vo + gates + 2 * states
    # the recurrence itself: decay and update of the state, and its product with the query
    if case["op"] == "prompt":
        return dict(bytes=fwd, flops=5 * cell)
    # backward: q, k, v, g, do, h0, dht read; dq, dk, dv, dg, dh0 written
    return dict(bytes=fwd + 4 * qk + 3 * vo + 2 * gates + 3 * states, flops=18 * cell)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        if case["op"] in ("norm", "norm_train"):
            return _exact_norm(s, case["op"] == "norm_train")
        if case["op"] == "step":
            return _exact_step(s)
        return _exact_attention(s, case["op"] == "train")


def _exact_step(s):
    q, k, v, g, state = (s[x].double() for x in ("q", "k", "v", "g", "state"))
    B, H, r = v.shape[0], v.shape[1], v.shape[1] // q.shape[1]
    o = torch.empty_like(v)
    g = g.expand(B, H)
    for i, slot in enumerate(s["slots"].tolist()):
        kk, qq = k[i].repeat_interleave(r, 0), q[i].repeat_interleave(r, 0)
        state[slot] = torch.exp(g[i])[:, None, None] * state[slot] + torch.einsum("hk,hv->hkv", kk, v[i])
        o[i] = s["scale"] * torch.einsum("hk,hkv->hv", qq, state[slot])
    return o, state


def _exact_attention(s, train):
    """The recurrence step by step: one step of all sequences at a time."""
    q, k, v, g = (s[x].double() for x in ("q", "k", "v", "g"))
    B, T, H, r = v.shape[0], v.shape[1], v.shape[2], v.shape[2] // q.shape[2]
    a = torch.exp(g.expand(B, T, H))
    S, scale, dev = s["h0"].double(), s["scale"], v.device
    if s["cu"] is None:
        cu, longest = [0, T], T
    else:
        cu = s["cu"].tolist()
        longest = max(b - a_ for a_, b in zip(cu, cu[1:]))
    q, k = q.repeat_interleave(r, 2), k.repeat_interleave(r, 2)

    def at(t):
        """Batch index and time index of step t of every sequence that has one, and those sequences."""
        if s["cu"] is None:
            return slice(None), t, slice(None)
        live = [i for i in range(len(cu) - 1) if cu[i] + t < cu[i + 1]]
        return 0, torch.tensor([cu[i] + t for i in live], device=dev), torch.tensor(live, device=dev)

    places = [at(t) for t in range(longest)]
    o = torch.zeros_like(v)
    if train:
        do = s["do"].double()
        dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for bi, ti, n in places:
        S[n] = a[bi, ti][..., None, None] * S[n] + k[bi, ti][..., :, None] * v[bi, ti][..., None, :]
        o[bi, ti] = scale * (q[bi, ti][..., None, :] @ S[n])[..., 0, :]
        if train:
            dq[bi, ti] = scale * (S[n] @ do[bi, ti][..., :, None])[..., 0]
    if not train:
        return o, S
    lam = s["dht"].double()
    run_dg = (lam * S).sum((-1, -2))  # [n, H]
    dg = torch.zeros_like(a)
    for bi, ti, n in reversed(places):
        lam[n] = lam[n] + scale * q[bi, ti][..., :, None] * do[bi, ti][..., None, :]
        dk[bi, ti] = (lam[n] @ v[bi, ti][..., :, None])[..., 0]
        dv[bi, ti] = (k[bi, ti][..., None, :] @ lam[n])[..., 0, :]
        # d/dg_t = <Lam_t, e^{g_t} S_{t-1}>, and <Lam_t, S_t> = <Lam_t, e^{g_t} S_{t-1}> + k_t . dk_t
        run_dg[n] = run_dg[n] + (q[bi, ti] * dq[bi, ti]).sum(-1) - (k[bi, ti] * dk[bi, ti]).sum(-1)
        dg[bi, ti] = run_dg[n]
        lam[n] = a[bi, ti][..., None, None] * lam[n]
    dq, dk = (x.reshape(B, T, H // r, r, -1).sum(3) for x in (dq, dk))
    if s["g"].dim() == 1:
        dg = dg.sum((0, 1))
    return o, S, dq, dk, dv, dg, lam


def _exact_norm(s, train):
    at = s["pos"].long()
    z = torch.complex(s["cos"].double(), s["sin"].double())[at][:, :, None]
    half = z.shape[-1]

    def turn(x, z):
        c = torch.complex(x[..., :half], x[..., half:2 * half]) * z
        return torch.cat([c.real, c.imag, x[..., 2 * half:]], -1)

    ys, dxs, dws = [], [], []
    for x, w, dy in (("q", "qw", "dq"), ("k", "kw", "dk")):
        x, w = s[x].double(), s[w].double()
        size = torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6)
        ys.append(turn(x / size * w, z))
        if train:
            dn = turn(s[dy].double(), z.conj())
            dws.append((dn * x / size).sum((0, 1, 2)))
            t = dn * w
            dxs.append(t / size - x * (t * x).mean(-1, keepdim=True) / size ** 3)
    return tuple(ys + dxs + dws)
