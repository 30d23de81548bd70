"""Linear attention and the query/key norm as torch.library ops: opcheck, autograd
against the 64-bit reference and against differences, torch.compile, captured and
replayed graphs, other streams, and the whole path (norm, rotation, attention over
a prompt, then token by token) as a layer runs it."""
import numpy as np
import pytest
import torch

import attention_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def m():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import associative_scan_amd as m
    return m


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def make(seed, B, T, H, Dk, Dv, dtype=torch.float32, Hk=None, n=None, gate="token"):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    r = lambda *s: torch.randn(s, device=DEV, generator=gen)  # noqa: E731
    Hk = Hk or H
    g = -r(B, T, H).abs() * 0.1 if gate == "token" else -r(H).abs() * 0.1
    return (r(B, T, Hk, Dk).to(dtype), r(B, T, Hk, Dk).to(dtype), r(B, T, H, Dv).to(dtype), g, r(n or B, H, Dk, Dv))


def tables(n, rot):
    pos = torch.arange(n, dtype=torch.float64)
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    return torch.cos(pos[:, None] * inv).float().to(DEV), torch.sin(pos[:, None] * inv).float().to(DEV)


def near(got, want, mag, steps):
    """fp32 results: `steps` roundings of 2^-24 of the magnitude."""
    off = np.abs(f64(got) - want)
    tol = steps * 2.0 ** -24 * mag + 1e-30
    assert np.all(off <= tol), np.max(off / tol)


def test_opcheck(m):
    q, k, v, g, h0 = (x.requires_grad_() for x in make(1, 1, 90, 2, 16, 24, n=2))
    cu = torch.tensor([0, 40, 90], dtype=torch.int32, device=DEV)
    torch.library.opcheck(torch.ops.mscan.linear_attention.default, (q, k, v, g, h0, cu, 0.25))
    q, k, v, g, h0 = (x.requires_grad_() for x in make(2, 2, 70, 4, 16, 24, torch.bfloat16, Hk=2, gate="head"))
    torch.library.opcheck(torch.ops.mscan.linear_attention.default, (q, k, v, g, None, None, 0.25))
    cos, sin = tables(100, 16)
    w = torch.rand(16, device=DEV).requires_grad_()
    torch.library.opcheck(torch.ops.mscan.qk_norm_rope.default, (q, k, None, None, cos, sin, None, 1e-6, False))
    q, k = (x.detach().float().requires_grad_() for x in (q, k))
    torch.library.opcheck(torch.ops.mscan.qk_norm_rope.default, (q, k, w, w.detach().clone(), cos, sin, None, 1e-6, True))
    q, k, v, g, _ = make(3, 3, 1, 2, 16, 24)
    torch.library.opcheck(torch.ops.mscan.linear_attention_step.default,
                          (q[:, 0], k[:, 0], v[:, 0], g[:, 0], torch.randn(3, 2, 16, 24, device=DEV), None, 0.5))


def test_autograd_matches_the_formula(m):
    x = [t.requires_grad_() for t in make(4, 1, 150, 4, 32, 16, Hk=2, n=3)]
    cu = [0, 60, 60, 150]
    c = torch.tensor(cu, dtype=torch.int32, device=DEV)
    o, ht = m.linear_attention(*x[:4], h0=x[4], cu_seqlens=c, scale=0.3)
    do, dht = torch.randn_like(o), torch.randn_like(ht)
    grads = torch.autograd.grad([o, ht], x, [do, dht])
    want = ref.backward(*(f64(t) for t in x[:4]), f64(do), f64(x[4]), f64(dht), cu, 0.3)
    rows = np.max((np.abs(f64(x[0])) * want[0][1]).sum(3) + (np.abs(f64(x[1])) * want[1][1]).sum(3))
    for i, (a, (w, mag)) in enumerate(zip(grads, want)):
        near(a, w, mag + (rows * 2 * 150 ** 0.5 if i == 3 else 0), 150 + 32 + 16 + 256)


def test_autograd_of_parts(m):
    """Only o, only ht, and only some leaves."""
    q, k, v, g, h0 = make(5, 2, 40, 2, 16, 16)
    for which in ("o", "ht"):
        x = [t.clone().requires_grad_() for t in (q, k, v, g, h0)]
        o, ht = m.linear_attention(*x[:4], h0=x[4], scale=0.3)
        (o if which == "o" else ht).square().sum().backward()
        do = 2 * o.detach() if which == "o" else torch.zeros_like(o)
        dht = 2 * ht.detach() if which == "ht" else None
        want = m.linear_attention_bwd(q, k, v, g, do, h0=h0, dht=dht, scale=0.3)
        for t, w in zip(x, want):
            assert torch.equal(t.grad, w)
    v2 = v.clone().requires_grad_()
    m.linear_attention(q, k, v2, g)[0].sum().backward()
    ones = torch.ones_like(v)
    w = m.linear_attention_bwd(q, k, v, g, ones, need_dg=False, need_dh0=False)[2]
    assert torch.equal(v2.grad, w) and q.grad is None


def test_gradients_against_differences(m):
    """Central differences of a loss in 64 bits from the reference, along random
    directions. With steps of 1e-4 their own error is some 1e-8 of the slope's
    terms; the gradients' is (T + Dk + Dv + 256) 2^-24 = 2e-5 of theirs (times
    root T more for dg, whose sums run over the steps): 1e-4 holds both."""
    x = make(6, 1, 30, 2, 8, 8)
    r = np.random.default_rng(0)
    w, wt = r.standard_normal((1, 30, 2, 8)), r.standard_normal((1, 2, 8, 8))
    leaves = [t.clone().requires_grad_() for t in x]
    o, ht = m.linear_attention(*leaves[:4], h0=leaves[4], scale=0.4)
    ((o * torch.tensor(w, device=DEV).float()).sum() + (ht * torch.tensor(wt, device=DEV).float()).sum()).backward()
    base = [f64(t) for t in x]

    def loss(v):
        (o, _), (ht, _) = ref.forward(*v[:4], v[4], None, 0.4)
        return (o * w).sum() + (ht * wt).sum()

    for i, t in enumerate(leaves):
        d = r.standard_normal(base[i].shape)
        h = 1e-4
        up, dn = list(base), list(base)
        up[i], dn[i] = base[i] + h * d, base[i] - h * d
        slope = (loss(up) - loss(dn)) / (2 * h)
        got = (f64(t.grad) * d).sum()
        assert abs(got - slope) <= 1e-4 * (np.abs(f64(t.grad)) * np.abs(d)).sum(), i


def test_norm_autograd(m):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(7)
    r = lambda *s: torch.randn(s, device=DEV, generator=gen)  # noqa: E731
    q, k, wq, wk = r(2, 20, 3, 64), r(2, 20, 2, 64), r(64), r(64)
    cos, sin = tables(50, 32)
    pos = torch.arange(7, 27, device=DEV)
    x = [t.clone().requires_grad_() for t in (q, k, wq, wk)]
    yq, yk = m.qk_norm_rope(*x, cos, sin, positions=pos)
    dq, dk = r(2, 20, 3, 64), r(2, 20, 2, 64)
    torch.autograd.backward([yq, yk], [dq, dk])
    for t, w in zip(x, m.qk_norm_rope_bwd(q, k, wq, wk, cos, sin, dq, dk, positions=pos)):
        assert torch.equal(t.grad, w)
    # bf16 weights get bf16 gradients; only the keys' result used
    x = [t.bfloat16().requires_grad_() for t in (q, k, wq, wk)]
    m.qk_norm_rope(*x, cos, sin)[1].float().sum().backward()
    assert x[2].grad.dtype == torch.bfloat16 and torch.equal(x[0].grad, torch.zeros_like(x[0]))
    assert x[1].grad.abs().sum() > 0


def layer(m, z, wq, wk, cos, sin, g, cu=None, h0=None, positions=None):
    """A mixer on one fused projection z [B, T, 3 H, D]."""
    H = z.shape[2] // 3
    return m.rotary_linear_attention(z[:, :, :H], z[:, :, H:2 * H], z[:, :, 2 * H:], g, wq, wk, cos, sin,
                                     positions=positions, h0=h0, cu_seqlens=cu)


def test_whole_path_prompt_then_tokens(m):
    """Norm, rotation, attention over a packed prompt, then decoding with a pool of
    states, against the same in 64 bits: o within its bf16 rounding and that of the
    rotated q and k, which are rounded to bf16 before the attention reads them."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(8)
    r = lambda *s: torch.randn(s, device=DEV, generator=gen)  # noqa: E731
    H, D, lens, steps = 4, 64, [37, 100, 1], 5
    T = sum(lens)
    cu = torch.tensor([0, 37, 137, 138], dtype=torch.int32, device=DEV)
    z = r(1, T, 3 * H, D).bfloat16()
    wq, wk = 1 + 0.1 * r(D), 1 + 0.1 * r(D)
    wq, wk = wq.bfloat16(), wk.bfloat16()
    g = -r(1, T, H).abs() * 0.05
    cos, sin = tables(200, D)
    pos = torch.cat([torch.arange(n) for n in lens]).to(DEV)
    o, ht = layer(m, z, wq, wk, cos, sin, g, cu=cu, positions=pos)
    # decoding: the three sequences sit in slots 4, 0, 2 of a pool of 6
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device=DEV)
    pool = r(6, H, D, D)
    keep = pool.clone()
    pool[slots.long()] = ht
    zs, gs, outs = r(steps, 3, 3 * H, D).bfloat16(), -r(steps, 3, H).abs() * 0.05, []
    for t in range(steps):
        x = zs[t]
        outs.append(m.rotary_linear_attention_step(x[:, :H], x[:, H:2 * H], x[:, 2 * H:], gs[t], pool, wq, wk, cos, sin,
                                                   positions=torch.tensor(lens, device=DEV) + t, slots=slots))
    for n in (1, 3, 5):
        assert torch.equal(pool[n], keep[n])

    def turned(x, w, p):
        x = f64(x)
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6) * f64(w)
        c, s = f64(cos)[p][..., None, :], f64(sin)[p][..., None, :]
        a, b = x[..., :D // 2], x[..., D // 2:]
        return torch.tensor(np.concatenate([a * c - b * s, b * c + a * s], -1)).bfloat16().double().numpy()

    for i, (s, e) in enumerate(zip(cu.tolist()[:-1], cu.tolist()[1:])):
        zi = torch.cat([z[0, s:e], zs[:, i]], 0)[None]
        gi = torch.cat([g[0, s:e], gs[:, i]], 0)[None]
        p = np.arange(e - s + steps)[None]
        q, k = turned(zi[:, :, :H], wq, p), turned(zi[:, :, H:2 * H], wk, p)
        (want, mag), (wh, hm) = ref.forward(q, k, f64(zi[:, :, 2 * H:]), f64(gi), None, None, D ** -0.5)
        got = np.concatenate([f64(o[0, s:e]), np.stack([f64(x[i]) for x in outs])])[None]
        # an entry of q or k next to a rounding border may round the other way: one
        # bf16 step, 2^-8 of it, and not all of them at once
        tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -9 * mag
        assert np.all(np.abs(got - want) <= tol), np.max(np.abs(got - want) / tol)
        assert np.all(np.abs(f64(pool[slots[i].item()]) - wh[0]) <= 2.0 ** -9 * hm[0])


def test_training_step_compiles(m):
    cos, sin = tables(128, 32)

    def step(z, wq, wk, a):
        g = torch.nn.functional.logsigmoid(a)
        o, ht = layer(m, z, wq, wk, cos, sin, g)
        return o.float().square().mean() + ht.mean()

    def inputs():
        torch.manual_seed(9)
        return [torch.randn(s, device=DEV).requires_grad_() for s in ((2, 128, 6, 32), (32,), (32,), (2, 128, 2))]

    a, b = inputs(), inputs()
    step(*a).backward()
    torch.compile(step, backend="aot_eager", fullgraph=True)(*b).backward()
    for x, y in zip(a, b):
        assert torch.allclose(x.grad, y.grad, rtol=1e-5, atol=1e-7)


def test_captured_forward_and_backward_replay(m):
    """A captured training step, replayed with new inputs, eager work between the
    replays, and a second graph of another size."""
    cos, sin = tables(2000, 64)

    def graph_of(T, seed):
        torch.manual_seed(seed)
        z, w = torch.randn(1, T, 6, 64, device=DEV).bfloat16(), torch.rand(64, device=DEV).bfloat16()
        g = -torch.rand(1, T, 2, device=DEV) * 0.01
        h0 = torch.randn(1, 2, 64, 64, device=DEV)
        leaves = [t.requires_grad_() for t in (z, w, g, h0)]

        def run():
            o, ht = layer(m, z, w, w, cos, sin, g, h0=h0)
            grads = torch.autograd.grad([o, ht], leaves, [torch.ones_like(o), torch.ones_like(ht)])
            return (o.detach(), ht.detach()) + grads

        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            run()
        torch.cuda.current_stream().wait_stream(s)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = run()
        return graph, out, z, run

    one, two = graph_of(1500, 1), graph_of(70, 2)
    for i in range(4):
        for graph, out, z, run in ((one, two)[i % 2], (one, two)[1 - i % 2]):
            with torch.no_grad():
                z.copy_(torch.randn_like(z.float()).bfloat16())
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip(out, run()):
                assert torch.equal(a, b)


def test_two_streams_at_once(m):
    """Calls that overlap on two streams, each with its own workspace."""
    x = [make(20 + i, 2, 1800, 3, 64, 64, torch.bfloat16) for i in range(2)]
    do = [torch.randn_like(t[2]) for t in x]
    want = [m.linear_attention_fwd(*t[:4], h0=t[4]) + m.linear_attention_bwd(*t[:4], d, h0=t[4]) for t, d in zip(x, do)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = [None, None]
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i] = m.linear_attention_fwd(*x[i][:4], h0=x[i][4]) + m.linear_attention_bwd(*x[i][:4], do[i], h0=x[i][4])
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            for a, b in zip(g, w):
                assert torch.equal(a, b)


def test_gradients_that_start_anywhere(m):
    """Outputs that went through torch.cat: their gradients are contiguous slices
    that start 2 or 4 bytes into 16."""
    def through_cat(*outs):
        loss, parts = 0.0, []
        for t in outs:
            w = torch.randn(t.numel() + 1, device=DEV).to(t.dtype)
            loss = loss + (torch.cat([t.new_zeros(1), t.reshape(-1)]) * w).float().sum()
            parts.append(w[1:].reshape(t.shape).clone())
        return loss, parts

    for dtype in (torch.bfloat16, torch.float32):
        x = [t.requires_grad_() for t in make(30, 1, 20, 2, 16, 8, dtype)]
        loss, (do, dht) = through_cat(*m.linear_attention(*x[:4], h0=x[4], scale=0.3))
        got = torch.autograd.grad(loss, x)
        want = m.linear_attention_bwd(*(t.detach() for t in x[:4]), do, h0=x[4].detach(), dht=dht, scale=0.3)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        cos, sin = tables(20, 16)
        w = torch.rand(16, device=DEV)
        loss, dy = through_cat(*m.qk_norm_rope(x[0], x[1], w, w, cos, sin))
        got = torch.autograd.grad(loss, x[:2])
        want = m.qk_norm_rope_bwd(x[0].detach(), x[1].detach(), w, w, cos, sin, *dy)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
