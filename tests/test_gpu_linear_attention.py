"""Linear attention on the GPU against the recurrence in 64 bits.

Tolerances. With M the result's sum over absolute values (attention_reference):
 - an fp32 sum of n terms is off by at most n 2^-24 M; the chunked form adds each
   term into a state (T steps), a product over Dk or Dv and one over a chunk. A
   decay e^x is off by |x| 2^-24 from the rounding of x plus 2^-23, and counts
   only while e^x does: |x| e^x stays below the factor's own share. So
   fp32 = (T + Dk + Dv + 256) 2^-24 M;
 - bf16 operands: the pieces of scores and states leave 2^-17 M in o, dq, dk, dv
   (2 pieces of 8 bits each, one rounding each);
 - the output's own rounding: eps / 2 of the value.
"""
import numpy as np
import pytest
import torch

import attention_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def m():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import associative_scan_amd as m
    return m


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def make(seed, B, T, H, Dk, Dv, dtype="bf16", Hk=None, gate="token", n=None, spread=(1.0, 6.0)):
    """q, k, v, g, h0, do, dht on the GPU."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    r = lambda *s: torch.randn(s, device=DEV, generator=gen)  # noqa: E731
    dt, Hk, n = TYPES[dtype], Hk or H, n or B
    far = torch.linspace(*spread, H, device=DEV)
    g = torch.nn.functional.logsigmoid(r(B, T, H) + far if gate == "token" else far)
    return (r(B, T, Hk, Dk).to(dt), r(B, T, Hk, Dk).to(dt), r(B, T, H, Dv).to(dt), g, r(n, H, Dk, Dv),
            r(B, T, H, Dv).to(dt), r(n, H, Dk, Dv))


def close(got, want, name, T, Dk, Dv, dtype):
    val, mag = want
    got64 = f64(got)
    assert got64.shape == val.shape, (name, got64.shape, val.shape)
    tol = (T + Dk + Dv + 256) * 2.0 ** -24 * mag + 1e-30
    if got.dtype != torch.float32:
        tol = tol + torch.finfo(got.dtype).eps / 2 * np.abs(val)
        tol = tol + torch.finfo(got.dtype).tiny  # fp16's subnormals: half a step of 2^-24
    if dtype == "bf16" and name in ("o", "dq", "dk", "dv"):
        tol = tol + 2.0 ** -17 * mag
    off = np.abs(got64 - val)
    assert np.all(np.isfinite(got64)), name
    worst = float(np.max(off / tol)) if off.size else 0.0
    assert worst <= 1.0, f"{name}: {worst:.2f} of the tolerance"


def check_forward(m, x, cu=None, scale=None, h0=True, dtype="bf16"):
    q, k, v, g, s0 = x[:5]
    s0 = s0 if h0 else None
    c = None if cu is None else torch.tensor(cu, dtype=torch.int32, device=DEV)
    o, ht = m.linear_attention_fwd(q, k, v, g, h0=s0, cu_seqlens=c, scale=scale)
    sc = q.shape[3] ** -0.5 if scale is None else scale
    wo, wh = ref.forward(f64(q), f64(k), f64(v), f64(g), f64(s0), cu, sc)
    d = (q.shape[1], q.shape[3], v.shape[3], dtype)
    close(o, wo, "o", *d)
    close(ht, wh, "ht", *d)
    return o, ht


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T", [1, 2, 31, 32, 33, 63, 64, 65, 127, 130, 255, 256, 257, 600])
def test_forward_lengths(m, T, dtype):
    check_forward(m, make(T, 2, T, 3, 64, 64, dtype), dtype=dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("Dk,Dv", [(8, 8), (16, 40), (40, 16), (64, 128), (128, 64), (72, 96), (96, 72), (128, 128),
                                   (120, 104), (8, 128), (128, 8)])
def test_forward_head_sizes(m, Dk, Dv, dtype):
    check_forward(m, make(Dk + Dv, 1, 300, 2, Dk, Dv, dtype), dtype=dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_forward_shared_heads_and_head_decays(m, dtype):
    check_forward(m, make(1, 2, 150, 6, 64, 32, dtype, Hk=2), dtype=dtype)
    check_forward(m, make(2, 1, 700, 4, 128, 64, dtype, Hk=1, gate="head"), dtype=dtype, h0=False, scale=0.5)


CUTS = [
    [0, 300],
    [0, 0, 300],
    [0, 300, 300],
    [0, 1, 2, 64, 128, 129, 300],
    [0, 0, 0, 7, 7, 263, 300, 300],
    [0, 255, 256, 300],
]


@pytest.mark.parametrize("cu", CUTS, ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_forward_packed(m, cu, dtype):
    check_forward(m, make(len(cu), 1, 300, 2, 64, 64, dtype, n=len(cu) - 1), cu=cu, dtype=dtype)


def test_forward_packed_many_spans(m):
    cu = [0, 900, 900, 901, 1300, 2600, 2601]
    check_forward(m, make(5, 1, 2601, 2, 128, 128, n=6, spread=(3.0, 9.0)), cu=cu)


def test_forward_spans(m):
    """Sequences cut into several spans, with memories across all of them."""
    check_forward(m, make(6, 2, 1500, 2, 128, 128, spread=(4.0, 12.0)))
    check_forward(m, make(7, 1, 1025, 1, 64, 64, "fp32", spread=(8.0, 8.0)), dtype="fp32")


def test_resets(m):
    """g = -inf and very strong decays: nothing before them is left, and no NaN appears."""
    q, k, v, g, h0, do, dht = make(8, 1, 200, 2, 64, 64)
    g[:, 0] = -float("inf")
    g[:, 63:66] = -float("inf")
    g[:, 100] = -1e30
    g[:, 101] = -200.0
    o, ht = check_forward(m, (q, k, v, g, h0))
    a, ha = m.linear_attention_fwd(q[:, 100:].contiguous(), k[:, 100:].contiguous(), v[:, 100:].contiguous(),
                                   g[:, 100:].contiguous())
    assert torch.allclose(o[:, 100:].float(), a.float(), rtol=2 ** -7, atol=1e-3)
    g[:] = -float("inf")
    check_forward(m, (q, k, v, g, h0))


def test_nan_stays_in_its_sequence(m):
    cu = [0, 70, 150, 300]
    q, k, v, g, h0, do, dht = make(9, 1, 300, 2, 64, 64, n=3)
    c = torch.tensor(cu, dtype=torch.int32, device=DEV)
    o, ht = m.linear_attention_fwd(q, k, v, g, h0=h0, cu_seqlens=c)
    for bad in (float("nan"), float("inf")):
        q2, k2, v2, g2, h2 = (x.clone() for x in (q, k, v, g, h0))
        for x in (q2, k2, v2, g2):
            x[:, 75:149] = bad
        h2[1] = bad
        o2, ht2 = m.linear_attention_fwd(q2, k2, v2, g2, h0=h2, cu_seqlens=c)
        for s, e, n in ((0, 70, 0), (150, 300, 2)):
            assert torch.equal(o2[:, s:e], o[:, s:e]) and torch.equal(ht2[n], ht[n])
        assert torch.isnan(o2[:, 75:149]).any()


def test_steps_behind_the_last_sequence_are_zero(m):
    q, k, v, g, h0, do, dht = make(10, 1, 700, 2, 64, 64, n=2)
    q[:, 310:] = float("nan")
    c = torch.tensor([0, 300, 310], dtype=torch.int32, device=DEV)
    o, ht = m.linear_attention_fwd(q, k, v, g, h0=h0, cu_seqlens=c)
    assert torch.equal(o[:, 310:], torch.zeros_like(o[:, 310:])) and torch.isfinite(o).all()
    cut = [f64(x[:, :310]) for x in (q, k, v, g)]
    wo, wh = ref.forward(*cut, f64(h0), [0, 300, 310], 0.125)
    close(o[:, :310], wo, "o", 310, 64, 64, "bf16")
    close(ht, wh, "ht", 310, 64, 64, "bf16")


def test_strides(m):
    """Head-major tensors, slices of one projection, broadcast inputs."""
    q, k, v, g, h0, do, dht = make(11, 2, 140, 4, 64, 32)
    o, ht = m.linear_attention_fwd(q, k, v, g, h0=h0)
    hm = lambda x: x.transpose(1, 2).contiguous().transpose(1, 2)  # noqa: E731
    o2, ht2 = m.linear_attention_fwd(hm(q), hm(k), hm(v), g.transpose(1, 2).contiguous().transpose(1, 2), h0=h0)
    assert torch.equal(o, o2) and torch.equal(ht, ht2)
    both = torch.cat([q, k, torch.cat([v, v], 3)], 2)
    o3, ht3 = m.linear_attention_fwd(both[:, :, :4], both[:, :, 4:8], both[:, :, 8:, :32], g, h0=h0)
    assert torch.equal(o, o3) and torch.equal(ht, ht3)
    kb = k[:1, :, :1].expand(2, 140, 4, 64)
    o4, ht4 = m.linear_attention_fwd(q, kb, v, g, h0=h0)
    o5, ht5 = m.linear_attention_fwd(q, kb.contiguous(), v, g, h0=h0)
    assert torch.equal(o4, o5) and torch.equal(ht4, ht5)


def test_repeatable_and_without_final_state(m):
    q, k, v, g, h0, do, dht = make(12, 2, 2100, 3, 128, 128)
    o, ht = m.linear_attention_fwd(q, k, v, g, h0=h0)
    for _ in range(3):
        o2, ht2 = m.linear_attention_fwd(q, k, v, g, h0=h0)
        assert torch.equal(o, o2) and torch.equal(ht, ht2)
    o3, none = m.linear_attention_fwd(q, k, v, g, h0=h0, need_ht=False)
    assert none is None and torch.equal(o, o3)


def test_empty_shapes(m):
    z = lambda *s: torch.zeros(s, device=DEV, dtype=torch.bfloat16)  # noqa: E731
    h0 = torch.randn(2, 3, 8, 16, device=DEV)
    o, ht = m.linear_attention_fwd(z(2, 0, 3, 8), z(2, 0, 3, 8), z(2, 0, 3, 16), torch.zeros(3, device=DEV), h0=h0)
    assert o.shape == (2, 0, 3, 16) and torch.equal(ht, h0)
    o, ht = m.linear_attention_fwd(z(0, 5, 3, 8), z(0, 5, 3, 8), z(0, 5, 3, 16), torch.zeros(3, device=DEV))
    assert o.shape == (0, 5, 3, 16) and ht.shape == (0, 3, 8, 16)


# ---------------------------------------------------------------------------
# backward. dg is a sum of differences q . dq - k . dk over the steps up to a
# span's end (at most 1024 here): beside its own magnitude it carries their
# rounding, (T + Dk + Dv + 256) 2^-24 of each one's magnitude. These are
# independent, so their sum is held to the root of their number times the largest.
# ---------------------------------------------------------------------------
def check_backward(m, x, cu=None, scale=None, h0=True, dht=True, dtype="bf16"):
    q, k, v, g, s0, do, dh = x
    s0, dh = s0 if h0 else None, dh if dht else None
    c = None if cu is None else torch.tensor(cu, dtype=torch.int32, device=DEV)
    got = m.linear_attention_bwd(q, k, v, g, do, h0=s0, dht=dh, cu_seqlens=c, scale=scale)
    sc = q.shape[3] ** -0.5 if scale is None else scale
    want = ref.backward(f64(q), f64(k), f64(v), f64(g), f64(do), f64(s0), f64(dh), cu, sc)
    T, Dk, Dv = q.shape[1], q.shape[3], v.shape[3]
    for n, a, w in zip(("dq", "dk", "dv", "dg", "dh0"), got, want):
        if n == "dg":
            val, mag = w
            rows = (np.abs(f64(q)) * want[0][1]).sum(3) + (np.abs(f64(k)) * want[1][1]).sum(3)
            r = v.shape[2] // q.shape[2]
            mag = mag + min(T, 1024) ** 0.5 * np.repeat(rows, r, 2).max(1, keepdims=True)
            if g.dim() == 1:
                val, mag = val.sum((0, 1)), mag.sum((0, 1))
            w = (val, mag)
        close(a, w, n, T, Dk, Dv, dtype)
    return got


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T", [1, 2, 31, 33, 64, 65, 130, 256, 257, 600])
def test_backward_lengths(m, T, dtype):
    check_backward(m, make(T, 2, T, 3, 64, 64, dtype), dtype=dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("Dk,Dv", [(8, 8), (16, 40), (40, 16), (64, 128), (128, 64), (72, 96), (96, 72), (128, 128),
                                   (120, 104), (8, 128), (128, 8)])
def test_backward_head_sizes(m, Dk, Dv, dtype):
    check_backward(m, make(Dk + Dv, 1, 300, 2, Dk, Dv, dtype), dtype=dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_backward_shared_heads_and_head_decays(m, dtype):
    check_backward(m, make(1, 2, 150, 6, 64, 32, dtype, Hk=2), dtype=dtype)
    check_backward(m, make(2, 1, 700, 4, 128, 64, dtype, Hk=1, gate="head"), dtype=dtype, h0=False, scale=0.5)
    check_backward(m, make(3, 3, 100, 11, 16, 16, dtype, gate="head"), dtype=dtype, dht=False)


@pytest.mark.parametrize("cu", CUTS, ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_backward_packed(m, cu, dtype):
    check_backward(m, make(len(cu), 1, 300, 2, 64, 64, dtype, n=len(cu) - 1), cu=cu, dtype=dtype)
    check_backward(m, make(len(cu), 1, 300, 2, 64, 64, dtype, n=len(cu) - 1), cu=cu, dtype=dtype, h0=False, dht=False)


def test_backward_packed_many_spans(m):
    cu = [0, 900, 900, 901, 1300, 2600, 2601]
    check_backward(m, make(5, 1, 2601, 2, 128, 128, n=6, spread=(3.0, 9.0)), cu=cu)
    check_backward(m, make(5, 1, 2601, 4, 64, 64, Hk=1, n=6, gate="head"), cu=cu)


def test_backward_spans(m):
    check_backward(m, make(6, 2, 1500, 2, 128, 128, spread=(4.0, 12.0)))
    check_backward(m, make(7, 1, 1025, 1, 64, 64, "fp32", spread=(8.0, 8.0)), dtype="fp32")


def test_backward_resets(m):
    x = make(8, 1, 200, 2, 64, 64)
    g = x[3]
    g[:, 0] = -float("inf")
    g[:, 63:66] = -float("inf")
    g[:, 100] = -1e30
    g[:, 101] = -200.0
    dg = check_backward(m, x)[3]
    g[:] = -float("inf")
    assert torch.isfinite(dg).all() and torch.isfinite(check_backward(m, x)[3]).all()


def test_backward_nan_stays_in_its_sequence(m):
    cu = [0, 70, 150, 300]
    q, k, v, g, h0, do, dht = make(9, 1, 300, 2, 64, 64, n=3)
    c = torch.tensor(cu, dtype=torch.int32, device=DEV)
    want = m.linear_attention_bwd(q, k, v, g, do, h0=h0, dht=dht, cu_seqlens=c)
    for bad in (float("nan"), float("inf")):
        y = [t.clone() for t in (q, k, v, g, do)]
        for t in y:
            t[:, 75:149] = bad
        h2, d2 = h0.clone(), dht.clone()
        h2[1], d2[1] = bad, bad
        got = m.linear_attention_bwd(*y, h0=h2, dht=d2, cu_seqlens=c)
        for a, w in zip(got[:4], want[:4]):
            assert torch.equal(a[:, :70], w[:, :70]) and torch.equal(a[:, 150:], w[:, 150:])
        assert torch.equal(got[4][0], want[4][0]) and torch.equal(got[4][2], want[4][2])


@pytest.mark.parametrize("Hk", [2, 1])
def test_backward_steps_behind_the_last_sequence(m, Hk):
    q, k, v, g, h0, do, dht = make(10, 1, 700, 2, 64, 64, n=2, Hk=Hk)
    do[:, 310:] = float("nan")
    c = torch.tensor([0, 300, 310], dtype=torch.int32, device=DEV)
    got = m.linear_attention_bwd(q, k, v, g, do, h0=h0, dht=dht, cu_seqlens=c)
    cut = [f64(x[:, :310]) for x in (q, k, v, g, do)]
    want = ref.backward(*cut, f64(h0), f64(dht), [0, 300, 310], 0.125)
    for n, a, w in zip(("dq", "dk", "dv"), got, want):
        assert torch.equal(a[:, 310:], torch.zeros_like(a[:, 310:]))
        close(a[:, :310], w, n, 310, 64, 64, "bf16")
    assert torch.equal(got[3][:, 310:], torch.zeros_like(got[3][:, 310:])) and torch.isfinite(got[3]).all()
    close(got[4], want[4], "dh0", 310, 64, 64, "bf16")
    d1 = m.linear_attention_bwd(q, k, v, g[0, 0].contiguous(), do, h0=h0, dht=dht, cu_seqlens=c)[3]
    assert torch.isfinite(d1).all()


def test_backward_parts_and_repeats(m):
    q, k, v, g, h0, do, dht = make(12, 2, 2100, 3, 128, 128)
    want = m.linear_attention_bwd(q, k, v, g, do, h0=h0, dht=dht)
    for _ in range(3):
        for a, b in zip(want, m.linear_attention_bwd(q, k, v, g, do, h0=h0, dht=dht)):
            assert torch.equal(a, b)
    dq, dk, dv, dg, dh0 = m.linear_attention_bwd(q, k, v, g, do, h0=h0, dht=dht, need_dg=False, need_dh0=False)
    assert dg is None and dh0 is None
    for a, b in zip((dq, dk, dv), want):
        # without dg the state enters a product as two pieces instead of three
        assert (a.float() - b.float()).norm() <= 2 ** -8 * b.float().norm()


def test_backward_strides(m):
    q, k, v, g, h0, do, dht = make(11, 2, 140, 4, 64, 32)
    want = m.linear_attention_bwd(q, k, v, g, do, h0=h0, dht=dht)
    hm = lambda x: x.transpose(1, 2).contiguous().transpose(1, 2)  # noqa: E731
    for a, b in zip(want, m.linear_attention_bwd(hm(q), hm(k), hm(v), hm(g), hm(do), h0=h0, dht=dht)):
        assert torch.equal(a, b)
    # the gradient of a sum: one broadcast row of do
    ones = torch.ones(1, 1, 1, 32, device=DEV, dtype=q.dtype).expand(2, 140, 4, 32)
    for a, b in zip(m.linear_attention_bwd(q, k, v, g, ones), m.linear_attention_bwd(q, k, v, g, ones.contiguous())):
        assert torch.equal(a, b)


# ---------------------------------------------------------------------------
# long spans and far addresses
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("Dk,Dv", [(8, 8), (16, 72), (72, 16), (72, 72)])
def test_many_chunks_of_one_workgroup(m, Dk, Dv, dtype):
    """So many sequences and heads that none is cut: each workgroup runs more chunks
    than it has waves. The first and the last sequence are compared."""
    x = make(9, 65, 700, 8, Dk, Dv, dtype, spread=(3.0, 9.0))
    q, k, v, g, h0, do, dht = x
    got = m.linear_attention_fwd(q, k, v, g, h0=h0) + m.linear_attention_bwd(q, k, v, g, do, h0=h0, dht=dht)
    pick = torch.tensor([0, 64], device=DEV)
    some = [f64(t[pick]) for t in x]
    sc = Dk ** -0.5
    want = ref.forward(*some[:4], some[4], None, sc) + ref.backward(*some[:4], some[5], some[4], some[6], None, sc)
    rows = (np.abs(some[0]) * want[2][1]).sum(3) + (np.abs(some[1]) * want[3][1]).sum(3)
    want[5][1][:] += 700 ** 0.5 * rows.max(1, keepdims=True)
    for n, a, w in zip(("o", "ht", "dq", "dk", "dv", "dg", "dh0"), got, want):
        close(a[pick], w, n, 700, Dk, Dv, dtype)


def test_offsets_past_32_bits(m):
    """Values and outputs of more than 2^31 elements: the last sequence of a packed
    row against the same steps by themselves."""
    T, n, H, Dk, Dv = 2 ** 18 + 100, 100, 64, 8, 128
    assert (T - n) * H * Dv >= 2 ** 31
    x = make(10, 1, n, H, Dk, Dv, Hk=1, n=1)
    q, k, v, g, h0, do, dht = x

    def far(t):
        out = torch.zeros((1, T) + t.shape[2:], dtype=t.dtype, device=DEV)
        out[:, T - n:] = t
        return out

    cu = torch.tensor([0, T - n, T], dtype=torch.int32, device=DEV)
    states = torch.cat([torch.zeros_like(h0), h0]), torch.cat([torch.zeros_like(dht), dht])
    far_x = [far(t) for t in (q, k, v, g, do)]
    o, ht = m.linear_attention_fwd(*far_x[:4], h0=states[0], cu_seqlens=cu)
    grads = m.linear_attention_bwd(*far_x, h0=states[0], dht=states[1], cu_seqlens=cu)
    sc = Dk ** -0.5
    y = [f64(t) for t in x]
    want = ref.forward(*y[:4], y[4], None, sc) + ref.backward(*y[:4], y[5], y[4], y[6], None, sc)
    rows = (np.abs(np.repeat(y[0], H, 2)) * np.repeat(want[2][1], H, 2)).sum(3)
    rows = rows + (np.abs(np.repeat(y[1], H, 2)) * np.repeat(want[3][1], H, 2)).sum(3)
    want[5][1][:] += n ** 0.5 * rows.max(1, keepdims=True)
    for name, a, w in zip(("o", "ht", "dq", "dk", "dv", "dg", "dh0"), (o, ht) + tuple(grads), want):
        last = a[1:] if name in ("ht", "dh0") else a[:, T - n:]
        close(last, w, name, n, Dk, Dv, "bf16")
    assert not o[:, :T - n].any() and not ht[0].any()
