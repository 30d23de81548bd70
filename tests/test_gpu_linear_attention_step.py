"""One step of linear attention against a pool of states, on the GPU, against the
formula in 64 bits. Tolerances: a state cell is one product and one sum in fp32
with e^g off by (|g| + 2) 2^-24 relative, which e^g bounds (|g| e^g < 1): 8 *
2^-24 of the magnitudes; o is a sum of Dk products of such cells, (Dk + 16) 2^-24
of theirs, and one rounding to its type, eps / 2."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def m():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import associative_scan_amd as m
    return m


def f64(t):
    return t.double().cpu().numpy()


def make(seed, B, pool, H, Hk, Dk, Dv, dtype="bf16", gate="token"):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    r = lambda *s: torch.randn(s, device=DEV, generator=gen)  # noqa: E731
    dt = TYPES[dtype]
    g = -r(B, H).abs() if gate == "token" else -r(H).abs()
    return r(B, Hk, Dk).to(dt), r(B, Hk, Dk).to(dt), r(B, H, Dv).to(dt), g, r(pool, H, Dk, Dv)


def check(m, x, slots=None, scale=None):
    q, k, v, g, state = x
    before = state.clone()
    s = None if slots is None else torch.tensor(slots, dtype=torch.int32, device=DEV)
    o = m.linear_attention_step(q, k, v, g, state, slots=s, scale=scale)
    B, H, r = v.shape[0], v.shape[1], v.shape[1] // q.shape[1]
    sc = q.shape[2] ** -0.5 if scale is None else scale
    S = f64(before)
    mag = np.abs(S)
    steps = np.zeros(S.shape[0])
    a = np.exp(np.broadcast_to(f64(g), (B, H)))
    Q, K, V = np.repeat(f64(q), r, 1), np.repeat(f64(k), r, 1), f64(v)
    for b in range(B):
        n = b if slots is None else slots[b]
        got = f64(o[b])
        if not 0 <= n < S.shape[0]:
            assert np.all(got == 0)
            continue
        kv = K[b][:, :, None] * V[b][:, None, :]
        S[n] = a[b][:, None, None] * S[n] + kv
        mag[n] = a[b][:, None, None] * mag[n] + np.abs(kv)
        steps[n] += 1
        want = sc * np.einsum("hk,hkv->hv", Q[b], S[n])
        m_o = sc * np.einsum("hk,hkv->hv", np.abs(Q[b]), mag[n])
        tol = (q.shape[2] + 16 + 8 * steps[n]) * 2.0 ** -24 * m_o
        if o.dtype != torch.float32:
            tol = tol + torch.finfo(o.dtype).eps / 2 * np.abs(want) + torch.finfo(o.dtype).tiny
        assert np.all(np.abs(got - want) <= tol), (b, np.max(np.abs(got - want) / tol))
    off = np.abs(f64(state) - S)
    assert np.all(off <= 8 * steps[:, None, None, None] * 2.0 ** -24 * mag), "state"
    return o


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("Dk,Dv", [(8, 8), (64, 64), (128, 128), (40, 72), (72, 40), (128, 8), (8, 128), (104, 120)])
def test_sizes(m, Dk, Dv, dtype):
    check(m, make(Dk + Dv, 3, 3, 4, 2, Dk, Dv, dtype))


def test_slots_padding_and_untouched_states(m):
    """A slot out of range is a row of padding; other states keep their bits."""
    x = make(1, 6, 9, 3, 3, 64, 64)
    before = x[4].clone()
    check(m, x, slots=[8, -1, 0, 5, 9, 1 << 30])
    for n in (1, 2, 3, 4, 6, 7):
        assert torch.equal(x[4][n], before[n])
    x = make(2, 2, 3, 2, 2, 64, 64)
    before = x[4].clone()
    check(m, x, slots=[-1, -5])
    assert torch.equal(x[4], before)


def test_rows_of_one_slot_are_consecutive_steps(m):
    check(m, make(3, 7, 4, 3, 1, 128, 64), slots=[2, 0, 2, 2, 1, 0, -1])
    check(m, make(4, 600, 3, 2, 2, 16, 16), slots=[i % 3 for i in range(600)])
    # the same as one step after the other
    q, k, v, g, state = make(5, 4, 2, 2, 2, 64, 64)
    other = state.clone()
    o = m.linear_attention_step(q, k, v, g, state, slots=torch.tensor([1, 1, 1, 1], dtype=torch.int32, device=DEV))
    for b in range(4):
        s = torch.tensor([1], dtype=torch.int32, device=DEV)
        ob = m.linear_attention_step(q[b:b + 1], k[b:b + 1], v[b:b + 1], g[b:b + 1], other, slots=s)
        assert torch.equal(ob[0], o[b])
    assert torch.equal(state, other)


def test_resets_and_shared_decays(m):
    q, k, v, g, state = make(6, 4, 4, 4, 4, 64, 64, gate="head")
    check(m, (q, k, v, g, state))
    g = torch.full((4, 4), -float("inf"), device=DEV)
    o = m.linear_attention_step(q, k, v, g, state, scale=1.0)
    assert torch.equal(state, k.float()[..., :, None] * v.float()[..., None, :])
    assert torch.isfinite(o).all()


def test_strided_rows(m):
    """Queries, keys and values as views of one projection."""
    q, k, v, g, state = make(7, 5, 5, 4, 4, 64, 64)
    other = state.clone()
    o = m.linear_attention_step(q, k, v, g, state)
    qkv = torch.cat([q, k, v], 1)
    o2 = m.linear_attention_step(qkv[:, :4], qkv[:, 4:8], qkv[:, 8:], g.t().contiguous().t(), other)
    assert torch.equal(o, o2) and torch.equal(state, other)


def test_empty_batch_and_pool(m):
    q, k, v, g, state = make(8, 3, 3, 2, 2, 16, 16)
    before = state.clone()
    o = m.linear_attention_step(q[:0], k[:0], v[:0], g[:0], state)
    assert o.shape == (0, 2, 16) and torch.equal(state, before)
    s = torch.zeros(3, dtype=torch.int32, device=DEV)
    o = m.linear_attention_step(q, k, v, g, state[:0], slots=s)
    assert torch.equal(o, torch.zeros_like(o))


def test_replayed_graph(m):
    """A captured step advances the states by one step at every replay."""
    q, k, v, g, state = make(9, 4, 6, 2, 2, 64, 64)
    s = torch.tensor([5, 0, 3, 1], dtype=torch.int32, device=DEV)
    want = state.clone()
    m.linear_attention_step(q, k, v, g, state.clone(), slots=s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = m.linear_attention_step(q, k, v, g, state, slots=s)
    for i in range(4):
        q.copy_(torch.randn_like(q.float()).to(q.dtype))
        graph.replay()
        w = m.linear_attention_step(q, k, v, g, want, slots=s)
        torch.cuda.synchronize()
        assert torch.equal(o, w) and torch.equal(state, want)


def test_prompt_then_steps(m):
    """A prompt's final state continued token by token gives the whole prompt's outputs:
    both are within their own tolerance of the exact result."""
    import attention_reference as ref
    gen = torch.Generator(device=DEV)
    gen.manual_seed(10)
    r = lambda *s: torch.randn(s, device=DEV, generator=gen)  # noqa: E731
    B, T, P, H, D = 2, 90, 70, 3, 64
    q, k, v = (r(B, T, H, D).bfloat16() for _ in range(3))
    g = -r(B, T, H).abs() * 0.1
    (want, mag), (wh, hm) = ref.forward(f64(q), f64(k), f64(v), f64(g), None, None, 0.125)
    o, state = m.linear_attention_fwd(q[:, :P], k[:, :P], v[:, :P], g[:, :P], scale=0.125)
    outs = [o] + [m.linear_attention_step(q[:, t], k[:, t], v[:, t], g[:, t], state, scale=0.125)[:, None]
                  for t in range(P, T)]
    o = torch.cat(outs, 1)
    fp32 = (8 * T + 2 * D + 256) * 2.0 ** -24
    assert np.all(np.abs(f64(o) - want) <= (fp32 + 2.0 ** -17) * mag + 2.0 ** -8 * np.abs(want))
    assert np.all(np.abs(f64(state) - wh) <= fp32 * hm)


def test_states_past_32_bits(m):
    """A pool of more than 2^32 elements: only the states of the batch are touched."""
    B, H, D = 3, 16, 128
    pool = 2 ** 32 // (H * D * D) + 5
    q, k, v, g, some = make(31, B, B, H, H, D, D)
    state = torch.empty(pool, H, D, D, device=DEV)
    slots = [pool - 1, 0, pool - 3]
    at = torch.tensor(slots, dtype=torch.int32, device=DEV)
    state[at.long()] = some
    state[pool - 2] = 7.0
    o = m.linear_attention_step(q, k, v, g, state, slots=at)
    want = some.clone()
    near = m.linear_attention_step(q, k, v, g, want)
    assert torch.equal(o, near) and torch.equal(state[at.long()], want) and bool((state[pool - 2] == 7.0).all())
