"""Refusals of the linear attention and query/key norm calls, on the host: the
binding's own checks on stand-ins for GPU tensors, and the C ABI's on its structs."""
import struct

import pytest
import torch


@pytest.fixture(scope="module")
def m():
    import associative_scan_amd as m
    return m


class OnGpu(torch.Tensor):
    """A CPU tensor that says it is on the GPU (no kernel is reached with it)."""

    @staticmethod
    def __new__(cls, t):
        return torch.Tensor._make_subclass(cls, t)

    @property
    def is_cuda(self):
        return True


def t(*shape, dtype=torch.bfloat16):
    return OnGpu(torch.zeros(shape, dtype=dtype))


def call(**change):
    x = dict(q=t(2, 5, 2, 16), k=t(2, 5, 2, 16), v=t(2, 5, 4, 24), g=t(2, 5, 4, dtype=torch.float32))
    x.update(change)
    return x


@pytest.mark.parametrize("change,text", [
    (dict(k=t(2, 5, 2, 24)), r"q and k must be"),
    (dict(v=t(2, 6, 4, 24)), r"q and k must be"),
    (dict(q=t(2, 5, 16), k=t(2, 5, 16)), r"q and k must be"),
    (dict(v=t(2, 5, 3, 24), g=t(3, dtype=torch.float32)), "multiple of the number of key heads"),
    (dict(v=t(2, 5, 0, 24)), "multiple of the number of key heads"),
    (dict(k=t(2, 5, 2, 16, dtype=torch.float16)), "same dtype"),
    (dict(q=t(2, 5, 2, 16, dtype=torch.float64), k=t(2, 5, 2, 16, dtype=torch.float64)), "float32, bfloat16 and float16"),
    (dict(q=t(2, 5, 2, 12), k=t(2, 5, 2, 12)), "Dk must be a multiple of 8"),
    (dict(v=t(2, 5, 4, 136)), "Dv must be a multiple of 8 up to 128"),
    (dict(g=t(2, 5, 4)), "float32"),
    (dict(g=t(2, 5, 2, dtype=torch.float32)), r"g must be \[B, T, H\]"),
    (dict(cu_seqlens=t(3, dtype=torch.int32)), "B = 1"),
    (dict(cu_seqlens=t(3, dtype=torch.int64)), "int32"),
    (dict(h0=t(2, 4, 16, 24)), "fp32"),
    (dict(h0=t(1, 4, 16, 24, dtype=torch.float32)), r"h0 must be \[N, H, Dk, Dv\]"),
    (dict(q=OnGpu(torch.zeros(2, 5, 16, 2, dtype=torch.bfloat16).transpose(2, 3))), "last axis must be contiguous"),
    (dict(v=OnGpu(torch.zeros(2, 5, 4, 28, dtype=torch.bfloat16)[..., :24])), "16-byte aligned"),
    (dict(v=OnGpu(torch.zeros(2 * 5 * 4 * 24 + 4, dtype=torch.bfloat16)[4:].view(2, 5, 4, 24))), "16-byte aligned"),
])
def test_attention_refuses(m, change, text):
    x = call(**change)
    with pytest.raises(ValueError, match=text):
        m.linear_attention_fwd(**x)
    do = x.pop("do", None) or t(*x["v"].shape)
    with pytest.raises(ValueError, match=text):
        m.linear_attention_bwd(**x, do=do)


def test_attention_refuses_host_tensors_and_bad_gradients(m):
    x = call()
    with pytest.raises(ValueError, match="GPU tensor"):
        m.linear_attention_fwd(**{**x, "q": torch.zeros(2, 5, 2, 16, dtype=torch.bfloat16)})
    for do in (t(2, 5, 4, 16), t(2, 5, 4, 24, dtype=torch.float32)):
        with pytest.raises(ValueError, match="do must have"):
            m.linear_attention_bwd(**x, do=do)
    with pytest.raises(ValueError, match="dht must be"):
        m.linear_attention_bwd(**x, do=t(2, 5, 4, 24), dht=t(2, 4, 24, 16, dtype=torch.float32))


@pytest.mark.parametrize("change,text", [
    (dict(q=t(3, 1, 2, 16), k=t(3, 1, 2, 16)), r"\[B, Hk, Dk\]"),
    (dict(v=t(2, 4, 24)), r"\[B, Hk, Dk\]"),
    (dict(g=t(3, 2, dtype=torch.float32)), r"g must be \[B, H\]"),
    (dict(g=t(3, 4)), "float32"),
    (dict(v=t(3, 3, 24)), "multiple of the number of key heads"),
    (dict(state=t(3, 4, 24, 16, dtype=torch.float32)), "state must be"),
    (dict(state=t(4, 16, 24, dtype=torch.float32)), "state must be"),
    (dict(state=t(3, 4, 16, 24)), "fp32"),
    (dict(state=OnGpu(torch.zeros(3, 4, 24, 16).transpose(2, 3))), "contiguous"),
    (dict(state=t(2, 4, 16, 24, dtype=torch.float32)), "as many states"),
    (dict(slots=t(3, dtype=torch.int64)), "int32"),
    (dict(slots=t(2, dtype=torch.int32)), "int32"),
])
def test_step_refuses(m, change, text):
    x = dict(q=t(3, 2, 16), k=t(3, 2, 16), v=t(3, 4, 24), g=t(3, 4, dtype=torch.float32),
             state=t(3, 4, 16, 24, dtype=torch.float32))
    x.update(change)
    with pytest.raises(ValueError, match=text):
        m.linear_attention_step(**x)


F = torch.float32


@pytest.mark.parametrize("change,text", [
    (dict(k=t(2, 5, 2, 16)), "q must be"),
    (dict(k=t(2, 6, 2, 32)), "q must be"),
    (dict(k=t(2, 5, 0, 32)), "both need heads"),
    (dict(k=t(2, 5, 2, 32, dtype=F)), "same dtype"),
    (dict(q=t(2, 5, 4, 36), k=t(2, 5, 2, 36)), "multiple of 8 up to 256"),
    (dict(q=t(2, 5, 4, 264), k=t(2, 5, 2, 264)), "multiple of 8 up to 256"),
    (dict(q_weight=t(32)), "both weights or neither"),
    (dict(q_weight=t(16), k_weight=t(16)), r"\[D\]"),
    (dict(q_weight=t(32), k_weight=t(32, dtype=F)), "same dtype"),
    (dict(cos=t(9, 16, dtype=F)), "both cos and sin"),
    (dict(cos=t(9, 16), sin=t(9, 16)), "fp32"),
    (dict(cos=t(9, 16, dtype=F), sin=t(8, 16, dtype=F)), "one shape"),
    (dict(cos=t(0, 16, dtype=F), sin=t(0, 16, dtype=F)), "at least one position"),
    (dict(cos=t(9, 4, dtype=F), sin=t(9, 4, dtype=F)), "multiple of 16"),
    (dict(cos=t(9, 24, dtype=F), sin=t(9, 24, dtype=F)), "up to the head size"),
    (dict(positions=t(5, dtype=F)), "int32 or int64"),
    (dict(positions=t(2, dtype=torch.int64)), "positions must be"),
    (dict(positions=t(5, 2, dtype=torch.int32)), "positions must be"),
    (dict(eps=-1.0), "eps"),
])
def test_norm_refuses(m, change, text):
    x = dict(q=t(2, 5, 4, 32), k=t(2, 5, 2, 32))
    x.update(change)
    with pytest.raises(ValueError, match=text):
        m.qk_norm_rope_fwd(**x)


# the C ABI on its own: every refusal comes before any HIP call
ATT, HEADS, NORM = struct.Struct("@qqiiiiPif3q"), struct.Struct("@P3q"), struct.Struct("@qqiiiiifPPqPiii4x")
P = 1 << 20  # an address that nothing reads


def problem(B=2, T=5, H=4, Hk=2, Dk=16, Dv=24, cu=0, nseg=2, scale=1.0, gs=(20, 4, 1)):
    return ATT.pack(B, T, H, Hk, Dk, Dv, cu, nseg, scale, *gs)


def test_abi_sizes_its_workspaces(m):
    ws = m.lib.linear_attention_workspace_bytes
    assert ws(problem(), 1, 0) > 0 and ws(problem(), 0, 1) > 0 and ws(problem(), 1, 2) == 0 and ws(problem(), 3, 0) == 0
    big = problem(B=1, T=65536, nseg=1, Dk=128, Dv=128)
    assert ws(big, 1, 0) > 65536 and ws(big, 1, 1) > ws(big, 1, 0)
    for bad in (problem(B=0), problem(T=0), problem(T=1 << 31), problem(H=3), problem(Hk=0), problem(Dk=12),
                problem(Dk=136), problem(Dv=0), problem(nseg=1), problem(B=2, cu=P), problem(B=1, cu=P + 2, nseg=1),
                problem(B=1, cu=P, nseg=0), problem(B=1 << 23, nseg=1 << 23)):
        assert ws(bad, 1, 0) == 0
    nb = m.lib.qk_norm_rope_workspace_bytes
    assert nb(norm()) > 0 and nb(norm(D=12)) == 0


INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
ROWS = HEADS.pack(P, 160, 32, 16)


def test_abi_refuses_attention(m):
    f = m.lib.linear_attention_fwd

    def fwd(prob=None, dtype=1, q=ROWS, k=ROWS, v=ROWS, g=P, h0=0, o=P, ht=0, ws=0, n=0):
        return f(prob or problem(), dtype, q, k, v, g, h0, o, ht, ws, n, None)

    assert fwd(prob=problem(H=3)) == INVALID and fwd(prob=problem(Dk=20)) == UNSUPPORTED
    assert fwd(dtype=3) == UNSUPPORTED and f(None, 1, ROWS, ROWS, ROWS, P, 0, P, 0, 0, 0, None) == INVALID
    for bad in (None, HEADS.pack(0, 0, 0, 0), HEADS.pack(P + 8, 160, 32, 16), HEADS.pack(P, 160, 33, 16),
                HEADS.pack(P, -160, 32, 16)):
        assert fwd(q=bad) == INVALID and fwd(k=bad) == INVALID and fwd(v=bad) == INVALID
    assert fwd(v=HEADS.pack(P, 160, 1 << 24, 16)) == UNSUPPORTED
    assert fwd(g=0) == INVALID and fwd(g=P + 2) == INVALID and fwd(o=0) == INVALID and fwd(o=P + 8) == INVALID
    assert fwd(h0=P + 8) == INVALID and fwd(ht=P + 4) == INVALID
    assert fwd(prob=problem(B=1, T=1 << 30, H=64, Hk=1, nseg=1 << 20, cu=P)) == UNSUPPORTED
    big = problem(B=1, T=65536, nseg=1)
    need = m.lib.linear_attention_workspace_bytes(big, 1, 0)
    assert fwd(prob=big) == WORKSPACE and fwd(prob=big, ws=P + 8, n=need) == WORKSPACE
    assert fwd(prob=big, ws=P, n=need - 1024) == WORKSPACE


def test_abi_refuses_backward_and_step(m):
    f = m.lib.linear_attention_bwd

    def bwd(dO=ROWS, dq=P, dk=P, dv=P, dg=P, dh0=P, dht=0, ws=P, n=1 << 40, dtype=1):
        return f(problem(), dtype, ROWS, ROWS, ROWS, P, dO, 0, dht, dq, dk, dv, dg, 0, dh0, ws, n, None)

    assert bwd(dO=None) == INVALID and bwd(dO=HEADS.pack(P + 2, 0, 0, 0)) == INVALID
    for n in ("dq", "dk", "dv"):
        assert bwd(**{n: 0}) == INVALID and bwd(**{n: P + 8}) == INVALID
    assert bwd(dg=P + 2) == INVALID and bwd(dh0=P + 8) == INVALID and bwd(dht=P + 8) == INVALID
    assert bwd(ws=0) == WORKSPACE and bwd(n=100) == WORKSPACE and bwd(dtype=7) == UNSUPPORTED
    s = m.lib.linear_attention_step

    def step(prob=None, q=ROWS, g=P, slots=P, pool=4, state=P, o=P, dtype=1):
        return s(prob or problem(T=1), dtype, q, ROWS, ROWS, g, slots, pool, state, o, None)

    assert step(prob=problem(T=2)) == INVALID and step(prob=problem(B=1, T=1, nseg=1, cu=P)) == INVALID
    assert step(pool=0) == INVALID and step(slots=0, pool=1) == INVALID and step(slots=P + 2) == INVALID
    assert step(state=0) == INVALID and step(state=P + 8) == INVALID and step(o=0) == INVALID and step(g=0) == INVALID
    assert step(q=HEADS.pack(P + 4, 0, 0, 0)) == INVALID and step(dtype=-1) == UNSUPPORTED


def norm(B=2, T=5, Hq=4, Hk=2, D=32, rot=16, il=0, eps=1e-6, cos=P, sin=P, table=9, pos=0, p64=0, per=0, wt=0):
    return NORM.pack(B, T, Hq, Hk, D, rot, il, eps, cos, sin, table, pos, p64, per, wt)


def test_abi_refuses_norm(m):
    f = m.lib.qk_norm_rope_fwd

    def fwd(p=None, dtype=1, q=ROWS, k=ROWS, wq=0, wk=0, yq=P, yk=P):
        return f(p or norm(), dtype, q, k, wq, wk, yq, yk, None)

    for p in (norm(B=0), norm(T=0), norm(Hq=0), norm(Hk=0), norm(rot=48), norm(rot=-16), norm(cos=0), norm(sin=P + 4),
              norm(table=0), norm(pos=P + 2), norm(pos=P + 4, p64=1), norm(eps=-1.0), norm(eps=float("nan"))):
        assert fwd(p) == INVALID
    for p in (norm(D=36), norm(D=264), norm(rot=8), norm(wt=3), norm(T=1 << 26), norm(B=1 << 40), norm(B=1 << 20, T=1 << 20)):
        assert fwd(p) == UNSUPPORTED
    assert fwd(dtype=5) == UNSUPPORTED and fwd(q=None) == INVALID and fwd(k=HEADS.pack(P + 1, 0, 0, 0)) == INVALID
    assert fwd(wq=P + 2) == INVALID and fwd(yq=0) == INVALID and fwd(yk=P + 8) == INVALID
    b = m.lib.qk_norm_rope_bwd

    def bwd(dyq=ROWS, dq=P, dwq=P, ws=P, n=1 << 30):
        return b(norm(), 1, ROWS, ROWS, P, P, dyq, ROWS, dq, P, dwq, P, ws, n, None)

    assert bwd(dyq=None) == INVALID and bwd(dq=0) == INVALID and bwd(dwq=P + 2) == INVALID
    assert bwd(ws=0) == WORKSPACE and bwd(n=16) == WORKSPACE


def test_ops_are_registered_with_fake_kernels(m):
    """Shapes and dtypes of the ops on meta tensors, as a traced program sees them."""
    e = lambda *s, dtype=torch.bfloat16: torch.empty(s, dtype=dtype, device="meta")  # noqa: E731
    q, k, v, g = e(1, 50, 2, 16), e(1, 50, 2, 16), e(1, 50, 4, 24), e(1, 50, 4, dtype=F)
    cu = e(4, dtype=torch.int32)
    o, ht = torch.ops.mscan.linear_attention(q, k, v, g, None, cu, 1.0)
    assert o.shape == v.shape and o.dtype == v.dtype and ht.shape == (3, 4, 16, 24) and ht.dtype == F
    dq, dk, dv, dg, dh0 = torch.ops.mscan.linear_attention_backward(q, k, v, g, o, None, None, cu, 1.0, True, False)
    assert dq.shape == q.shape and dv.dtype == v.dtype and dg.shape == g.shape and dh0.numel() == 0
    y = torch.ops.mscan.linear_attention_step(q[0], k[0], v[0], g[0], e(50, 4, 16, 24, dtype=F), None, 1.0)
    assert y.shape == (50, 4, 24)
    a, b = torch.ops.mscan.qk_norm_rope(q, k, None, None, None, None, None, 1e-6, False)
    assert a.shape == q.shape and b.dtype == k.dtype


def test_tables_get_no_gradient(m):
    q, t = torch.zeros(1, 2, 1, 16), torch.zeros(4, 8)
    for cos, sin, name in ((t.clone().requires_grad_(), t, "cos"), (t, t.clone().requires_grad_(), "sin")):
        with pytest.raises(ValueError, match=name):
            m.qk_norm_rope(q, q, cos=cos, sin=sin)
