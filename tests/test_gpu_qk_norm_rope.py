"""Per-head norm and rotation of queries and keys on the GPU against the formula in
64 bits. Tolerances: with u = 2^-24, a row's mean of squares is off by (D + 2) u
relative, so r = (mean + eps)^-1/2 by D / 2 + 4 of them; n is a few products on it
and the rotation one sum: (D + 16) u of the magnitudes, plus the output's rounding.
Backward: t = dn w, its mean over D and a difference: 2 (D + 16) u of the
magnitudes. dw is a sum over `rows` products of such: (rows + D + 32) u."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
U = 2.0 ** -24


@pytest.fixture(scope="module")
def m():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import associative_scan_amd as m
    return m


def f64(t):
    return t.double().cpu().numpy()


def tables(n, rot):
    pos = torch.arange(n, dtype=torch.float64)
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    return torch.cos(pos[:, None] * inv).float().to(DEV), torch.sin(pos[:, None] * inv).float().to(DEV)


def rotation(x, c, s, interleaved):
    """x [.., D] rotated by c, s [.., rot / 2], and the same over absolute values."""
    x = x.copy()
    half = c.shape[-1]
    if interleaved:
        a, b = x[..., 0:2 * half:2].copy(), x[..., 1:2 * half:2].copy()
        x[..., 0:2 * half:2], x[..., 1:2 * half:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., :half].copy(), x[..., half:2 * half].copy()
        x[..., :half], x[..., half:2 * half] = a * c - b * s, b * c + a * s
    return x


def spread(x, c, s, interleaved):
    return rotation(np.abs(x), np.abs(c), -np.abs(s), interleaved) if c.shape[-1] == 0 else np.maximum(
        rotation(np.abs(x), np.abs(c), -np.abs(s), interleaved), rotation(np.abs(x), np.abs(c), np.abs(s), interleaved))


def one_side(x, w, c, s, dy, eps, interleaved):
    """y, dx, dw of one side with their magnitudes."""
    x, dy = f64(x), f64(dy)
    D = x.shape[-1]
    w = np.ones(D) if w is None else f64(w)
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n = x * r * w
    dn, dnm = rotation(dy, c, -s, interleaved), spread(dy, c, s, interleaved)
    hat = x * r
    t, tm = dn * w, dnm * np.abs(w)
    mean, mm = (t * hat).mean(-1, keepdims=True), (tm * np.abs(hat)).mean(-1, keepdims=True)
    return ((rotation(n, c, s, interleaved), spread(n, c, s, interleaved)),
            (r * (t - hat * mean), r * (tm + np.abs(hat) * mm)),
            ((dn * hat).sum((0, 1, 2)), (dnm * np.abs(hat)).sum((0, 1, 2))))


def close(got, want, factor, name):
    val, mag = want
    tol = factor * U * mag + 1e-35
    if got.dtype != torch.float32:
        tol = tol + torch.finfo(got.dtype).eps / 2 * np.abs(val) + torch.finfo(got.dtype).tiny
    off = np.abs(f64(got) - val)
    assert np.all(np.isfinite(f64(got))), name
    assert np.all(off <= tol), f"{name}: {np.max(off / tol):.2f} of the tolerance"


def check(m, B, T, Hq, Hk, D, rot, dtype="bf16", wtype=None, interleaved=False, positions="batch", eps=1e-6, seed=0,
          views=False, table=500):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    dt = TYPES[dtype]
    r = lambda *s: torch.randn(s, device=DEV, generator=gen).to(dt)  # noqa: E731
    if views:
        qkv = r(B, T, Hq + 2 * Hk, D)
        q, k = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk]
        dyq, dyk = r(B, Hq, T, D).transpose(1, 2), r(B, Hk, T, D).transpose(1, 2)
    else:
        q, k, dyq, dyk = r(B, T, Hq, D), r(B, T, Hk, D), r(B, T, Hq, D), r(B, T, Hk, D)
    wq = wk = None
    if wtype:
        wq, wk = ((1 + 0.3 * torch.randn(D, device=DEV, generator=gen)).to(TYPES[wtype]) for _ in range(2))
    cos = sin = None
    c = s = np.zeros((B, T, 1, 0))
    pos = None
    if rot:
        cos, sin = tables(table, rot)
        if positions == "batch":
            pos = torch.randint(0, table, (B, T), device=DEV, generator=gen)
        elif positions == "shared":
            pos = torch.randint(0, table, (T,), device=DEV, generator=gen).to(torch.int32)
        at = np.arange(T) if pos is None else pos.cpu().numpy()
        at = np.broadcast_to(at, (B, T))
        c, s = f64(cos)[at][:, :, None], f64(sin)[at][:, :, None]
    args = dict(positions=pos, eps=eps, interleaved=interleaved)
    yq, yk = m.qk_norm_rope_fwd(q, k, wq, wk, cos, sin, **args)
    dq, dk, dwq, dwk = m.qk_norm_rope_bwd(q, k, wq, wk, cos, sin, dyq, dyk, **args)
    for x, w, dy, y, dx, dw, n in ((q, wq, dyq, yq, dq, dwq, "q"), (k, wk, dyk, yk, dk, dwk, "k")):
        wy, wdx, wdw = one_side(x, w, c, s, dy, eps, interleaved)
        close(y, wy, D + 16, n)
        close(dx, wdx, 2 * (D + 16), "d" + n)
        if w is not None:
            close(dw, wdw, B * T * x.shape[2] + D + 32, "dw" + n)
        else:
            assert dw is None


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("D,rot", [(8, 0), (16, 16), (64, 64), (64, 32), (72, 64), (80, 16), (128, 128), (128, 32),
                                   (136, 128), (192, 192), (256, 256), (256, 64), (256, 16)])
def test_sizes(m, D, rot, dtype):
    check(m, 2, 9, 3, 2, D, rot, dtype, wtype=dtype, seed=D)
    check(m, 2, 9, 3, 2, D, rot, dtype, wtype="fp32", seed=D, interleaved=True)


@pytest.mark.parametrize("Hq,Hk", [(1, 1), (4, 1), (5, 3), (12, 12), (7, 2)])
@pytest.mark.parametrize("B,T", [(1, 1), (3, 1), (1, 33), (2, 700)])
def test_rows(m, B, T, Hq, Hk):
    check(m, B, T, Hq, Hk, 128, 64, "bf16", wtype="bf16", seed=T)


def test_many_rows(m):
    """The path with several heads per lane group, and many rows per workgroup in the backward."""
    check(m, 2, 3001, 7, 3, 128, 128, "bf16", wtype="fp32", seed=1)
    check(m, 1, 2500, 6, 1, 64, 64, "fp32", wtype="fp32", seed=2)


@pytest.mark.parametrize("positions", ["batch", "shared", "none"])
def test_positions(m, positions):
    check(m, 3, 40, 2, 2, 64, 64, "fp32", positions=positions)


def test_views_without_weights(m):
    check(m, 2, 50, 4, 2, 128, 128, "bf16", views=True)


def test_zero_rows_and_eps(m):
    """A head of zeros stays zero, with a finite gradient; eps matters next to it."""
    q = torch.zeros(1, 2, 2, 64, device=DEV)
    q[0, 1] = 1e-4
    w = torch.ones(64, device=DEV)
    y, _ = m.qk_norm_rope_fwd(q, q, w, w, eps=1e-5)
    assert torch.equal(y[0, 0], torch.zeros_like(y[0, 0]))
    want = 1e-4 / (1e-8 + 1e-5) ** 0.5
    assert torch.allclose(y[0, 1], torch.full_like(y[0, 1], want), rtol=2e-6)
    dq, dk, dwq, dwk = m.qk_norm_rope_bwd(q, q, w, w, None, None, torch.ones_like(q), torch.ones_like(q), eps=1e-5)
    assert torch.isfinite(dq).all() and torch.isfinite(dwq).all()
    assert torch.allclose(dq[0, 0], torch.full_like(dq[0, 0], 1e-5 ** -0.5), rtol=2e-6)


def test_positions_outside_the_table_are_clamped(m):
    q = torch.randn(1, 4, 1, 64, device=DEV)
    cos, sin = tables(10, 64)
    p = torch.tensor([-5, 0, 10, 1 << 30], dtype=torch.int64, device=DEV)
    y, _ = m.qk_norm_rope_fwd(q, q, None, None, cos, sin, positions=p)
    z, _ = m.qk_norm_rope_fwd(q, q, None, None, cos, sin, positions=p.clamp(0, 9))
    assert torch.equal(y, z)


def test_repeatable(m):
    q, k = torch.randn(2, 900, 6, 128, device=DEV).bfloat16(), torch.randn(2, 900, 2, 128, device=DEV).bfloat16()
    w = torch.rand(128, device=DEV)
    cos, sin = tables(900, 128)
    first = m.qk_norm_rope_bwd(q, k, w, w, cos, sin, q, k)
    for _ in range(3):
        for a, b in zip(first, m.qk_norm_rope_bwd(q, k, w, w, cos, sin, q, k)):
            assert torch.equal(a, b)


def test_empty(m):
    q = torch.zeros(2, 0, 3, 64, device=DEV)
    w = torch.ones(64, device=DEV)
    assert m.qk_norm_rope_fwd(q, q, w, w)[0].shape == q.shape
    assert torch.equal(m.qk_norm_rope_bwd(q, q, w, w, None, None, q, q)[2], torch.zeros_like(w))


def test_offsets_past_32_bits(m):
    """Rows of more than 2^31 elements: the last tokens against the same ones by themselves."""
    T, n, H, D = 2 ** 17 + 9, 9, 128, 128
    assert (T - n) * H * D >= 2 ** 31
    gen = torch.Generator(device=DEV)
    gen.manual_seed(3)
    q = torch.zeros(1, T, H, D, dtype=torch.bfloat16, device=DEV)
    k = torch.zeros(1, T, 1, D, dtype=torch.bfloat16, device=DEV)
    for x in (q, k):
        x[:, T - n:] = torch.randn(1, n, x.shape[2], D, device=DEV, generator=gen).bfloat16()
    w = torch.rand(D, device=DEV, generator=gen)
    near = [x[:, T - n:].contiguous() for x in (q, k)]
    for a, b in zip(m.qk_norm_rope_fwd(q, k, w, w), m.qk_norm_rope_fwd(*near, w, w)):
        assert torch.equal(a[:, T - n:], b) and not a[:, :T - n].any()
    far, by = m.qk_norm_rope_bwd(q, k, w, w, None, None, q, k), m.qk_norm_rope_bwd(*near, w, w, None, None, *near)
    for a, b in zip(far[:2], by[:2]):
        assert torch.equal(a[:, T - n:], b) and not a[:, :T - n].any()
