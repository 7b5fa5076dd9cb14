"""Root-mean-square norm with the residual's addition, its 8-bit output and its
backward pass against the formulas in 64 bits (GPU).

Tolerances, from the arithmetic: a sum of D squares in fp32 is within D * 2^-24
of itself (all terms positive), so r is within (D / 2 + 4) * 2^-24 relative, y
within that plus the output's half ulp (2^-9 for bf16, taken as 2^-8).  The
dot product of the backward pass is within D * 2^-24 * sum |w n| of itself.
8 bits: q lies within half an e4m3 step of y / scale (2^-4 relative, 2^-10
absolute in the subnormal range), or one ulp of the quotient further where the
fp32 quotient rounds across the middle.
"""
import pytest
import torch

from jagged_embedding_gb300 import binding as B
from tests.helpers import Guarded

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16, E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
U = 2.0 ** -24


def _inputs(T, D, dt, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    level = torch.exp(2 * torch.randn(T, 1, generator=g, device=DEV))
    n = lambda: (torch.randn(T, D, generator=g, device=DEV) * level).to(dt)  # noqa: E731
    return n(), n(), 1 + 0.2 * torch.randn(D, generator=g, device=DEV), g


WIDTHS = [1, 7, 8, 64, 100, 128, 256, 264, 512, 520, 1000, 1024, 2048, 2056, 4096, 8191, 8192]


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("bits8", [False, True])
@pytest.mark.parametrize("with_res", [False, True])
@pytest.mark.parametrize("D", WIDTHS)
def test_norm(dt, bits8, with_res, D):
    T = 37 if D > 300 else 301
    eps = 1e-5
    x, res, gamma, _ = _inputs(T, D, dt, D)
    y, rstd = Guarded((T, D), E4M3 if bits8 else dt), Guarded(T, F32)
    sc = Guarded(T, F32) if bits8 else None
    h_out = Guarded((T, D), dt) if with_res else None
    B.fs_rmsnorm(x, gamma, eps, res=res if with_res else None, sum_out=h_out.t if with_res else None, y=y.t,
                 y_scale=sc.t if bits8 else None, rstd=rstd.t)
    for g in (y, rstd, sc, h_out):
        if g is not None:
            g.check()
    h = x
    if with_res:
        h = (x.float() + res.float()).to(dt)
        assert torch.equal(h_out.t, h)
    h = h.double()
    r = ((h * h).mean(1) + eps) ** -0.5
    rel = (D / 2 + 4) * U
    assert bool(((rstd.t.double() - r).abs() <= rel * r).all())
    ref = h * r[:, None] * gamma.double()
    if not bits8:
        tol = ref.abs() * (rel + 4 * U + (2.0 ** -8 if dt == BF16 else 0))
        assert bool(((y.t.double() - ref).abs() <= tol).all())
        return
    top = ref.abs().amax(1) / 448
    assert bool(((sc.t.double() - top).abs() <= top * (rel + 6 * U)).all())
    z = ref / top[:, None]
    got = y.t.float().double()
    assert bool(torch.isfinite(got).all()) and bool((got.abs().amax(1) == 448).all())
    step = torch.clamp(2.0 ** (torch.floor(torch.log2(z.abs().clamp(min=2.0 ** -6))) - 3), min=2.0 ** -9)
    assert bool(((got - z).abs() <= step * 0.5 + z.abs() * (2 * rel + 16 * U)).all())


def test_norm_of_zero_rows_and_non_finite_values():
    x = torch.randn(6, 64, device=DEV)
    x[1] = 0
    x[2, 5] = float("nan")
    x[3, 7] = float("inf")
    x[4] = 1e30  # the squares overflow
    g = torch.ones(64, device=DEV)
    y, _, _, rstd = B.fs_rmsnorm(x, g, 1e-6)
    assert not y[1].any() and bool(torch.isfinite(y[0]).all()) and bool(torch.isfinite(y[5]).all())
    assert bool(y[2].isnan().all()) and bool(y[3, 7].isnan()) and not y[4].any()
    q, sc, _, _ = B.fs_rmsnorm(x, g, 1e-6, y_dtype=E4M3)
    assert float(sc[1]) == 0 and not q[1].float().any()
    assert bool(sc[2].isnan()) and bool(sc[3].isnan()) and bool(torch.isfinite(q[0].float()).all())
    y, _, _, rstd = B.fs_rmsnorm(torch.zeros(2, 64, device=DEV), g, 0.0)  # eps = 0 on a zero row: 0 * inf
    assert bool(y.isnan().all()) and bool(rstd.isinf().all())


def test_norm_in_place_and_unaligned():
    T, D = 77, 64
    x, res, gamma, _ = _inputs(T, D, F32, 1)
    want = B.fs_rmsnorm(x, gamma, 1e-6, res=res)
    for target in ("x", "res"):
        a, b = x.clone(), res.clone()
        y, _, h, _ = B.fs_rmsnorm(a, gamma, 1e-6, res=b, sum_out=a if target == "x" else b)
        assert torch.equal(h, want[2]) and torch.equal(y, want[0])
    u = torch.empty(T * D + 1, device=DEV)[1:].view(T, D).copy_(x)
    y, _, _, _ = B.fs_rmsnorm(u, gamma, 1e-6)
    ref = x.double() * ((x.double() ** 2).mean(1, keepdim=True) + 1e-6) ** -0.5 * gamma.double()
    assert bool(((y.double() - ref).abs() <= ref.abs() * (D + 8) * U).all())


def test_norm_of_no_rows():
    x = torch.empty(0, 64, device=DEV)
    g = torch.ones(64, device=DEV)
    y, _, _, rstd = B.fs_rmsnorm(x, g, 1e-6)
    assert y.shape == (0, 64)
    dh, dg = B.fs_rmsnorm_backward(x, x, g, rstd, dgamma=torch.full((64,), 3.0, device=DEV))
    assert dh.shape == (0, 64) and not dg.any()


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("with_sum", [False, True])
@pytest.mark.parametrize("D", WIDTHS)
def test_norm_backward(dt, with_sum, D):
    T = 33 if D > 300 else 1301
    h, dy, gamma, g = _inputs(T, D, dt, 5 * D)
    dsum = torch.randn(T, D, generator=g, device=DEV).to(dt) if with_sum else None
    rstd = ((h.double() ** 2).mean(1) + 1e-6).rsqrt().float()
    dh, dgm = Guarded((T, D), dt), Guarded(D, F32)
    ws = Guarded((B.rmsnorm_backward_workspace_size(T, D) + 15) // 16 * 16, torch.uint8)
    B.fs_rmsnorm_backward(dy, h, gamma, rstd, dsum=dsum, dh=dh.t, dgamma=dgm.t, ws=ws.t)
    for x in (dh, dgm, ws):
        x.check()
    r = rstd.double()[:, None]
    n, w = h.double() * r, dy.double() * gamma.double()
    dot = (w * n).mean(1, keepdim=True)
    ref = r * (w - n * dot) + (dsum.double() if with_sum else 0)
    size = r * (w.abs() + n.abs() * (dot.abs() + D * (w * n).abs().mean(1, keepdim=True))) + (
        dsum.double().abs() if with_sum else 0)
    tol = 8 * U * size + (ref.abs() * 2.0 ** -8 if dt == BF16 else 0)
    assert bool(((dh.t.double() - ref).abs() <= tol).all())
    ref, mag = (dy.double() * n).sum(0), (dy.double() * n).abs().sum(0)
    assert bool(((dgm.t.double() - ref).abs() <= (min(T, 64) + 8) * U * mag).all())
    again = B.fs_rmsnorm_backward(dy, h, gamma, rstd, dsum=dsum)
    assert torch.equal(again[0], dh.t) and torch.equal(again[1], dgm.t)


def test_norm_backward_in_place():
    h, dy, gamma, g = _inputs(99, 128, BF16, 3)
    dsum = torch.randn(99, 128, generator=g, device=DEV).to(BF16)
    rstd = ((h.float() ** 2).mean(1) + 1e-6).rsqrt()
    want = B.fs_rmsnorm_backward(dy, h, gamma, rstd, dsum=dsum)
    for k in range(2):
        a, b = dy.clone(), dsum.clone()
        dh, dg = B.fs_rmsnorm_backward(a, h, gamma, rstd, dsum=b, dh=(a, b)[k])
        assert torch.equal(dh, want[0]) and torch.equal(dg, want[1])


def test_norm_backward_equals_differences():
    """Central differences of sum(dy * norm(x + res)) along random directions, the norm in 64 bits."""
    T, D, eps = 9, 48, 1e-4
    x, dy, gamma, g = _inputs(T, D, F32, 11)
    y, _, _, rstd = B.fs_rmsnorm(x, gamma, eps)
    dh, dg = B.fs_rmsnorm_backward(dy, x, gamma, rstd)

    def loss(a, w):
        return float((dy.double() * a * ((a * a).mean(1, keepdim=True) + eps) ** -0.5 * w).sum())

    a, w = x.double(), gamma.double()
    for _ in range(4):
        V = torch.randn(T, D, generator=g, device=DEV).double() * a.abs().mean(1, keepdim=True)
        Z = torch.randn(D, generator=g, device=DEV).double()
        slope = (loss(a + 1e-5 * V, w + 1e-5 * Z) - loss(a - 1e-5 * V, w - 1e-5 * Z)) / 2e-5
        mine = float((dh.double() * V).sum() + (dg.double() * Z).sum())
        assert abs(slope - mine) < 1e-4 * float((dh.double() * V).abs().sum() + (dg.double() * Z).abs().sum())


def test_norm_long_batch_on_another_stream():
    T, D = 100_003, 64
    x, dy, gamma, _ = _inputs(T, D, BF16, 8)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        y, _, _, rstd = B.fs_rmsnorm(x, gamma, 1e-6)
        dh, dg = B.fs_rmsnorm_backward(dy, x, gamma, rstd)
    s.synchronize()
    n = x.double() * rstd.double()[:, None]
    mag = (dy.double() * n).abs().sum(0)
    # each thread of the pass adds at most ceil(T / rows in flight) terms, then the block and the blocks
    assert bool(((dg.double() - (dy.double() * n).sum(0)).abs() <= 256 * U * mag).all())
    assert bool(((y.double() - n * gamma.double()).abs() <= (n * gamma.double()).abs() * 2.0 ** -8).all())
