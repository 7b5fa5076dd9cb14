"""Row kernels of the sequence block on batches of several rows a thread: each loops over its rows, the next row held
in registers while this one is worked on (GPU).

The forward norm launches at most 32 blocks per SM, the lookup and the norm's backward pass at most 8.  The sizes
follow from the SM count with room above those factors, so that most blocks take two or three turns.  Every output row
depends on its input row alone, so a batch that repeats a few rows must repeat their results bit for bit; those few are
compared with 64 bits first, with the bounds of the arithmetic: a sum of D squares within D * 2^-24 of itself, one
rounding of the result.
"""
import pytest
import torch

from jagged_embedding_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16, E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
U = 2.0 ** -24


def _sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def _turns(blocks_per_sm, rows_per_block):
    """Rows for 2.2 turns of the largest grid."""
    return int(2.2 * blocks_per_sm * _sms() * rows_per_block) + 5


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def _rows_a_block(D, dt):
    """Rows that a block of 256 threads holds: a thread takes 16 bytes of a row where the width allows it."""
    vec = (4 if dt == F32 else 8)
    chunks = -(-D // (vec if D % vec == 0 else 1))
    return next((256 // g for g, most in ((8, 8), (16, 16), (32, 64)) if chunks <= most), 1)


@pytest.mark.parametrize("D,dt,bits8,res", [
    (64, BF16, True, "x"), (64, F32, False, None), (128, BF16, False, "res"), (512, BF16, True, "new"),
    (520, F32, False, None), (520, BF16, True, "res"), (1001, BF16, False, "new"), (2056, BF16, True, "x"),
    (2056, F32, True, None), (8192, BF16, False, "x"), (8192, F32, True, "new"), (8191, BF16, True, "res")])
def test_norm_over_several_rows_a_thread(D, dt, bits8, res):
    T, few, eps = _turns(32, _rows_a_block(D, dt)), 29, 1e-5
    g = _gen(D)
    level = torch.exp(2 * torch.randn(few, 1, generator=g, device=DEV))
    x, r = ((torch.randn(few, D, generator=g, device=DEV) * level).to(dt) for _ in range(2))
    gamma = 1 + 0.2 * torch.randn(D, generator=g, device=DEV)
    y_dtype = E4M3 if bits8 else dt
    y, sc, h, rstd = B.fs_rmsnorm(x, gamma, eps, res=r if res else None, y_dtype=y_dtype)
    hh = (x.float() + r.float()).to(dt) if res else x
    assert not res or torch.equal(h, hh)
    hd = hh.double()
    inv = ((hd * hd).mean(1, keepdim=True) + eps) ** -0.5
    ref = hd * inv * gamma.double()
    rel = (D / 2 + 10) * U
    got = y.float().double() * sc.double()[:, None] if bits8 else y.double()
    # e4m3: half a step of 2^-3 relative, or of 2^-9 scales below 2^-6; bf16: 2^-8 relative
    tol = ref.abs() * (rel + (2.0 ** -4 + 2.0 ** -20 if bits8 else 2.0 ** -8 if dt == BF16 else 2 * U))
    if bits8:
        tol = tol + sc.double()[:, None] * 2.0 ** -10
    assert bool(((got - ref).abs() <= tol).all()) and bool(((rstd.double() - inv[:, 0]).abs() <= rel * inv[:, 0]).all())

    at = torch.randint(0, few, (T,), generator=g, device=DEV)
    X, R = x[at], (r[at] if res else None)
    out = {"x": X, "res": R}.get(res)
    Y, SC, H, RSTD = B.fs_rmsnorm(X, gamma, eps, res=R, sum_out=out, y_dtype=y_dtype)
    assert _same_bits(Y, y.view(torch.uint8)[at]) and _same_bits(RSTD, rstd[at])
    assert not bits8 or _same_bits(SC, sc[at])
    assert not res or _same_bits(H, h[at])


@pytest.mark.parametrize("D,dt", [(520, BF16), (2056, BF16), (2056, F32), (4096, BF16), (8191, BF16), (8192, F32),
                                  (512, F32), (300, BF16)])
@pytest.mark.parametrize("with_sum", [False, True])
def test_norm_backward_over_several_rows_a_thread(D, dt, with_sum):
    T, few = max(_turns(8, _rows_a_block(D, dt)), 100 * _rows_a_block(D, dt)), 23
    g = _gen(D + 1)
    level = torch.exp(torch.randn(few, 1, generator=g, device=DEV))
    h, dy, ds = ((torch.randn(few, D, generator=g, device=DEV) * level).to(dt) for _ in range(3))
    gamma = 1 + 0.2 * torch.randn(D, generator=g, device=DEV)
    rstd = ((h.double() ** 2).mean(1) + 1e-6).rsqrt().float()
    r = rstd.double()[:, None]
    n, w = h.double() * r, dy.double() * gamma.double()
    dot = (w * n).mean(1, keepdim=True)
    ref = r * (w - n * dot) + (ds.double() if with_sum else 0)
    size = r * (w.abs() + n.abs() * (dot.abs() + D * (w * n).abs().mean(1, keepdim=True))) + (ds.double().abs() if with_sum else 0)
    tol = 8 * U * size + (ref.abs() * 2.0 ** -8 if dt == BF16 else 0)
    at = torch.randint(0, few, (T,), generator=g, device=DEV)
    A, Y = h[at], dy[at]
    dh, dgamma = B.fs_rmsnorm_backward(Y, A, gamma, rstd[at], dsum=ds[at] if with_sum else None,
                                       dh=Y if with_sum else None)  # (in place of dy, once)
    first = torch.stack([(at == k).nonzero()[0, 0] for k in range(few)])
    assert bool(((dh[first].double() - ref).abs() <= tol).all())
    assert _same_bits(dh, dh[first][at])  # every row as its first copy
    times = torch.bincount(at, minlength=few).double()[:, None]
    total, mag = (dy.double() * n * times).sum(0), (dy.double() * n * times).abs().sum(0)
    # at most T / SMs rows a thread one after another, a block's 32 shares, then an eighth of at most 8 blocks per SM
    depth = T / _sms() + 32 + _sms() + 8 + 4
    assert bool(((dgamma.double() - total).abs() <= depth * U * mag).all())


@pytest.mark.parametrize("table_dtype,out_dtype", [(F32, F32), (BF16, BF16), (BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("D", [32, 64, 128, 7])
def test_lookup_over_several_rows_a_thread(D, table_dtype, out_dtype):
    T, R = _turns(8, 256), 3000
    g = _gen(D)
    table = torch.randn(R, D, generator=g, device=DEV).to(table_dtype)
    ids = torch.randint(0, R, (T,), generator=g, device=DEV)
    ids[T // 2], ids[T - 1] = R, -1
    out, err = B.fs_emb_lookup_scaled(table, ids, 1.25, out_dtype=out_dtype)
    assert int(err) == 2
    good = (ids >= 0) & (ids < R)
    want = (table[ids.clamp(0, R - 1)].float() * 1.25).to(out_dtype) * good[:, None]
    assert torch.equal(out, want)
