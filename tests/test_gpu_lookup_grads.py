"""Scaled lookup and its row gradients against a plain computation in 64 bits (GPU).

Tolerances, from the arithmetic: the lookup is one fp32 product rounded once to
the output's type, so it equals the same product of torch, bit for bit.  A row
gradient is an fp32 sum of m terms in a fixed tree of runs of at most 128
(within a tile), then of tiles; its error stays below 2^-24 * (128 + tiles' depth)
* sum |g| for any order, taken here as 2^-24 * min(m, 256) * sum |g|; a bf16
result adds half an ulp, 2^-9 of the value (2^-8 covers it), the final product
with the scale 2^-24.
"""
import numpy as np
import pytest
import torch

from jagged_embedding_gb300 import binding as B
from tests.helpers import Guarded

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16


def _ids(kind, T, R, seed):
    r = np.random.default_rng(seed)
    if kind == "zipf":
        ids = np.minimum(np.exp(r.random(T) * np.log(R + 1)).astype(np.int64) - 1, R - 1)
    elif kind == "one":
        ids = np.full(T, R - 1)
    elif kind == "distinct":
        ids = r.permutation(R)[:T]
    elif kind == "ascending":
        ids = np.sort(r.integers(0, R, T))
    else:
        ids = r.integers(0, R, T)
    return torch.from_numpy(np.ascontiguousarray(ids.astype(np.int64))).to(DEV)


@pytest.mark.parametrize("table_dtype", [F32, BF16])
@pytest.mark.parametrize("out_dtype", [F32, BF16])
@pytest.mark.parametrize("T,R,D", [(1, 1, 64), (257, 1000, 64), (1000, 77, 32), (1003, 5000, 128), (333, 500, 256),
                                   (129, 300, 1), (65, 300, 7), (41, 100, 20), (100, 300, 100), (19, 50, 1000),
                                   (70000, 300, 64)])
def test_lookup_is_one_rounded_product(table_dtype, out_dtype, T, R, D):
    g = torch.Generator(device=DEV).manual_seed(T + D)
    table = torch.randn(R, D, generator=g, device=DEV).to(table_dtype)
    ids = _ids("zipf", T, R, T)
    out = Guarded((T, D), out_dtype)
    _, err = B.fs_emb_lookup_scaled(table, ids, 1.7, out=out.t)
    B.check(err)
    out.check("lookup")
    assert torch.equal(out.t, (table[ids].float() * np.float32(1.7)).to(out_dtype))


def test_lookup_of_unaligned_rows():
    table = torch.randn(50 * 64 + 1, device=DEV)[1:].view(50, 64)  # 4-byte aligned
    ids = _ids("uniform", 300, 50, 1)
    out, err = B.fs_emb_lookup_scaled(table, ids, 8.0, out_dtype=BF16)
    B.check(err)
    assert torch.equal(out, (table[ids] * 8.0).to(BF16))


def test_lookup_edges_and_bad_ids():
    table = torch.randn(10, 64, device=DEV)
    out, err = B.fs_emb_lookup_scaled(table, torch.empty(0, dtype=torch.int64, device=DEV), 1.0)
    B.check(err)
    assert out.shape == (0, 64)
    for bad in (-1, 10, 1 << 40):
        ids = torch.tensor([3, bad, 7], device=DEV)
        out, err = B.fs_emb_lookup_scaled(table, ids, 2.0)
        with pytest.raises(B.FsError) as e:
            B.check(err)
        assert e.value.code == 2
        assert torch.equal(out[0], table[3] * 2) and torch.equal(out[2], table[7] * 2) and not out[1].any()
    t = torch.tensor([[float("nan"), float("inf"), -float("inf"), 0.0] * 8], device=DEV)
    out, _ = B.fs_emb_lookup_scaled(t, torch.zeros(1, dtype=torch.int64, device=DEV), 2.0)
    assert torch.equal(out.isnan(), t.isnan()) and torch.equal(out.isinf(), t.isinf())


def test_lookup_offsets_past_32_bits():
    """Element offsets above 2^32 in the table and in the output."""
    R, D = (1 << 26) + 3, 64
    table = torch.empty(R, D, dtype=BF16, device=DEV)
    rows = torch.tensor([0, 1 << 25, (1 << 26) + 2, (1 << 26) - 1], device=DEV)
    table[rows] = torch.randn(4, D, device=DEV).to(BF16)
    out, err = B.fs_emb_lookup_scaled(table, rows, 3.0)
    B.check(err)
    assert torch.equal(out, (table[rows].float() * 3.0).to(BF16))


def _reference(ids, dout, scale):
    uniq, inv = torch.unique(ids, return_inverse=True)
    g = dout.double().cpu()
    inv = inv.cpu()
    ref = torch.zeros(uniq.numel(), dout.shape[1], dtype=torch.float64).index_add_(0, inv, g)
    mag = torch.zeros_like(ref).index_add_(0, inv, g.abs())
    m = torch.bincount(inv, minlength=uniq.numel()).clamp(max=256).double()[:, None]
    return uniq, ref * scale, m * mag * abs(scale) * 2.0 ** -24


def _check_grads(ids, dout, R, scale, grad_dtype, cap=None):
    T, D = dout.shape
    uniq, ref, tol = _reference(ids, dout, scale)
    n = uniq.numel()
    cap = min(T, R) if cap is None else cap
    rows = Guarded(cap, torch.int64, DEV, torch.full((cap,), -7, dtype=torch.int64))
    grads = Guarded((cap, D), grad_dtype, DEV, torch.full((cap, D), 5.0))
    count = Guarded(1, torch.int64)
    ws = Guarded(B.emb_grad_rows_workspace_size(T, R, D), torch.uint8)
    _, _, _, err = B.fs_emb_grad_rows(ids, dout, R, scale, rows=rows.t, row_grads=grads.t, count=count.t, ws=ws.t)
    B.check(err)
    for x in (rows, grads, count, ws):
        x.check()
    assert int(count.t) == n
    assert torch.equal(rows.t[:n], uniq) and bool((rows.t[n:] == -7).all()) and bool((grads.t[n:] == 5.0).all())
    if grad_dtype == BF16:
        tol = tol + ref.abs() * 2.0 ** -8
    tol = tol + ref.abs() * 2.0 ** -23
    bad = (grads.t[:n].double().cpu() - ref).abs() > tol
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} out of tolerance"
    return grads.t[:n].clone()


@pytest.mark.parametrize("dout_dtype", [F32, BF16])
@pytest.mark.parametrize("grad_dtype", [F32, BF16])
@pytest.mark.parametrize("kind,T,R,D", [("uniform", 1, 1, 64), ("uniform", 2, 9, 32), ("zipf", 1000, 300, 64),
                                        ("one", 1025, 5, 64), ("zipf", 2049, 100_000, 128), ("zipf", 8192, 257, 32),
                                        ("zipf", 8193, 100_000, 64), ("one", 50_001, 70_000, 32),
                                        ("distinct", 30_000, 40_000, 64), ("ascending", 20_011, 3_000, 128)])
def test_row_grads(dout_dtype, grad_dtype, kind, T, R, D):
    g = torch.Generator(device=DEV).manual_seed(T)
    _check_grads(_ids(kind, T, R, T), torch.randn(T, D, generator=g, device=DEV).to(dout_dtype), R, 1.5, grad_dtype)


@pytest.mark.parametrize("D", [1, 3, 20, 100, 256, 520])
@pytest.mark.parametrize("T", [300, 9001])
def test_row_grads_of_other_widths(D, T):
    g = torch.Generator(device=DEV).manual_seed(D)
    for dt in (F32, BF16):
        _check_grads(_ids("zipf", T, 1000, D), torch.randn(T, D, generator=g, device=DEV).to(dt), 1000, -0.25, F32)


def test_row_grads_of_unaligned_dout():
    T, D = 9000, 64
    dout = torch.randn(T * D + 1, device=DEV)[1:].view(T, D)
    _check_grads(_ids("zipf", T, 500, 3), dout, 500, 1.0, F32)


def test_row_grads_hot_rows_are_the_same_run_to_run():
    T, R, D = 600_007, 1_000_000, 64
    g = torch.Generator(device=DEV).manual_seed(0)
    ids, dout = _ids("zipf", T, R, 5), torch.randn(T, D, generator=g, device=DEV)
    a = _check_grads(ids, dout, R, 8.0, F32)
    b = _check_grads(ids, dout, R, 8.0, F32)
    assert torch.equal(a, b)


@pytest.mark.parametrize("T,R,hot", [(9_000, 200, 1), (700_001, 1 << 16, 3), (2_600_003, (1 << 24) + 1, 1_000),
                                     (5_000_003, (1 << 32) - 1, 7)])
def test_row_grads_of_whole_numbers_are_exact(T, R, hot):
    """One to four sorting passes, ranges of several tiles, rows over thousands of tiles, IDs out of range among
    them: sums of small whole numbers are exact in 32 bits, in any order."""
    D = 4
    g = torch.Generator(device=DEV).manual_seed(T)
    ids = torch.randint(0, R, (T,), generator=g, device=DEV)
    ids = torch.where(torch.rand(T, generator=g, device=DEV) < 0.5, ids % hot * (R // hot), ids)
    ids[torch.rand(T, generator=g, device=DEV) < 0.01] = R
    dout = torch.randint(-2, 3, (T, D), generator=g, device=DEV).to(BF16)
    rows, grads, count, err = B.fs_emb_grad_rows(ids, dout, R, 2.0)
    with pytest.raises(B.FsError) as e:
        B.check(err)
    assert e.value.code == 2
    keep = ids < R
    uniq, inv = torch.unique(ids[keep], return_inverse=True)
    ref = torch.zeros(uniq.numel(), D, dtype=torch.float64).index_add_(0, inv.cpu(), dout[keep].double().cpu())
    n = uniq.numel()
    assert int(count) == n and torch.equal(rows[:n], uniq)
    assert torch.equal(grads[:n].double().cpu(), ref * 2.0)


def test_row_grads_equal_differences():
    """The gradient of sum(dout * lookup(W)) in W, by central differences along random directions (64 bits)."""
    T, R, D, scale = 500, 40, 16, 3.0
    g = torch.Generator(device=DEV).manual_seed(2)
    ids, dout = _ids("zipf", T, R, 9), torch.randn(T, D, generator=g, device=DEV)
    rows, grads, count, err = B.fs_emb_grad_rows(ids, dout, R, scale)
    B.check(err)
    n = int(count)
    W = torch.randn(R, D, generator=g, device=DEV).double()
    loss = lambda w: float((dout.double() * w[ids] * scale).sum())  # noqa: E731
    for _ in range(4):
        V = torch.randn(R, D, generator=g, device=DEV).double()
        slope = (loss(W + V * 1e-3) - loss(W - V * 1e-3)) / 2e-3
        assert abs(slope - float((grads[:n].double() * V[rows[:n]]).sum())) < 1e-4 * abs(slope) + 1e-3


@pytest.mark.parametrize("T", [100, 20_000])
def test_row_grads_errors(T):
    R, D = 50, 32
    dout = torch.randn(T, D, device=DEV)
    ids = _ids("uniform", T, R, 4)
    n = ids.unique().numel()
    # fewer places than rows: the first ones are right, the count is the full one
    rows = Guarded(7, torch.int64)
    grads = Guarded((7, D), F32)
    _, _, count, err = B.fs_emb_grad_rows(ids, dout, R, rows=rows.t, row_grads=grads.t)
    with pytest.raises(B.FsError) as e:
        B.check(err)
    assert e.value.code == 4 and int(count) == n
    rows.check(), grads.check()
    uniq, ref, tol = _reference(ids, dout, 1.0)
    assert torch.equal(rows.t, uniq[:7])
    assert not ((grads.t.double().cpu() - ref[:7]).abs() > tol[:7] + ref[:7].abs() * 2.0 ** -23).any()
    # an ID out of range is left out
    bad = ids.clone()
    bad[3], bad[T // 2], bad[T - 1] = -5, R, 1 << 45
    keep = (bad >= 0) & (bad < R)
    rows, grads, count, err = B.fs_emb_grad_rows(bad, dout, R)
    with pytest.raises(B.FsError) as e:
        B.check(err)
    assert e.value.code == 2
    uniq, ref, tol = _reference(bad[keep], dout[keep], 1.0)
    assert int(count) == uniq.numel() and torch.equal(rows[:uniq.numel()], uniq)
    assert not ((grads[:uniq.numel()].double().cpu() - ref).abs() > tol + ref.abs() * 2.0 ** -23).any()
    # nothing but bad IDs, and nothing at all
    rows, grads, count, err = B.fs_emb_grad_rows(torch.full((T,), -1, device=DEV), dout, R)
    assert int(count) == 0 and int(err) == 2
    rows, grads, count, err = B.fs_emb_grad_rows(ids[:0], dout[:0], R)
    B.check(err)
    assert int(count) == 0


def test_lookup_and_grads_on_another_stream():
    s = torch.cuda.Stream()
    table = torch.randn(1000, 64, device=DEV)
    ids = _ids("zipf", 30_000, 1000, 8)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        x, e1 = B.fs_emb_lookup_scaled(table, ids, 2.0)
        rows, grads, count, e2 = B.fs_emb_grad_rows(ids, x, 1000)
    s.synchronize()
    assert int(e1) == 0 and int(e2) == 0
    uniq, ref, tol = _reference(ids, (table[ids] * 2.0), 1.0)
    assert not ((grads[:uniq.numel()].double().cpu() - ref).abs() > tol + ref.abs() * 2.0 ** -23).any()
