"""Sequence-block calls on tensors of more than 2^32 elements, checked where the offsets are that large (GPU)."""
import pytest
import torch

from jagged_embedding_gb300 import binding as B
from tests.test_gpu_attn import Case, _near

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16
T, D = (1 << 25) + 3, 128


@pytest.fixture(autouse=True)
def _give_back():
    yield
    torch.cuda.empty_cache()


def test_lookup_output():
    table = torch.randn(1000, D, device=DEV).to(BF16)
    ids = torch.arange(T, device=DEV) % 1000
    out, err = B.fs_emb_lookup_scaled(table, ids, 2.0)
    B.check(err)
    want = (table.float() * 2).to(BF16)
    for a in (0, (1 << 25) - 1000, T - 1000):
        assert torch.equal(out[a:a + 1000], want[ids[a:a + 1000]])


def test_row_gradients():
    """All rows distinct: dout and the gradients both pass 2^32 elements."""
    rows_in = torch.arange(T, device=DEV)
    dout = (rows_in % 251).to(BF16)[:, None].expand(T, D).contiguous()
    rows, grads, count, err = B.fs_emb_grad_rows(rows_in.flip(0), dout, T, 2.0)
    B.check(err)
    assert int(count) == T and torch.equal(rows, rows_in)
    for a in (0, (1 << 25) - 5000, T - 5000):
        want = ((T - 1 - rows_in[a:a + 5000]) % 251).to(F32) * 2
        assert torch.equal(grads[a:a + 5000], want[:, None].expand(5000, D))


def test_norm_and_its_backward_pass():
    few = 512
    g = torch.Generator(device=DEV).manual_seed(0)
    x, dy = (torch.randn(few, D, generator=g, device=DEV).to(BF16) for _ in range(2))
    gamma = torch.ones(D, device=DEV)
    y, _, _, rstd = B.fs_rmsnorm(x, gamma, 1e-6)
    dh, _ = B.fs_rmsnorm_backward(dy, x, gamma, rstd)
    at = torch.arange(T, device=DEV) % few
    Y, _, _, RSTD = B.fs_rmsnorm(x[at], gamma, 1e-6)
    for a in (0, (1 << 25) - few, T - few):
        assert torch.equal(Y[a:a + few], y[at[a:a + few]])
    assert torch.equal(RSTD, rstd[at])
    del Y
    DH, _ = B.fs_rmsnorm_backward(dy[at], x[at], gamma, RSTD)
    for a in (0, (1 << 25) - few, T - few):
        assert torch.equal(DH[a:a + few], dh[at[a:a + few]])


def test_attention():
    """Two samples at the end of 2^22 positions of 8 heads of 128."""
    c = Case([300, 130], 8, 1, D, cand=[20, 0])
    r, t = c.reference()
    n, big = sum(c.lens), (1 << 22) + 1000
    qkv = torch.empty(big, 10, D, dtype=BF16, device=DEV)
    q, k, v = qkv.split([8, 1, 1], dim=1)
    for to, x in ((q, c.q), (k, c.k), (v, c.v)):
        to[big - n:] = x
    off = c.offsets + (big - n)
    out, lse, err = B.fs_jagged_attn(q, k, v, off, c.scale, cand_len=c.cand_len)
    B.check(err)
    _near(out[big - n:], r["out"], t["out"], "out")
    _near(lse[:, big - n:], r["lse"], t["lse"], "lse")
    out[big - n:], lse[:, big - n:] = r["out"].to(BF16), r["lse"].float()
    dout = torch.empty(big, 8, D, dtype=BF16, device=DEV)
    dout[big - n:] = c.dout
    dq, dk, dv, err = B.fs_jagged_attn_backward(q, k, v, out, lse, dout, off, c.scale, cand_len=c.cand_len)
    B.check(err)
    for name, x in (("dq", dq), ("dk", dk), ("dv", dv)):
        _near(x[big - n:], r[name], t[name], name)
