"""Gradients of attention over small batches, whose p and ds enter their products as pairs of bf16 (GPU).

A value x rounded to bf16 leaves a rest of at most 2^-9 |x|, and the rest rounded to bf16 leaves 2^-18 |x|: a pair is
within 2^-17 of the value with a factor of two.  Otherwise as in the tests of larger batches: x = scale q.k and the exp2 of
it move p by at most E = 2^-22 * (Dh / 4 * scale * max |q|.|k| + X + 4) relative; where a query tile meets more than
one key tile, delta comes from the rounded out, off by at most d = 2^-8 * |dout|.|out|; results are rounded to bf16 once,
within 2^-8 of the value.
"""
import pytest
import torch

from jagged_embedding_gb300 import binding as B
from tests.test_gpu_attn import Case, _mask, _near

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def _reference(c):
    """64-bit gradients and their bounds, pairs of bf16 in place of single roundings."""
    H, Hkv = c.H, c.Hkv
    shape = lambda h: torch.zeros(c.T, h, c.Dh, dtype=torch.float64, device="cuda")  # noqa: E731
    r = {"dq": shape(H), "dk": shape(Hkv), "dv": shape(Hkv)}
    t = {n: torch.zeros_like(x) for n, x in r.items()}
    out, lse = shape(H), torch.zeros(H, c.T, dtype=torch.float64, device="cuda")
    for s, L in enumerate(c.lens):
        if L == 0:
            continue
        a = slice(c.off[s], c.off[s] + L)
        see = _mask(L, 0 if c.cand is None else c.cand[s], c.causal)
        for h in range(H):
            hk = h * Hkv // H
            q, k, v, g = (x.double() for x in (c.q[a, h], c.k[a, hk], c.v[a, hk], c.dout[a, h]))
            x = (q @ k.T * c.scale).masked_fill(~see, -float("inf"))
            lse[h, a] = torch.logsumexp(x, 1)
            p = torch.exp(x - lse[h, a][:, None])
            out[a, h] = p @ v
            E = 2.0 ** -22 * (c.Dh / 4 * float((q.abs() @ k.abs().T).max()) * c.scale + float(x[see].abs().max()) + 4)
            dp, delta = g @ v.T, (g * out[a, h]).sum(1, keepdim=True)
            ds = p * (dp - delta)
            b = 2.0 ** -17 + 2 * E
            es = b * ds.abs() + 2 * E * p * (dp.abs() + delta.abs() + g.abs() @ v.abs().T)
            if L > 128:
                es = es + p * (2.0 ** -8 * (g.abs() * out[a, h].abs()).sum(1, keepdim=True))
            r["dq"][a, h], t["dq"][a, h] = ds @ k * c.scale, es @ k.abs() * c.scale
            r["dk"][a, hk] += ds.T @ q * c.scale
            t["dk"][a, hk] += es.T @ q.abs() * c.scale
            r["dv"][a, hk] += p.T @ g
            t["dv"][a, hk] += b * (p.T @ g.abs())
    for n in r:
        t[n] += 2.0 ** -8 * r[n].abs()
    return out.to(BF16), lse.float(), r, t


@pytest.mark.parametrize("Dh", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,cand,H,Hkv", [([1], None, 2, 2), ([9], [1], 4, 4), ([128, 127, 0, 64], [5, 0, 0, 64], 4, 2),
                                             ([41, 0, 35], [40, 0, 32], 4, 2), ([30] * 32, [i % 4 for i in range(32)], 3, 1),
                                             ([129, 300], [3, 64], 2, 1)])
def test_gradients_within_one_rounding(lens, cand, H, Hkv, causal, Dh):
    c = Case(lens, H, Hkv, Dh, causal, cand=cand)
    out, lse, r, t = _reference(c)
    dq, dk, dv, err = c.backward(out, lse)
    B.check(err)
    for n, x in (("dv", dv), ("dk", dk), ("dq", dq)):
        _near(x, r[n], t[n], n)
