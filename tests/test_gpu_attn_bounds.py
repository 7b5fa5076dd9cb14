"""Jagged attention where sizes and offsets go to extremes (GPU)."""
import random

import pytest
import torch

from jagged_embedding_gb300 import binding as B
from tests.helpers import Guarded
from tests.test_gpu_attn import Case, _near

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16


def test_offsets_of_more_tiles_than_32_bits_count():
    """Offsets 0, T, 0, T, ...: every second sample is refused, the others describe 2^19 * 2^13 = 2^32 tiles, which
    is 0 in 32 bits.  The lists hold T / 128 + S entries: nothing may be listed, and nothing written."""
    T = S = 1 << 20
    offsets = torch.zeros(S + 1, dtype=torch.int64, device=DEV)
    offsets[1::2] = T
    x = torch.zeros(T, 1, 64, dtype=BF16, device=DEV)
    ws = Guarded(B.jagged_attn_workspace_size(T, S, 1, 1, 64), torch.uint8)
    out, lse = torch.full((T, 1, 64), 7.0, dtype=BF16, device=DEV), torch.full((1, T), 7.0, device=DEV)
    _, _, err = B.fs_jagged_attn(x, x, x, offsets, 0.1, out=out, lse=lse, ws=ws.t)
    assert int(err) == 3
    assert bool((out == 7).all()) and bool((lse == 7).all())
    d = [torch.full((T, 1, 64), 7.0, dtype=BF16, device=DEV) for _ in range(3)]
    _, _, _, err = B.fs_jagged_attn_backward(x, x, x, out, lse, x, offsets, 0.1, dq=d[0], dk=d[1], dv=d[2], ws=ws.t)
    assert int(err) == 3
    assert all(bool((t == 7).all()) for t in d)
    ws.check()


def _only(c, samples):
    """Reference results of these samples alone (the others' are zero)."""
    lens = c.lens
    c.lens = [n if s in samples else 0 for s, n in enumerate(lens)]
    try:
        return c.reference()
    finally:
        c.lens = lens


def _check_samples(c, samples):
    out, lse, err = c.forward()
    B.check(err)
    r, t = _only(c, samples)
    grads = c.backward(out, lse)
    B.check(grads[3])
    assert all(bool(x.isfinite().all()) for x in (out, lse, *grads[:3]))
    for s in samples:
        a = slice(c.off[s], c.off[s + 1])
        _near(out[a], r["out"][a], t["out"][a], f"out of sample {s}")
        _near(lse[:, a], r["lse"][:, a], t["lse"][:, a], f"lse of sample {s}")
        for name, x in zip(("dq", "dk", "dv"), grads):
            # out and lse are the call's own here: another 2^-8 of out in delta, which the bound has once, and lse's error
            _near(x[a], r[name][a], 2 * t[name][a], f"{name} of sample {s}")
    return out, lse, grads


@pytest.mark.parametrize("Dh,H,Hkv", [(64, 4, 2), (128, 2, 1), (64, 3, 1)])
def test_batch_of_a_rank(Dh, H, Hkv):
    """A few hundred samples of lognormal lengths up to 8192, about a quarter of a million positions, with candidates."""
    rng = random.Random(Dh + H)
    uih = [min(8100, round(rng.lognormvariate(6.0, 1.5))) for _ in range(300)]
    uih[7], uih[20], uih[33] = 8100, 0, 0
    cand = [rng.randint(0, 64) for _ in uih]
    cand[7], cand[20], cand[33] = 64, 0, 17
    c = Case([u + b for u, b in zip(uih, cand)], H, Hkv, Dh, cand=cand)
    assert c.T > 150_000
    first = _check_samples(c, [0, 7, 33, 151, 298, 299])
    again = (*c.forward()[:2], *c.backward(first[0], first[1])[:3])
    assert all(torch.equal(x, y) for x, y in zip((first[0], first[1], *first[2][:3]), again))


@pytest.mark.parametrize("causal", [True, False])
def test_sample_of_16384(causal):
    _check_samples(Case([5, 16384, 40], 1, 1, 64, causal=causal, cand=[0, 33, 40]), [0, 1, 2])
