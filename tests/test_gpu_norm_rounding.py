"""The 8-bit output of the RMS norm, bit for bit (GPU).

Rows of +-2^k have a mean square of 4^k, so with eps = 0 the norm of each is +-1 exactly and y = +-gamma exactly.  Then
the scale is the fp32 quotient max |gamma| / 448 and q the e4m3 value nearest to the fp32 quotient y / scale, ties to
even: nothing is left to a tolerance.  (1 + 2^-13 steps of the scales leave room for exact products with e4m3 values
and with the middles between them.)
"""
import numpy as np
import pytest
import torch

from jagged_embedding_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16, E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn


def _rows(D, dt, seed):
    """Rows of signs times 1, 1/2 and 4."""
    g = torch.Generator().manual_seed(seed)
    sign = torch.randint(0, 2, (3, D), generator=g) * 2 - 1
    return sign, (sign * torch.tensor([[1.0], [0.5], [4.0]])).to(dt).to(DEV)


def _check(gamma, dt, seed):
    sign, x = _rows(gamma.size, dt, seed)
    q, scale, _, rstd = B.fs_rmsnorm(x, torch.from_numpy(gamma).to(DEV), 0.0, y_dtype=E4M3)
    assert torch.equal(rstd.cpu(), torch.tensor([1.0, 2.0, 0.25]))
    s = np.float32(np.abs(gamma).max()) / np.float32(448)
    assert (scale.cpu().numpy() == s).all()
    want = (sign * torch.from_numpy(gamma / s)).to(E4M3)
    got = q.cpu()
    bad = (got.view(torch.uint8) != want.view(torch.uint8)).sum()
    assert bad == 0, f"{int(bad)} of {got.numel()}"


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("D", [512, 1001, 8192])
def test_quotients_in_the_middle_go_to_even(D, dt):
    r = np.random.default_rng(D)
    # 448 first, then the middles between e4m3 values (normal ones, and multiples of 2^-10 below 2^-6)
    mids = np.array([448.0] + [(8 + k + 0.5) / 8 * 2.0 ** e for e in range(-6, 9) for k in range(8) if (8 + k + 0.5) / 8 * 2.0 ** e < 448]
                    + [(2 * k + 1) * 2.0 ** -10 for k in range(8)], dtype=np.float32)
    for i in range(12):
        s = np.float32((1 + r.integers(0, 1 << 13) / 2.0 ** 13) * 2.0 ** r.integers(-20, 20))
        m = mids[np.concatenate([[0], r.integers(0, mids.size, D - 1)])]
        gamma = (m * s).astype(np.float32)
        assert (gamma.astype(np.float64) == m.astype(np.float64) * np.float64(s)).all()
        _check(gamma, dt, i)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("exponent", [0, 60, 118, -80, -96, -105, -118, -124, -127, -136])
def test_quotients_of_any_scale(exponent, dt):
    """Scales from 2^118 to below 2^-126, where a reciprocal would overflow and fp32 has fewer bits."""
    r = np.random.default_rng(exponent & 0xFF)
    for D in (256, 2056):
        v = (r.standard_normal(D) * np.exp(2 * r.standard_normal(D))).astype(np.float32)
        gamma = (v / np.abs(v).max() * np.float32(448) * np.float32(2.0) ** np.float32(exponent)).astype(np.float32)
        assert np.abs(gamma).max() > 0 and np.isfinite(gamma).all()
        _check(gamma, dt, D)


def test_infinite_scale():
    """gamma * h overflows in one place: the scale is infinite, the others' quotients are 0, its own is NaN."""
    x = torch.ones(1, 64, device=DEV)
    x[0, 3] = 8.0
    gamma = torch.ones(64, device=DEV)
    gamma[3] = 3.0e38
    q, scale, _, _ = B.fs_rmsnorm(x, gamma, 0.0, y_dtype=E4M3)
    assert bool(scale.isinf().all()) and bool(q.float()[0, 3].isnan())
    rest = torch.ones(64, dtype=torch.bool, device=DEV)
    rest[3] = False
    assert not q.float()[0, rest].any()
