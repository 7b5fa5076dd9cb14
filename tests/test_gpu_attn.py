"""Jagged attention and its backward pass against the formulas in 64 bits (GPU).

Tolerances, from the arithmetic, element by element.  The probabilities p enter
their product with v rounded to bf16 (relative 2^-9), products accumulate in
fp32, results are rounded to bf16 (relative 2^-9): |out - ref| <= 2^-8 * (p |v| + |ref|)
covers both with a factor of two.  x = scale q.k is an fp32 sum of Dh products,
within Dh * 2^-24 * scale * |q|.|k| of itself: with the inputs here (|x| up to X)
that and the exp2 of a product rounded to fp32 move p by at most
E = 2^-22 * (Dh / 4 * scale * max |q|.|k| + X + 4) relative, and lse by E absolute.
Backward: ds rounded to bf16 likewise, and delta = dout.out is taken from the
rounded out, off by at most 2^-9 * |dout|.|out| =: d_i; so
|dv - ref| <= (2^-8 + 2 E) p'|dout| + 2^-8 |ref|,
|dq - ref| <= scale * (2^-8 + 2 E) (|ds| + p (|dp| + |delta|) 2 E) |k| + 2 scale (p d_i) |k| + 2^-8 |ref|, dk with q.
"""
import pytest
import torch

from jagged_embedding_gb300 import binding as B
from tests.helpers import Guarded

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16


def _mask(L, cand, causal):
    i = torch.arange(L, device=DEV)
    see = (i[None] < L - cand) | (i[:, None] == i[None])
    return see & (i[None] <= i[:, None]) if causal else see


class Case:
    """Inputs as a user has them (q, k, v slices of one projection) and the 64-bit results with their tolerances."""

    def __init__(self, lens, H, Hkv, Dh, causal=True, cand=None, seed=0, lead=0, tail=0, gain=1.0, scale=None,
                 contiguous=False):
        g = torch.Generator(device=DEV).manual_seed(seed + 1000 * Dh + sum(lens))
        T = lead + sum(lens) + tail
        self.lens, self.H, self.Hkv, self.Dh, self.T = lens, H, Hkv, Dh, T
        self.causal, self.cand = causal, cand
        off = [lead]
        for n in lens:
            off.append(off[-1] + n)
        self.off = off
        self.offsets = torch.tensor(off, dtype=torch.int64, device=DEV)
        self.cand_len = None if cand is None else torch.tensor(cand, dtype=torch.int32, device=DEV)
        self.scale = Dh ** -0.5 if scale is None else scale
        qkv = (torch.randn(T, H + 2 * Hkv, Dh, generator=g, device=DEV) * gain).to(BF16)
        self.q, self.k, self.v = qkv.split([H, Hkv, Hkv], dim=1)
        if contiguous:
            self.q, self.k, self.v = (t.contiguous() for t in (self.q, self.k, self.v))
        self.dout = torch.randn(T, H, Dh, generator=g, device=DEV).to(BF16)

    def forward(self, **kw):
        return B.fs_jagged_attn(self.q, self.k, self.v, self.offsets, self.scale, causal=self.causal,
                                cand_len=self.cand_len, **kw)

    def backward(self, out, lse, **kw):
        return B.fs_jagged_attn_backward(self.q, self.k, self.v, out, lse, self.dout, self.offsets, self.scale,
                                         causal=self.causal, cand_len=self.cand_len, **kw)

    def reference(self):
        H, Hkv, Dh, T = self.H, self.Hkv, self.Dh, self.T
        z = lambda h: torch.zeros(T, h, Dh, dtype=torch.float64, device=DEV)  # noqa: E731
        r = {"out": z(H), "dq": z(H), "dk": z(Hkv), "dv": z(Hkv)}
        t = {n: torch.zeros_like(x) for n, x in r.items()}
        r["lse"] = torch.zeros(H, T, dtype=torch.float64, device=DEV)
        t["lse"] = torch.zeros_like(r["lse"])
        for s, L in enumerate(self.lens):
            if L == 0:
                continue
            a = slice(self.off[s], self.off[s] + L)
            see = _mask(L, 0 if self.cand is None else self.cand[s], self.causal)
            for h in range(H):
                hk = h * Hkv // H
                q, k, v, g = (x.double() for x in (self.q[a, h], self.k[a, hk], self.v[a, hk], self.dout[a, h]))
                x = (q @ k.T * self.scale).masked_fill(~see, -float("inf"))
                lse = torch.logsumexp(x, 1)
                p = torch.exp(x - lse[:, None])
                o = p @ v
                mag = float((q.abs() @ k.abs().T).max()) * self.scale
                E = 2.0 ** -22 * (Dh / 4 * mag + float(x[see].abs().max()) + 4)
                r["out"][a, h], t["out"][a, h] = o, (2.0 ** -8 + 2 * E) * (p @ v.abs() + o.abs())
                r["lse"][h, a], t["lse"][h, a] = lse, E + 2.0 ** -22 * lse.abs()
                dp, delta = g @ v.T, (g * o).sum(1, keepdim=True)
                ds = p * (dp - delta)
                d = 2.0 ** -8 * (g.abs() * o.abs()).sum(1, keepdim=True)
                b = 2.0 ** -8 + 2 * E
                es = b * ds.abs() + 2 * E * p * (dp.abs() + delta.abs() + (g.abs() @ v.abs().T)) + p * d
                r["dq"][a, h] = ds @ k * self.scale
                t["dq"][a, h] = es @ k.abs() * self.scale
                r["dk"][a, hk] += ds.T @ q * self.scale
                t["dk"][a, hk] += es.T @ q.abs() * self.scale
                r["dv"][a, hk] += p.T @ g
                t["dv"][a, hk] += b * (p.T @ g.abs())
        for n in ("dq", "dk", "dv"):
            t[n] += 2.0 ** -8 * r[n].abs()
        return r, t

    def inside(self):
        m = torch.zeros(self.T, dtype=torch.bool, device=DEV)
        m[self.off[0]:self.off[-1]] = True
        return m


def _near(got, ref, tol, what):
    bad = ~((got.double() - ref).abs() <= tol + 1e-30)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} out of tolerance, first {bad.nonzero()[0].tolist()}"


def _check(c):
    r, t = c.reference()
    T, H, Hkv, Dh = c.T, c.H, c.Hkv, c.Dh
    m = c.inside()
    mark = 77.0
    out = Guarded((T, H, Dh), BF16, DEV, torch.full((T, H, Dh), mark))
    lse = Guarded((H, T), torch.float32, DEV, torch.full((H, T), mark))
    ws = Guarded(B.jagged_attn_workspace_size(T, len(c.lens), H, Hkv, Dh), torch.uint8)
    _, _, err = c.forward(out=out.t, lse=lse.t, ws=ws.t)
    B.check(err)
    for x in (out, lse, ws):
        x.check()
    _near(out.t[m], r["out"][m], t["out"][m], "out")
    _near(lse.t[:, m], r["lse"][:, m], t["lse"][:, m], "lse")
    assert bool((out.t[~m] == mark).all()) and bool((lse.t[:, ~m] == mark).all())
    dqkv = Guarded((T, H + 2 * Hkv, Dh), BF16, DEV, torch.full((T, H + 2 * Hkv, Dh), mark))
    dq, dk, dv = dqkv.t.split([H, Hkv, Hkv], dim=1)
    _, _, _, err = c.backward(r["out"].to(BF16), r["lse"].float(), dq=dq, dk=dk, dv=dv, ws=ws.t)
    B.check(err)
    dqkv.check(), ws.check()
    for n, x in (("dv", dv), ("dq", dq), ("dk", dk)):
        _near(x[m], r[n][m], t[n][m], n)
    assert bool((dqkv.t[~m] == mark).all())
    return out.t, lse.t, dqkv.t


LENS = {"one": [1], "empty": [0, 1, 0, 0], "tile": [128], "around": [127, 129, 63, 65, 1, 64], "two": [256, 2],
        "long": [517], "mixed": [300, 0, 7, 411, 128, 33]}


@pytest.mark.parametrize("Dh", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens", list(LENS))
def test_attention_over_lengths(lens, causal, Dh):
    _check(Case(LENS[lens], 2, 2, Dh, causal))


@pytest.mark.parametrize("Dh", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("cand", ["none", "some", "all", "tile"])
def test_attention_with_candidates(cand, causal, Dh):
    lens = [300, 0, 7, 411, 128, 33, 260]
    c = {"none": [0] * 7, "some": [31, 0, 3, 64, 1, 32, 130], "all": lens, "tile": [172, 0, 0, 283, 128, 5, 132]}[cand]
    _check(Case(lens, 2, 1, Dh, causal, cand=c))


@pytest.mark.parametrize("H,Hkv", [(1, 1), (4, 1), (6, 2), (6, 3), (3, 3), (16, 4)])
def test_attention_with_shared_heads(H, Hkv):
    _check(Case([200, 77, 140], H, Hkv, 64, cand=[20, 0, 9]))
    _check(Case([150, 64], H, Hkv, 128, contiguous=True))


def test_attention_of_a_long_sample():
    _check(Case([2100, 1, 1033], 2, 1, 128, cand=[64, 1, 40]))
    _check(Case([1500], 1, 1, 64, causal=False))


def test_many_short_samples():
    lens = [(7 * i) % 23 for i in range(700)]
    _check(Case(lens, 1, 1, 64, cand=[min(n, i % 3) for i, n in enumerate(lens)]))


def test_positions_of_no_sample_are_untouched():
    _check(Case([70, 200], 2, 1, 64, lead=13, tail=150))
    _check(Case([40], 1, 1, 128, lead=300, tail=1))


@pytest.mark.parametrize("Dh", [64, 128])
def test_large_and_equal_logits(Dh):
    _check(Case([140, 65], 2, 2, Dh, gain=6.0, scale=1.0))    # |x| to several thousand: one key takes all
    _check(Case([140, 65], 2, 2, Dh, gain=0.0))               # every visible key alike
    c = Case([200], 1, 1, Dh, gain=1e-3)
    _check(c)


@pytest.mark.parametrize("Dh", [64, 128])
def test_samples_do_not_mix(Dh):
    """NaN and infinities in one sample, and in positions of no sample, reach no other sample."""
    lens = [100, 90, 131, 50]
    c = Case(lens, 2, 1, Dh, lead=40, tail=40)
    clean = _check(c)
    bad = torch.zeros(c.T, dtype=torch.bool, device=DEV)
    bad[:c.off[0]] = True
    bad[c.off[1]:c.off[2]] = True
    bad[c.off[-1]:] = True
    out, lse = clean[0].clone(), clean[1].clone()
    lse[:, ~c.inside()] = float("nan")
    out[~c.inside()] = float("nan")
    for value in (float("nan"), float("inf")):
        for x in (c.q, c.k, c.v, c.dout):
            x[bad] = value
        o, l, err = c.forward()
        B.check(err)
        good = c.inside() & ~bad
        assert torch.equal(o[good], clean[0][good]) and torch.equal(l[:, good], clean[1][:, good])
        r, _ = Case(lens, 2, 1, Dh, lead=40, tail=40).reference()
        dq, dk, dv, err = c.backward(torch.where(good[:, None, None], r["out"].to(BF16), out),
                                     torch.where(good[None], r["lse"].float(), lse))
        B.check(err)
        H, Hkv = c.H, c.Hkv
        for x, y in zip((dq, dk, dv), clean[2].split([H, Hkv, Hkv], dim=1)):
            assert torch.equal(x[good], y[good])


def test_the_same_bits_run_to_run_and_on_another_stream():
    c = Case([700, 3, 400, 129], 4, 2, 64, cand=[10, 0, 64, 2])
    a = _check(c)
    b = _check(c)
    assert all(torch.equal(x.view(torch.int32) if x.dtype == torch.float32 else x, y.view(torch.int32)
                           if y.dtype == torch.float32 else y) for x, y in zip(a, b))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        out, lse, err = c.forward()
    s.synchronize()
    assert int(err) == 0 and torch.equal(out, a[0]) and torch.equal(lse, a[1])


def test_gradients_equal_differences():
    """Central differences of sum(dout * attention) along random directions, the attention in 64 bits."""
    c = Case([37, 90], 2, 1, 64, cand=[5, 20])
    r, _ = c.reference()
    dq, dk, dv, err = c.backward(r["out"].to(BF16), r["lse"].float())
    B.check(err)
    q, k, v, g = (x.double() for x in (c.q, c.k, c.v, c.dout))

    def loss(q, k, v):
        n = 0.0
        for s, L in enumerate(c.lens):
            a = slice(c.off[s], c.off[s] + L)
            see = _mask(L, c.cand[s], True)
            for h in range(c.H):
                x = (q[a, h] @ k[a, 0].T * c.scale).masked_fill(~see, -float("inf"))
                n += float((g[a, h] * (torch.softmax(x, 1) @ v[a, 0])).sum())
        return n

    gen = torch.Generator(device=DEV).manual_seed(1)
    for _ in range(3):
        d = [torch.randn(x.shape, generator=gen, device=DEV, dtype=torch.float64) for x in (q, k, v)]
        e = 1e-4
        slope = (loss(q + e * d[0], k + e * d[1], v + e * d[2]) - loss(q - e * d[0], k - e * d[1], v - e * d[2])) / (2 * e)
        terms = [(x.double() * y) for x, y in zip((dq, dk, dv), d)]
        # each gradient element is within about 2^-7 of its size: random signs, so far below the sum of all
        tol = 2.0 ** -7 * sum(float(t.square().sum()) for t in terms) ** 0.5 * 4
        assert abs(slope - sum(float(t.sum()) for t in terms)) < tol


def test_data_errors():
    c = Case([50, 60], 1, 1, 64, cand=[3, 4])
    for off in ([0, 60, 50], [0, 50, 111], [-1, 50, 110]):
        c.offsets = torch.tensor(off, device=DEV)
        out = Guarded((c.T, 1, 64), BF16)
        lse = Guarded((1, c.T), torch.float32)
        _, _, err = c.forward(out=out.t, lse=lse.t)
        with pytest.raises(B.FsError) as e:
            B.check(err)
        assert e.value.code == 3
        out.check(), lse.check()
        r = [Guarded((c.T, 1, 64), BF16) for _ in range(3)]
        _, _, _, err = c.backward(torch.zeros(c.T, 1, 64, dtype=BF16, device=DEV), torch.zeros(1, c.T, device=DEV),
                                  dq=r[0].t, dk=r[1].t, dv=r[2].t)
        with pytest.raises(B.FsError) as e:
            B.check(err)
        assert e.value.code == 3
        for x in r:
            x.check()
    c.offsets = torch.tensor([0, 50, 110], device=DEV)
    for bad, as_if in (([-1, 4], [0, 4]), ([3, 61], [3, 60])):
        c.cand_len = torch.tensor(bad, dtype=torch.int32, device=DEV)
        out, _, err = c.forward()
        with pytest.raises(B.FsError) as e:
            B.check(err)
        assert e.value.code == 1
        c.cand_len = torch.tensor(as_if, dtype=torch.int32, device=DEV)
        want, _, err = c.forward()
        B.check(err)
        assert torch.equal(out, want)


def test_nothing_to_do():
    e = torch.empty(0, 2, 64, dtype=BF16, device=DEV)
    out, lse, err = B.fs_jagged_attn(e, e, e, torch.zeros(4, dtype=torch.int64, device=DEV), 0.1)
    B.check(err)
    assert out.shape == (0, 2, 64)
    x = torch.randn(5, 2, 64, device=DEV).to(BF16)
    out, lse, err = B.fs_jagged_attn(x, x, x, torch.zeros(1, dtype=torch.int64, device=DEV), 0.1)
    B.check(err)
    dq, dk, dv, err = B.fs_jagged_attn_backward(x, x, x, out, lse, x, torch.zeros(3, dtype=torch.int64, device=DEV), 0.1)
    B.check(err)


def test_many_units_a_block_and_heavy_key_tiles_in_halves():
    """More units than SMs (lists, several units a block), and a batch in which a few long samples hold most of the
    work, so that their key tiles are cut in half."""
    lens = [(37 * i) % 331 for i in range(60)]
    _check(Case(lens, 4, 2, 64, cand=[min(n, i % 5) for i, n in enumerate(lens)]))
    _check(Case(lens, 3, 3, 128, causal=False))
    heavy = [1700, 1500] + [20 + i for i in range(40)]
    a = _check(Case(heavy, 8, 2, 128))
    b = _check(Case(heavy, 8, 2, 128))
    assert torch.equal(a[2], b[2])  # (which half comes first does not show)
    _check(Case(heavy, 4, 1, 64, causal=False, cand=[min(n, 64) for n in heavy]))


@pytest.mark.parametrize("S", [32, 33])
def test_around_the_batch_without_lists(S):
    lens = [3 + 2 * i for i in range(S)]
    _check(Case(lens, 2, 2, 64, cand=[i % 3 for i in range(S)]))


def test_empty_samples_only():
    c = Case([0] * 40, 2, 1, 64, tail=50)
    out, lse, err = c.forward()
    B.check(err)
    c.backward(out, lse, err=err)
    B.check(err)


@pytest.mark.parametrize("Dh", [64, 128])
@pytest.mark.parametrize("lens", [[400], [90, 700, 5], [50] * 40])
def test_waits_that_run_out(Dh, lens):
    """A tile that is never loaded: every wait ends, the error word says so, and the context stays usable."""
    c = Case(lens, 2, 2, Dh)
    want = c.forward()
    B.check(want[2])
    grads = c.backward(want[0], want[1])
    B.check(grads[3])
    before = B.spin_limit()
    try:
        B.set_spin_limit(2000)  # about half a millisecond a wait
        B.debug_skip_publish(0)
        _, _, err = c.forward()
        with pytest.raises(B.FsError) as e:
            B.check(err)
        assert e.value.code == 6
        _, _, _, err = c.backward(want[0], want[1])
        with pytest.raises(B.FsError) as e:
            B.check(err)
        assert e.value.code == 6
    finally:
        B.debug_skip_publish(-1)
        B.set_spin_limit(before)
    again = c.forward()
    B.check(again[2])
    m = c.inside()
    assert torch.equal(again[0][m], want[0][m])
    g2 = c.backward(want[0], want[1])
    B.check(g2[3])
    assert all(torch.equal(x[m], y[m]) for x, y in zip(grads[:3], g2[:3]))
