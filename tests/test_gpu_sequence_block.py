"""The sequence block on a prepared batch: the five calls together, forward and backward, against the same
layer in 32 bits with torch's own differentiation (GPU).

Activations are bf16, so each result carries a few roundings of 2^-9 relative to its size: results are compared
by the norm of the difference, at most 2^-6 of the norm (the worst of the products here passes eight roundings
one after another, each of at most 2^-9 of the norm).
"""
import math

import numpy as np
import pytest
import torch

from jagged_embedding_gb300 import binding as B
from jagged_embedding_gb300 import synthetic
from jagged_embedding_gb300.pipeline import Pipeline
from jagged_embedding_gb300.sequence_block import SequenceBlock

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _norm(x, w, eps):
    return x * torch.rsqrt((x * x).mean(1, keepdim=True) + eps) * w


def _reference(blk, table, ids, off, cand):
    p = {n: getattr(blk, n).float().requires_grad_() for n in ("w_qkv", "w_out", "gamma_in", "gamma_out")}
    t = table.float().requires_grad_()
    x = t[ids] * blk.emb_scale
    T, H, Hkv, Dh = ids.numel(), blk.heads, blk.kv_heads, blk.head_dim
    q, k, v = (_norm(x, p["gamma_in"], blk.eps) @ p["w_qkv"]).view(T, H + 2 * Hkv, Dh).split([H, Hkv, Hkv], dim=1)
    k, v = k.repeat_interleave(H // Hkv, 1), v.repeat_interleave(H // Hkv, 1)
    outs = []
    for s in range(len(off) - 1):
        a = slice(off[s], off[s + 1])
        L = off[s + 1] - off[s]
        i = torch.arange(L, device=DEV)
        see = ((i[None] < L - cand[s]) | (i[:, None] == i[None])) & (i[None] <= i[:, None])
        w = (torch.einsum("ihd,jhd->hij", q[a], k[a]) * blk.scale).masked_fill(~see, -float("inf"))
        outs.append(torch.einsum("hij,jhd->ihd", torch.softmax(w, 2), v[a]))
    h = x + torch.cat(outs).reshape(T, H * Dh) @ p["w_out"]
    return _norm(h, p["gamma_out"], blk.eps), h, t, p


def _close(got, ref, what):
    rel = float((got.double() - ref.double()).norm() / ref.double().norm())
    assert rel < 2.0 ** -6, f"{what}: {rel:.4f}"


def test_block_on_a_prepared_batch():
    w = synthetic.WORKLOADS["tiny-fbs-sgd"].scaled(n=4, B=6, R=3000, lmax=300, mu=4.0)
    b = synthetic.batch(w, 0)
    table = torch.randn(w.R, w.D, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1)) * 0.1
    pipe = Pipeline(w, torch.device(DEV), b["T"], table, torch.zeros(w.R, device=DEV))
    pipe.prepare({k: (v.to(DEV) if torch.is_tensor(v) else v) for k, v in b.items()}, 0)
    B.check(pipe.err)
    slot = pipe.slots[0]
    T, S = b["T"], w.S
    ids, off = slot.ids[:T], slot.offsets[: S + 1]
    cand = torch.from_numpy(np.minimum(3, np.diff(off.cpu().numpy())).astype(np.int32)).to(DEV)
    blk = SequenceBlock(w.D, 4, 2, 64, generator=torch.Generator(device=DEV).manual_seed(2))
    out, scale, saved = blk.forward(table, ids, off, cand)
    blk.check()
    ref, h, t, p = _reference(blk, table, ids, off.tolist(), cand.tolist())
    _close(out, ref.detach(), "out")
    g = torch.Generator(device=DEV).manual_seed(3)
    dout, dh = (torch.randn(T, w.D, device=DEV, generator=g).to(torch.bfloat16) for _ in range(2))
    grads = blk.backward(dout, saved, dh=dh)
    blk.check()
    (ref * dout.float()).sum().add((h * dh.float()).sum()).backward()
    n = int(grads["count"])
    rows = torch.unique(ids)
    assert torch.equal(grads["rows"][:n], rows)
    _close(grads["row_grads"][:n], t.grad[rows], "row_grads")
    for name in ("w_qkv", "w_out", "gamma_in", "gamma_out"):
        _close(grads[name], p[name].grad, name)
    # 8 bits for a projection that takes them: the same output within half an e4m3 step, 2^-4 of each value
    q8, s8, _ = blk.forward(table, ids, off, cand, bits8=True)
    blk.check()
    back = q8.float() * s8[:, None]
    assert bool(((back - out.float()).abs() <= out.float().abs() * (2.0 ** -4 + 2.0 ** -7) + s8[:, None] * 2.0 ** -9).all())


def test_training_steps_lower_the_loss():
    """A few steps of plain SGD on the table through the row gradients."""
    gen = torch.Generator(device=DEV).manual_seed(4)
    R, D, T = 500, 64, 2000
    off = torch.tensor([0, 700, 700, 1200, 2000], device=DEV)
    table = torch.randn(R, D, device=DEV, generator=gen) * 0.05
    ids = torch.randint(0, R, (T,), device=DEV, generator=gen)
    target = torch.randn(T, D, device=DEV, generator=gen)
    blk = SequenceBlock(D, 2, 1, 64, generator=gen)
    losses = []
    for _ in range(6):
        out, _, saved = blk.forward(table, ids, off)
        diff = out.float() - target
        losses.append(float(diff.square().mean()))
        grads = blk.backward((2 * diff / T).to(torch.bfloat16), saved)
        n = int(grads["count"])
        table[grads["rows"][:n]] -= 0.05 * grads["row_grads"][:n]
    blk.check()
    assert all(b < a for a, b in zip(losses, losses[1:])) and math.isfinite(losses[-1])
