"""Row gradients of small batches, which one block sorts while the kernel that sums is already in place (GPU).

Gradients are small whole numbers, whose fp32 sums are exact in any order, so every result is compared bit for bit.
"""
import pytest
import torch

from jagged_embedding_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16


def _batch(T, R, D, seed, hot=0.5):
    """IDs, half of them few, and whole-number gradients."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    ids = torch.randint(0, R, (T,), generator=g, device=DEV)
    few = torch.rand(T, generator=g, device=DEV) < hot
    ids = torch.where(few, R - 1 - ids % min(7, R), ids)
    return ids, torch.randint(-3, 4, (T, D), generator=g, device=DEV).to(BF16)


def _expect(ids, dout, R):
    keep = (ids >= 0) & (ids < R)
    uniq, inv = torch.unique(ids[keep], return_inverse=True)
    ref = torch.zeros(uniq.numel(), dout.shape[1], dtype=torch.float64)
    return uniq, ref.index_add_(0, inv.cpu(), dout[keep].double().cpu())


def test_batches_in_turn_over_one_workspace():
    """Calls back to back, each leaving its predecessor's entries in the workspace that it sorts into."""
    R, D = 5000, 64
    batches = [_batch(T, R, D, T) for T in (2049, 1, 700, 4000, 33, 1024)]
    ws = B.workspace(B.emb_grad_rows_workspace_size(4000, R, D), DEV)
    err = B.new_err(DEV)
    got = []
    torch.cuda.synchronize()
    for k in range(120):
        ids, dout = batches[k * 5 % 6 if k % 2 else k % 6]
        got.append((k, ids, dout, B.fs_emb_grad_rows(ids, dout, R, err=err, ws=ws)))
    B.check(err)
    want = {id(ids): _expect(ids, dout, R) for ids, dout in batches}
    for k, ids, dout, (rows, grads, count, _) in got:
        uniq, ref = want[id(ids)]
        n = uniq.numel()
        assert int(count) == n and torch.equal(rows[:n], uniq), k
        assert torch.equal(grads[:n].double().cpu(), ref), k


@pytest.mark.parametrize("R", [10_000_000, 1 << 31, (1 << 32) - 1])
@pytest.mark.parametrize("T", [1024, 1025, 2048, 3073, 4096, 4097, 6144, 6145, 8192])
def test_every_block_shape_and_number_of_passes(T, R):
    """One to eight entries a thread, three and four passes; IDs out of range sort behind the last row."""
    ids, dout = _batch(T, R, 32, T)
    for bad in (False, True):
        if bad:
            ids = ids.clone()
            ids[1], ids[T // 3], ids[T - 1] = -1, R, 1 << 40
        rows, grads, count, err = B.fs_emb_grad_rows(ids, dout, R, 2.0)
        assert int(err) == (2 if bad else 0)
        uniq, ref = _expect(ids, dout, R)
        n = uniq.numel()
        assert int(count) == n and torch.equal(rows[:n], uniq)
        assert torch.equal(grads[:n].double().cpu(), ref * 2)
