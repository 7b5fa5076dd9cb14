"""Sequence-block calls in a CUDA graph: captured once, replayed on other inputs (GPU)."""
import pytest
import torch

from jagged_embedding_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16, E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn


@pytest.mark.parametrize("lens", [[200, 0, 31, 90], [700, 1, 400] * 30])
def test_replay_equals_the_calls(lens):
    """Small batches take other launches than large ones (one cluster, one sorting block, no lists): both forms."""
    T, R, D, H, Hkv, Dh = sum(lens), 5000, 64, 4, 2, 64
    off = torch.tensor([0] + lens, device=DEV).cumsum(0)
    cand = torch.tensor([min(n, 5) for n in lens], dtype=torch.int32, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    table = torch.randn(R, D, generator=g, device=DEV)
    gamma = 1 + 0.1 * torch.randn(D, generator=g, device=DEV)
    inputs = [(torch.randint(0, R, (T,), generator=g, device=DEV),
               *(torch.randn(T, n, Dh, generator=g, device=DEV).to(BF16) for n in (H + 2 * Hkv, H)),
               torch.randn(T, D, generator=g, device=DEV).to(BF16)) for _ in range(3)]
    ids, qkv, dout, dy = (torch.empty_like(x) for x in inputs[0])
    ws = {"rows": B.workspace(B.emb_grad_rows_workspace_size(T, R, D), DEV),
          "norm": B.workspace(B.rmsnorm_backward_workspace_size(T, D), DEV),
          "attn": B.workspace(B.jagged_attn_workspace_size(T, len(lens), H, Hkv, Dh), DEV)}
    err = B.new_err(DEV)

    def calls():
        q, k, v = qkv.split([H, Hkv, Hkv], dim=1)
        x, _ = B.fs_emb_lookup_scaled(table, ids, 8.0, out_dtype=BF16, err=err)
        y, scale, h, rstd = B.fs_rmsnorm(x, gamma, 1e-6, res=dy, y_dtype=E4M3)
        out, lse, _ = B.fs_jagged_attn(q, k, v, off, 0.125, cand_len=cand, err=err, ws=ws["attn"])
        dq, dk, dv, _ = B.fs_jagged_attn_backward(q, k, v, out, lse, dout, off, 0.125, cand_len=cand, err=err, ws=ws["attn"])
        dh, dgamma = B.fs_rmsnorm_backward(dy, h, gamma, rstd, ws=ws["norm"])
        rows = torch.zeros(min(T, R), dtype=torch.int64, device=DEV)
        grads = torch.zeros(min(T, R), D, device=DEV)
        _, _, count, _ = B.fs_emb_grad_rows(ids, dh, R, 8.0, rows=rows, row_grads=grads, err=err, ws=ws["rows"])
        return x, y.view(torch.uint8), scale, h, rstd, out, lse, dq, dk, dv, dh, dgamma, rows, grads, count

    def load(i):
        for to, x in zip((ids, qkv, dout, dy), inputs[i]):
            to.copy_(x)

    load(0)
    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        calls()
    torch.cuda.current_stream().wait_stream(s)
    with torch.cuda.graph(graph):
        got = calls()
    for i in (1, 2, 0):
        load(i)
        graph.replay()
        B.check(err)
        kept = [x.clone() for x in got]
        want = calls()
        B.check(err)
        for k, (a, b) in enumerate(zip(kept, want)):
            assert torch.equal(a, b), k
