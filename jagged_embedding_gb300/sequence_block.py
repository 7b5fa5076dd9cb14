"""The first layer of a sequence model over the gathered rows of a jagged batch, with its gradients.

What stands between the embedding table and the rest of the model, in the library's calls:

    x  = sqrt(dim) * table[ids]                     fs_emb_lookup_scaled
    y  = norm(x)                                    fs_rmsnorm
    q, k, v = y @ w_qkv                             (library product)
    o  = attention inside each sample               fs_jagged_attn
    h  = x + o @ w_out;  out = norm(h)              fs_rmsnorm with the residual's addition
and back:
    d h, d gamma                                    fs_rmsnorm_backward
    d q, d k, d v                                   fs_jagged_attn_backward
    d x, d gamma                                    fs_rmsnorm_backward, the residual's gradient added
    rows, d table[rows]                             fs_emb_grad_rows

The batch is one that `Pipeline.prepare` leaves (IDs sample by sample, [UIH | candidates]) or any other jagged one.
Positions of no sample (before offsets[0], from offsets[-1] on, of a sample with bad offsets) attend to nothing: o = 0.
The row gradients are for an optimizer of the caller's own; the fused update (fs_emb_update_sorted) takes d x directly.
"""
from __future__ import annotations

import math

import torch

from . import binding as B


class SequenceBlock:
    """One pre-norm attention layer: bf16 activations and projections, fp32 norm weights."""

    def __init__(self, dim, heads, kv_heads, head_dim, device="cuda", eps=1e-6, generator=None):
        if heads % kv_heads:
            raise ValueError("heads must be a multiple of kv_heads")
        self.dim, self.heads, self.kv_heads, self.head_dim, self.eps = dim, heads, kv_heads, head_dim, eps
        self.scale = 1.0 / math.sqrt(head_dim)
        self.emb_scale = math.sqrt(dim)
        width = (heads + 2 * kv_heads) * head_dim

        def weight(rows, cols):
            w = torch.randn(rows, cols, device=device, generator=generator) / math.sqrt(rows)
            return w.to(torch.bfloat16)

        self.w_qkv, self.w_out = weight(dim, width), weight(heads * head_dim, dim)
        self.gamma_in = torch.ones(dim, device=device)
        self.gamma_out = torch.ones(dim, device=device)
        self.err = B.new_err(device)
        self._ws = {}

    def _workspace(self, name, nbytes, device):
        """Workspaces are kept and grow with the batch, each for the current stream alone: calls on several streams
        may run at once, and what a stream outgrows is freed in that stream's order."""
        key = name, device, B.current_stream(device)
        ws = self._ws.get(key)
        if ws is None or ws.numel() < nbytes:
            ws = self._ws[key] = B.workspace(nbytes, device)
        return ws

    def forward(self, table, ids, offsets, cand_len=None, bits8=False):
        """Returns (out, out_scale, saved): out [T, dim] in bf16, or with bits8 in torch.float8_e4m3fn with a scale per
        row (out_scale, None otherwise)."""
        T, H, Hkv, Dh = ids.numel(), self.heads, self.kv_heads, self.head_dim
        x, _ = B.fs_emb_lookup_scaled(table, ids, self.emb_scale, out_dtype=torch.bfloat16, err=self.err)
        y, _, _, rstd = B.fs_rmsnorm(x, self.gamma_in, self.eps)
        qkv = (y @ self.w_qkv).view(T, H + 2 * Hkv, Dh)
        q, k, v = qkv.split([H, Hkv, Hkv], dim=1)
        ws = self._workspace("attn", B.jagged_attn_workspace_size(T, offsets.numel() - 1, H, Hkv, Dh), ids.device)
        # positions of no sample are left as they are by the call, and the products take every position
        o = torch.zeros(T, H, Dh, dtype=torch.bfloat16, device=ids.device)
        _, lse, _ = B.fs_jagged_attn(q, k, v, offsets, self.scale, cand_len=cand_len, out=o, err=self.err, ws=ws)
        z = o.view(T, H * Dh) @ self.w_out
        out, out_scale, h, rstd_out = B.fs_rmsnorm(z, self.gamma_out, self.eps, res=x,
                                                   y_dtype=torch.float8_e4m3fn if bits8 else None)
        saved = (ids, offsets, cand_len, x, rstd, y, qkv, o, lse, h, rstd_out, table.shape[0])
        return out, out_scale, saved

    def backward(self, dout, saved, dh=None, grad_dtype=torch.float32):
        """Gradients from dout [T, dim] (of the unrounded output) and dh, the gradient that reaches h by other ways.
        Returns a dict: rows, row_grads, count (the table's, see fs_emb_grad_rows), w_qkv, w_out, gamma_in, gamma_out."""
        ids, offsets, cand_len, x, rstd, y, qkv, o, lse, h, rstd_out, num_rows = saved
        T, H, Hkv, Dh = ids.numel(), self.heads, self.kv_heads, self.head_dim
        norm_ws = self._workspace("norm", B.rmsnorm_backward_workspace_size(T, self.dim), ids.device)
        dz, dgamma_out = B.fs_rmsnorm_backward(dout, h, self.gamma_out, rstd_out, dsum=dh, ws=norm_ws)
        do = (dz @ self.w_out.T).view(T, H, Dh)
        dw_out = o.view(T, H * Dh).T @ dz
        dqkv = torch.zeros_like(qkv)  # (as o in the forward pass)
        q, k, v = qkv.split([H, Hkv, Hkv], dim=1)
        dq, dk, dv = dqkv.split([H, Hkv, Hkv], dim=1)
        ws = self._workspace("attn", B.jagged_attn_workspace_size(T, offsets.numel() - 1, H, Hkv, Dh), ids.device)
        B.fs_jagged_attn_backward(q, k, v, o, lse, do, offsets, self.scale, cand_len=cand_len, dq=dq, dk=dk, dv=dv,
                                  err=self.err, ws=ws)
        flat = dqkv.view(T, (H + 2 * Hkv) * Dh)
        dx, dgamma_in = B.fs_rmsnorm_backward(flat @ self.w_qkv.T, x, self.gamma_in, rstd, dsum=dz, ws=norm_ws)
        grad_ws = self._workspace("rows", B.emb_grad_rows_workspace_size(T, num_rows, self.dim), ids.device)
        rows, row_grads, count, _ = B.fs_emb_grad_rows(ids, dx, num_rows, self.emb_scale, grad_dtype=grad_dtype,
                                                       err=self.err, ws=grad_ws)
        return {"rows": rows, "row_grads": row_grads, "count": count, "w_qkv": y.T @ flat, "w_out": dw_out,
                "gamma_in": dgamma_in, "gamma_out": dgamma_out}

    def check(self):
        """Wait for the stream and raise if any call reported an error."""
        B.check(self.err, "SequenceBlock")
