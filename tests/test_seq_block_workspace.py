"""Workspaces that the sequence-block calls cannot use are refused before anything is launched (no GPU needed)."""
import ctypes as C

import pytest

from jagged_embedding_gb300 import binding as B

P = C.c_void_p
F = C.c_float
ERR = P(0x1000)


def _grad_rows(ws, size):
    return B.lib().fs_emb_grad_rows(1000, 64, P(0x200), 50, P(0x300), 0, F(1), P(0x400), P(0x500), 0, 50, P(0x600), ERR, ws,
                                    size, None)


def _norm_backward(ws, size):
    return B.lib().fs_rmsnorm_backward(P(0x100), P(0x200), P(0x300), 5, 64, 0, P(0x400), P(0x500), P(0x600), P(0x700), ws,
                                       size, None)


def _attention(ws, size):
    return B.lib().fs_jagged_attn(P(0x100), 768, P(0x200), 768, P(0x300), 768, P(0x400), 4, 100, 8, 2, 64, P(0x500), 1,
                                  F(0.1), P(0x600), P(0x700), ERR, ws, size, None)


def _attention_backward(ws, size):
    return B.lib().fs_jagged_attn_backward(P(0x100), 768, P(0x200), 768, P(0x300), 768, P(0x600), P(0x700), P(0x800),
                                           P(0x400), 4, 100, 8, 2, 64, P(0x500), 1, F(0.1), P(0x900), 768, P(0xa00), 768,
                                           P(0xb00), 768, ERR, ws, size, None)


@pytest.mark.parametrize("call", [_grad_rows, _norm_backward, _attention, _attention_backward])
def test_misaligned_small_or_missing(call):
    big = 1 << 40
    for at in (0x2001, 0x2004, 0x2008):
        assert call(P(at), big) == 8, hex(at)
    assert call(P(0x2000), 16) == 5 and call(None, big) == 5
