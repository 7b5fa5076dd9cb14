"""Batches without rows: every pointer of an empty tensor is NULL, and the calls have nothing to do (no GPU needed)."""
import ctypes as C

import pytest

from jagged_embedding_gb300 import binding as B

P = C.c_void_p
F = C.c_float


@pytest.mark.parametrize("y_dtype", [1, 2])
def test_norm_of_no_rows(y_dtype):
    f = B.lib().fs_rmsnorm
    assert f(None, None, 0, 64, 1, P(0x300), F(1e-6), None, None, y_dtype, None, None, None) == 0
    assert f(None, None, 1, 64, 1, P(0x300), F(1e-6), None, None, y_dtype, None, None, None) == 1
    assert f(None, None, 0, 64, 1, P(0x300), F(1e-6), None, None, 1, P(0x600), None, None) == 1  # a scale without 8 bits


def test_lookup_and_attention_of_no_rows():
    L = B.lib()
    err = P(0x1000)
    assert L.fs_emb_lookup_scaled(P(0x100), 10, 64, 0, None, 0, F(1), None, 1, err, None) == 0
    assert L.fs_jagged_attn(None, 768, None, 768, None, 768, P(0x400), 4, 0, 8, 2, 64, P(0x500), 1, F(0.1), None, None,
                            err, None, 0, None) == 0
    assert L.fs_jagged_attn_backward(None, 768, None, 768, None, 768, None, None, None, P(0x400), 4, 0, 8, 2, 64,
                                     P(0x500), 1, F(0.1), None, 768, None, 768, None, 768, err, None, 0, None) == 0
