"""Host checks of the sequence-block calls: bad arguments are refused before anything is launched (no GPU needed)."""
import ctypes as C

import pytest
import torch

from jagged_embedding_gb300 import binding as B

P = C.c_void_p
ERR, WS, BIG = P(0x1000), P(0x2000), 1 << 40


def _swap(args, at, value):
    return args[:at] + [value] + args[at + 1:]


def test_lookup_refusals():
    f = B.lib().fs_emb_lookup_scaled
    a = [P(0x100), 10, 64, 0, P(0x200), 5, C.c_float(1), P(0x300), 1, ERR, None]
    for at, v in ((0, None), (1, 0), (2, 0), (3, 2), (3, 7), (4, None), (5, -1), (5, 1 << 31), (7, None), (8, 2), (9, None)):
        assert f(*_swap(a, at, v)) == 1, (at, v)
    for at, v in ((0, P(0x102)), (4, P(0x204)), (7, P(0x301))):
        assert f(*_swap(a, at, v)) == 8, (at, v)
    assert f(*_swap(a, 5, 0)) == 0


def test_row_grads_refusals():
    L = B.lib()
    need = L.fs_emb_grad_rows_workspace_size(50, 1000, 64)
    assert need > 0 and L.fs_emb_grad_rows_workspace_size(-1, 1000, 64) == 0
    assert L.fs_emb_grad_rows_workspace_size(50, 0, 64) == 0 and L.fs_emb_grad_rows_workspace_size(50, 1 << 32, 64) == 0
    a = [1000, 64, P(0x200), 50, P(0x300), 0, C.c_float(1), P(0x400), P(0x500), 0, 50, P(0x600), ERR, WS, need, None]
    for at, v in ((0, 0), (0, 1 << 32), (1, 0), (2, None), (3, -1), (4, None), (5, 2), (7, None), (8, None), (9, 5), (10, -1),
                  (11, None), (12, None)):
        assert L.fs_emb_grad_rows(*_swap(a, at, v)) == 1, (at, v)
    for at, v in ((2, P(0x204)), (4, P(0x302)), (7, P(0x404)), (8, P(0x502)), (11, P(0x604))):
        assert L.fs_emb_grad_rows(*_swap(a, at, v)) == 8, (at, v)
    assert L.fs_emb_grad_rows(*_swap(a, 14, need - 1)) == 5 and L.fs_emb_grad_rows(*_swap(a, 13, None)) == 5


def test_norm_refusals():
    L = B.lib()
    f32 = C.c_float
    a = [P(0x100), P(0x200), 5, 64, 1, P(0x300), f32(1e-6), P(0x400), P(0x500), 2, P(0x600), None, None]
    for at, v in ((0, None), (1, None), (2, -1), (3, 0), (3, 8193), (4, 2), (5, None), (6, f32(-1)), (6, f32(float("nan"))),
                  (7, None), (8, None), (9, 0), (10, None)):
        assert L.fs_rmsnorm(*_swap(a, at, v)) == 1, (at, v)
    assert L.fs_rmsnorm(*_swap(a, 9, 1)) == 1        # a scale without 8 bits
    for at, v in ((0, P(0x101)), (5, P(0x302)), (10, P(0x602)), (11, P(0x702))):
        assert L.fs_rmsnorm(*_swap(a, at, v)) == 8, (at, v)
    assert L.fs_rmsnorm(*_swap(a, 2, 0)) == 0
    need = L.fs_rmsnorm_backward_workspace_size(5, 64)
    assert need > 0 and L.fs_rmsnorm_backward_workspace_size(5, 8193) == 0
    b = [P(0x100), P(0x200), P(0x300), 5, 64, 0, P(0x400), P(0x500), P(0x600), P(0x700), P(0x2000), need, None]
    for at, v in ((0, None), (2, None), (3, -1), (4, 0), (5, 2), (6, None), (7, None), (8, None), (9, None)):
        assert L.fs_rmsnorm_backward(*_swap(b, at, v)) == 1, (at, v)
    for at, v in ((0, P(0x102)), (1, P(0x202)), (9, P(0x701)), (10, P(0x2008))):
        assert L.fs_rmsnorm_backward(*_swap(b, at, v)) == 8, (at, v)
    assert L.fs_rmsnorm_backward(*_swap(b, 11, need - 1)) == 5


def test_attention_refusals():
    L = B.lib()
    need = L.fs_jagged_attn_workspace_size(100, 4, 8, 2, 64)
    assert need > 0 and L.fs_jagged_attn_workspace_size(100, 4, 8, 2, 96) == 0
    f32 = C.c_float
    a = [P(0x100), 768, P(0x200), 768, P(0x300), 768, P(0x400), 4, 100, 8, 2, 64, P(0x500), 1, f32(0.1), P(0x600),
         P(0x700), ERR, WS, need, None]
    bad = ((0, None), (1, 511), (2, None), (3, 127), (4, None), (6, None), (7, -1), (8, -1), (8, 1 << 31), (9, 7), (9, 1),
           (10, 0), (11, 96), (11, 32), (14, f32(0)), (14, f32(-1)), (14, f32(float("inf"))), (14, f32(float("nan"))),
           (15, None), (16, None), (17, None))
    for at, v in bad:
        assert L.fs_jagged_attn(*_swap(a, at, v)) == 1, (at, v)
    for at, v in ((0, P(0x108)), (1, 770), (2, P(0x202)), (5, 772), (6, P(0x404)), (12, P(0x502)), (15, P(0x604)),
                  (16, P(0x702))):
        assert L.fs_jagged_attn(*_swap(a, at, v)) == 8, (at, v)
    assert L.fs_jagged_attn(*_swap(a, 19, need - 1)) == 5 and L.fs_jagged_attn(*_swap(a, 18, None)) == 5
    assert L.fs_jagged_attn(*_swap(a, 8, 0)) == 0
    b = [P(0x100), 768, P(0x200), 768, P(0x300), 768, P(0x600), P(0x700), P(0x800), P(0x400), 4, 100, 8, 2, 64, P(0x500), 1,
         f32(0.1), P(0x900), 768, P(0xa00), 768, P(0xb00), 768, ERR, WS, need, None]
    for at, v in ((0, None), (6, None), (7, None), (8, None), (9, None), (12, 9), (14, 80), (18, None), (19, 256), (20, None),
                  (21, 64), (22, None), (24, None)):
        assert L.fs_jagged_attn_backward(*_swap(b, at, v)) == 1, (at, v)
    for at, v in ((8, P(0x808)), (18, P(0x904)), (19, 770), (22, P(0xb02))):
        assert L.fs_jagged_attn_backward(*_swap(b, at, v)) == 8, (at, v)
    assert L.fs_jagged_attn_backward(*_swap(b, 26, need - 1)) == 5


def test_binding_refuses_cpu_tensors():
    x, i = torch.zeros(4, 64), torch.zeros(4, dtype=torch.int64)
    g = torch.ones(64)
    h = torch.zeros(4, 1, 64, dtype=torch.bfloat16)
    for f in (lambda: B.fs_emb_lookup_scaled(x, i), lambda: B.fs_emb_grad_rows(i, x, 10), lambda: B.fs_rmsnorm(x, g, 1e-6),
              lambda: B.fs_rmsnorm_backward(x, x, g, torch.ones(4)), lambda: B.fs_jagged_attn(h, h, h, i, 0.1),
              lambda: B.fs_jagged_attn_backward(h, h, h, h, torch.zeros(1, 4), h, i, 0.1)):
        with pytest.raises(B.FsError):
            f()
