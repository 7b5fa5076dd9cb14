"""Row strides that the attention calls hand over (no GPU needed)."""
import pytest
import torch

from jagged_embedding_gb300 import binding as B

CPU = torch.device("cpu")


def test_the_stride_of_a_single_row_does_not_count():
    """A dimension of one has no stride of its own: 68 or 1 there must not refuse rows that are in order."""
    x = torch.zeros(5, 1, 68, dtype=torch.bfloat16)
    assert B._rows(x[2:3, :, :64], 1, 1, 64, "q", CPU) == 64
    assert B._rows(torch.as_strided(x, (1, 2, 64), (1, 64, 1)), 1, 2, 64, "q", CPU) == 128
    assert B._rows(torch.empty(0, 2, 64, dtype=torch.bfloat16), 0, 2, 64, "q", CPU) == 128


def test_the_stride_of_several_rows_is_theirs():
    x = torch.zeros(5, 6, 64, dtype=torch.bfloat16)
    q, k, v = x.split([4, 1, 1], dim=1)
    assert [B._rows(t, 5, t.shape[1], 64, "t", CPU) for t in (q, k, v)] == [384] * 3
    assert B._rows(x[::2, :2], 3, 2, 64, "t", CPU) == 768
    for bad in (x.transpose(0, 1), x.transpose(1, 2), x[:, ::2]):
        with pytest.raises(B.FsError):
            B._rows(bad, *bad.shape, "t", CPU)


def test_rows_that_share_memory_are_refused():
    """Fewer elements between two rows than a row has (an expanded tensor): the library refuses the stride."""
    x = torch.zeros(1, 2, 64, dtype=torch.bfloat16).expand(4, 2, 64)
    s = B._rows(x, 4, 2, 64, "k", CPU)
    P, F = B.C.c_void_p, B.C.c_float
    need = B.lib().fs_jagged_attn_workspace_size(4, 1, 2, 2, 64)
    assert B.lib().fs_jagged_attn(P(0x100), 128, P(0x200), s, P(0x300), 128, P(0x400), 1, 4, 2, 2, 64, None, 1, F(0.1),
                                  P(0x600), P(0x700), P(0x1000), P(0x2000), need, None) == 1
