"""Jagged attention where sizes and offsets go to extremes (GPU)."""
import pytest
import torch

from jagged_embedding_gb300 import binding as B
from tests.helpers import Guarded

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16


def test_offsets_of_more_tiles_than_32_bits_count():
    """Offsets 0, T, 0, T, ...: every second sample is refused, the others describe 2^19 * 2^13 = 2^32 tiles, which
    is 0 in 32 bits.  The lists hold T / 128 + S entries: nothing may be listed, and nothing written."""
    T = S = 1 << 20
    offsets = torch.zeros(S + 1, dtype=torch.int64, device=DEV)
    offsets[1::2] = T
    x = torch.zeros(T, 1, 64, dtype=BF16, device=DEV)
    ws = Guarded(B.jagged_attn_workspace_size(T, S, 1, 1, 64), torch.uint8)
    out, lse = torch.full((T, 1, 64), 7.0, dtype=BF16, device=DEV), torch.full((1, T), 7.0, device=DEV)
    _, _, err = B.fs_jagged_attn(x, x, x, offsets, 0.1, out=out, lse=lse, ws=ws.t)
    assert int(err) == 3
    assert bool((out == 7).all()) and bool((lse == 7).all())
    d = [torch.full((T, 1, 64), 7.0, dtype=BF16, device=DEV) for _ in range(3)]
    _, _, _, err = B.fs_jagged_attn_backward(x, x, x, out, lse, x, offsets, 0.1, dq=d[0], dk=d[1], dv=d[2], ws=ws.t)
    assert int(err) == 3
    assert all(bool((t == 7).all()) for t in d)
    ws.check()
