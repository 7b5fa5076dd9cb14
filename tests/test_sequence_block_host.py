"""Host side of the sequence block (no GPU needed)."""
import torch

from jagged_embedding_gb300 import binding as B
from jagged_embedding_gb300.sequence_block import SequenceBlock


def test_each_stream_has_its_own_workspaces(monkeypatch):
    blk = SequenceBlock(64, 2, 1, 64, device="cpu")
    cpu, now = torch.device("cpu"), [1]
    monkeypatch.setattr(B, "_stream", lambda device: now[0])
    first = blk._workspace("attn", 1000, cpu)
    assert blk._workspace("attn", 900, cpu) is first and blk._workspace("norm", 900, cpu) is not first
    now[0] = 2
    other = blk._workspace("attn", 1000, cpu)
    assert other is not first and other.data_ptr() != first.data_ptr()
    grown = blk._workspace("attn", 5000, cpu)
    assert grown.numel() >= 5000
    now[0] = 1
    assert blk._workspace("attn", 1000, cpu) is first  # (what another stream outgrows does not touch this one's)
