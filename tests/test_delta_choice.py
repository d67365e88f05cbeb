"""From how many tokens on the gated delta rule goes in chunks (a workspace is needed for them)."""
import pytest
import torch

import linear_rnn_recurrent_amd as L


@pytest.mark.parametrize("batch,heads,d,least", [(1, 32, 128, 18), (64, 32, 128, 18), (64, 8, 256, 18), (1, 8, 64, 18),
                                                 (32, 8, 64, 18), (64, 8, 64, 36), (1, 8, 32, 24), (64, 8, 32, 50)])
@pytest.mark.parametrize("io", [torch.bfloat16, torch.float16, torch.float32])
def test_tokens_from_which_chunks_are_taken(batch, heads, d, least, io):
    need = [L.delta_workspace_bytes(batch, t, heads // 2, heads, d, io) for t in (1, least - 1, least, 4096)]
    assert need[0] == need[1] == 0 and need[2] > 0 and need[3] > 0
