"""Calls of the convolution, scan and draft verification at the edges of what the
header allows: empty batches, streams, layouts."""
import pytest
import torch

import linear_rnn_recurrent_amd as L
from gpu_helpers import assert_bitwise

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("batch,seq_len", [(0, 64), (0, 1), (0, 2048), (3, 0), (0, 0)])
def test_empty_calls_do_nothing(batch, seq_len):
    dim, dstate = 96, 16
    new = lambda *s: torch.zeros(s, device="cuda")  # noqa: E731
    x = new(batch, seq_len, dim)
    B = new(batch, seq_len, 1, dstate)
    state, conv = torch.randn(4, dim, dstate, device="cuda"), torch.randn(4, dim, 3, device="cuda")
    before = state.clone(), conv.clone()
    idx = torch.zeros(batch, dtype=torch.int32, device="cuda")
    for out in (torch.empty_like(x), None):
        L.ssu_scan_prefill(x, -torch.ones(dim, dstate, device="cuda"), B, B, x.clone(), state, out,
                           state_indices=idx, context_lengths=idx)
        L.ssu_conv_prefill(x, new(dim, 4), None, conv, out, state_indices=idx, context_lengths=idx)
    if batch == 0:
        one = new(0, dim)
        L.ssu_scan_decode(one, -torch.ones(dim, dstate, device="cuda"), new(0, 1, dstate),
                          new(0, 1, dstate), one.clone(), state, one, state_indices=idx)
        L.ssu_conv_decode(one, new(dim, 4), None, conv, one, state_indices=idx)
        i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
        L.ssu_draft_verify(i32(0, 5), new(0, 5, 70000), new(0, 5), i32(0), i32(0))
    torch.cuda.synchronize()
    assert_bitwise(state, before[0], "state")
    assert_bitwise(conv, before[1], "conv_state")
