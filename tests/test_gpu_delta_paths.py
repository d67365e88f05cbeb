"""Gated delta rule in chunks: the forms of its kernels that other tests do not reach. Commits without
outputs, windows that leave the state, several segments of them, head ratios, workgroups of a whole head;
outputs by their own norm. Against the fp64 oracle."""
import numpy as np
import pytest
import torch

import linear_rnn_recurrent_amd as L
from gpu_helpers import assert_bitwise
from sequence_helpers import check, f64
from serving_helpers import delta_inputs, delta_reference, norm_error
from test_gpu_delta import call, verify
from test_gpu_delta_values import near

pytestmark = pytest.mark.gpu


def commit(T):
    """The state alone, against the oracle and by its own norm."""
    _, _, state, sbound = delta_reference(T)
    assert call(T, out=False) is None
    check(T["state"], state, sbound, T["state"].dtype, "committed")
    rows = [r for r in T["idx"].tolist() if r >= 0]
    near(T["state"][rows].float(), state[rows], T["v"].shape[1], T["v"].shape[-1], "committed", T["state"].dtype)


@pytest.mark.parametrize("io", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("seq_len", [18, 33, 64, 150, 200])
def test_commits_without_outputs(io, d, seq_len):
    T = delta_inputs(201, batch=3, seq_len=seq_len, d=d, io=io, ctx=[seq_len, seq_len // 2, 5])
    T["idx"][2] = -1
    commit(T)


@pytest.mark.parametrize("st", ["f16", "bf16"])
def test_commits_to_16_bit_states(st):
    commit(delta_inputs(202, batch=2, seq_len=90, d=64, st=st, row_pad=8))


@pytest.mark.parametrize("io", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("seq_len", [18, 33, 64, 150])
def test_long_windows_leave_the_state(io, d, seq_len):
    T = delta_inputs(203, batch=3, seq_len=seq_len, d=d, io=io, ctx=[seq_len, 0, seq_len - 7])
    verify(T, update=False)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hv", [(1, 1), (3, 3), (1, 8), (2, 6), (5, 20), (1, 5)])
@pytest.mark.parametrize("seq_len", [40, 150])
def test_head_ratios(io, hq, hv, seq_len):
    T = delta_inputs(204, batch=2, seq_len=seq_len, hq=hq, hv=hv, d=64, io=io)
    twin = {**T, "state": T["state"].clone()}
    verify(T)
    commit(twin)


@pytest.mark.parametrize("io,d,hv,batch", [("bf16", 128, 16, 9), ("bf16", 256, 8, 9), ("f16", 128, 16, 9),
                                           ("f16", 256, 8, 9), ("f32", 128, 16, 9), ("f32", 256, 8, 9),
                                           ("f32", 64, 16, 17), ("bf16", 64, 16, 17)])
@pytest.mark.parametrize("seq_len", [31, 70])
def test_many_heads(io, d, hv, batch, seq_len):
    """More than 256 workgroups of 64 value columns."""
    assert batch * hv * d > 256 * 64
    T = delta_inputs(205, batch=batch, seq_len=seq_len, hq=hv // 4, hv=hv, d=d, io=io)
    twin = {**T, "state": T["state"].clone()}
    out, bound, state, sbound = delta_reference(T)
    y = call(T)
    check(y, out, bound, y.dtype, "out")
    near(y.float(), out, seq_len, d, "out", y.dtype)
    check(T["state"], state, sbound, torch.float32, "state")
    near(T["state"], state, seq_len, d, "state")
    call(twin, out=False)
    check(twin["state"], state, sbound, torch.float32, "committed")


@pytest.mark.parametrize("io,d,hq,hv,batch", [("bf16", 128, 16, 32, 40), ("f32", 64, 16, 32, 40), ("f16", 128, 16, 32, 24)])
def test_segments_of_windows_and_commits(io, d, hq, hv, batch):
    """A workspace that holds a part of the chunks at a time: the read-only window and the commit
    against the call that does both."""
    seq_len = 420
    ctx = [seq_len - 61 * (i % 4) - (300 if i == 3 else 0) for i in range(batch)]
    T = delta_inputs(206, batch=batch, seq_len=seq_len, hq=hq, hv=hv, d=d, io=io, ctx=ctx)
    start = T["state"].clone()
    one = L.delta_workspace_bytes(1, seq_len, hq, hv, d, T["q"].dtype)
    assert L.delta_workspace_bytes(batch, seq_len, hq, hv, d, T["q"].dtype) - 4 * batch * hv * d * d < 0.9 * one * batch
    want = call(T)
    after = T["state"].clone()
    T["state"].copy_(start)
    assert_bitwise(call(T, update=False), want, "window")
    assert_bitwise(T["state"], start, "state")
    call(T, out=False)
    # two orders of the same sums of d + 64 products a step, over the longest row's steps
    lim = 2 * (np.sqrt(d + 64) + 3 * np.sqrt(seq_len)) * 2.0 ** -24
    assert norm_error(T["state"], f64(after)) <= lim


@pytest.mark.parametrize("io", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("seq_len", [5, 40, 150])
def test_outputs_by_their_own_norm(io, d, seq_len):
    T = delta_inputs(207, batch=2, seq_len=seq_len, d=d, io=io)
    out, _, state, _ = delta_reference(T)
    y = call(T)
    near(y.float(), out, seq_len, d, "out", y.dtype)
    near(T["state"], state, seq_len, d, "state")


@pytest.mark.parametrize("io", ["f32", "bf16", "f16"])
def test_calls_repeat_themselves(io):
    T = delta_inputs(208, batch=5, seq_len=210, hq=4, hv=16, d=128, io=io, ctx=[210, 3, 64, 100, 209])
    start = T["state"].clone()
    want = call(T)
    after = T["state"].clone()
    for _ in range(3):
        T["state"].copy_(start)
        assert_bitwise(call(T), want, "out")
        assert_bitwise(T["state"], after, "state")


@pytest.mark.parametrize("rows,n,group,block", [(515, 2048, 2048, 2048), (64, 5120, 5120, 128), (130, 4096, 128, 0)])
def test_norms_repeat_themselves(rows, n, group, block):
    g = torch.Generator().manual_seed(209)
    x = torch.randn(rows, n, generator=g).cuda().bfloat16()
    residual = torch.randn(rows, n, generator=g).cuda().bfloat16()
    w = (torch.randn(group, generator=g) * 0.2).cuda().bfloat16()
    seen = []
    for _ in range(4):
        r = residual.clone()
        y = torch.empty(rows, n, dtype=torch.float8_e4m3fn if block else torch.bfloat16, device="cuda")
        s = torch.empty(rows, n // block, device="cuda") if block else None
        L.ssu_rms_norm(x, w, y, residual=r, scales=s, group_size=group, unit_offset=True)
        seen.append([t.view(torch.uint8) for t in (y, r, s) if t is not None])
    for other in seen[1:]:
        assert all(torch.equal(a, b) for a, b in zip(seen[0], other))
