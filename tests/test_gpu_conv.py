"""The causal convolution (prompts, single tokens) against the fp64 oracle."""
import numpy as np
import pytest
import torch

import oracle
from linear_rnn_recurrent_amd import ssu_conv_decode, ssu_conv_prefill
from gpu_helpers import assert_bitwise, touched_rows
from sequence_helpers import check, conv_bound, conv_inputs, f64

pytestmark = pytest.mark.gpu


def run_both(T, *, silu=True, update=True, with_out=True, step=False):
    """Runs the call and the oracle on the same inputs and compares everything."""
    width = T["weight"].shape[1]
    ref_state = f64(T["conv_state"]).copy()
    ref, mag = oracle.causal_conv(f64(T["x"]), f64(T["weight"]), f64(T["bias"]), ref_state,
                                  silu=silu, ctx=f64(T["ctx"]), idx=f64(T["idx"]), update=update)
    state = T["conv_state"]
    before = state.cpu()
    out = torch.full(T["x"].shape, float("nan"), dtype=T["x"].dtype, device="cuda")
    if step:
        ssu_conv_decode(T["x"][:, 0], T["weight"], T["bias"], state, out[:, 0], silu=silu,
                        state_indices=T["idx"])
    else:
        ssu_conv_prefill(T["x"], T["weight"], T["bias"], state, out if with_out else None,
                         silu=silu, context_lengths=T["ctx"], state_indices=T["idx"],
                         update_state=update)
    torch.cuda.synchronize()
    if with_out:
        bound = conv_bound(ref, mag, width) if silu else (width + 1) * 2.0 ** -24 * mag
        check(out, ref, bound, out.dtype, "out")
        zero = (ref == 0) & (mag == 0)
        assert not np.signbit(f64(out)[zero]).any()  # +0.0 past a row's end
    if width > 1:
        # kept inputs are copies: rounded once to the pool's type; the other rows keep their bits
        want = before.clone()
        rows = touched_rows(T["idx"], T["x"].shape[0])
        want[rows] = torch.from_numpy(ref_state[rows]).to(state.dtype)
        assert_bitwise(state, want, "conv_state")
    return out


@pytest.mark.parametrize("width", [1, 2, 3, 4, 5, 8])
@pytest.mark.parametrize("io,wt,st", [("bf16", "bf16", "bf16"), ("f16", "f32", "f16"),
                                      ("f32", "f32", "f32"), ("bf16", "f16", "f32"),
                                      ("f32", "bf16", "f16")])
def test_types_and_widths(width, io, wt, st):
    run_both(conv_inputs(11 + width, batch=3, seq_len=21, channels=136, width=width, io=io, wt=wt,
                         st=st, ctx=[21, 9, 2]))


@pytest.mark.parametrize("channels", [1, 7, 64, 250, 514, 2056])
@pytest.mark.parametrize("seq_len", [1, 2, 3, 16, 17, 65])
def test_sizes(channels, seq_len):
    run_both(conv_inputs(channels + seq_len, batch=2, seq_len=seq_len, channels=channels, width=4))


@pytest.mark.parametrize("layout", ["chan", "tap", "padded"])
@pytest.mark.parametrize("wide", [0, 1, 16, 128])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_strides(layout, wide, io):
    run_both(conv_inputs(5, batch=3, seq_len=19, channels=128, width=4, io=io, layout=layout,
                         wide=wide, ctx=[19, 1, 0], idx=[4, 0, 2], pool=6))


def test_lengths_shorter_than_the_window_empty_negative_and_too_long():
    for width in (2, 4, 8):
        T = conv_inputs(width, batch=9, seq_len=12, channels=72, width=width,
                        ctx=[0, 1, 2, 3, -5, 12, 99, 6, 7])
        for b, n in enumerate([0, 1, 2, 3, 0, 12, 12, 6, 7]):
            T["x"][b, n:] = float("nan")  # never read
        run_both(T)


def test_padding_rows_touch_nothing():
    T = conv_inputs(3, batch=4, seq_len=6, channels=64, width=4, idx=[2, -1, 0, -7], pool=5)
    T["x"][1] = float("nan")
    T["x"][3] = float("inf")
    T["conv_state"][[1, 3, 4]] = float("nan")
    run_both(T)


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("bias", [True, False])
def test_activation_and_bias(silu, bias):
    run_both(conv_inputs(8, batch=2, seq_len=9, channels=40, width=3, io="f32", bias=bias), silu=silu)


def test_large_values_through_silu():
    T = conv_inputs(9, batch=1, seq_len=8, channels=64, width=2, io="f32")
    T["x"] *= 200.0
    run_both(T)


def test_window_is_read_only_and_commit_takes_the_accepted_tokens():
    acc = [3, 0, 5, 1]
    T = conv_inputs(21, batch=4, seq_len=5, channels=320, width=4)
    before = T["conv_state"].clone()
    run_both(T, update=False)
    assert_bitwise(T["conv_state"], before, "pool after a window")
    T["ctx"] = torch.tensor(acc, dtype=torch.int32, device="cuda")
    run_both(T, with_out=False)


@pytest.mark.parametrize("channels,width,batch", [(5376, 4, 64), (70, 3, 3), (8, 1, 2), (33, 8, 5),
                                                  (2560, 2, 1)])
@pytest.mark.parametrize("layout", ["chan", "tap"])
@pytest.mark.parametrize("io,st", [("bf16", "bf16"), ("f32", "f16"), ("f16", "f32")])
def test_single_token(channels, width, batch, layout, io, st):
    run_both(conv_inputs(2, batch=batch, seq_len=1, channels=channels, width=width, io=io, st=st,
                         layout=layout), step=True)


def test_single_token_in_place_and_strided():
    T = conv_inputs(31, batch=6, seq_len=1, channels=96, width=4, idx=[5, -1, 0, 3, 8, 1], wide=32)
    ref = run_both({**T, "conv_state": T["conv_state"].clone()}, step=True)[:, 0]
    x, state = T["x"][:, 0], T["conv_state"]
    ssu_conv_decode(x, T["weight"], T["bias"], state, x, state_indices=T["idx"])
    assert_bitwise(x.contiguous(), ref.contiguous(), "out in x's place")


def test_prompt_is_its_tokens_one_by_one():
    T = conv_inputs(41, batch=3, seq_len=23, channels=200, width=4)
    out = run_both({**T, "conv_state": T["conv_state"].clone()})
    state = T["conv_state"]
    for t in range(23):
        one = torch.empty_like(out[:, t])
        ssu_conv_decode(T["x"][:, t], T["weight"], T["bias"], state, one, state_indices=T["idx"])
        assert_bitwise(one.contiguous(), out[:, t].contiguous(), f"token {t}")


def test_full_size_prompts():
    T = conv_inputs(51, batch=8, seq_len=512, channels=5376, width=4, pool=64,
                    ctx=[512, 64, 301, 77, 500, 3, 0, 129])
    run_both(T)


def test_rows_far_into_a_large_pool():
    """Row offsets past 2^31 elements."""
    channels, taps = 4096, 7
    rows = (1 << 31) // (channels * taps) + 40
    state = torch.zeros(rows, channels, taps, dtype=torch.bfloat16, device="cuda")
    T = conv_inputs(61, batch=2, seq_len=4, channels=channels, width=8, pool=2)
    state[[rows - 1, rows - 30]] = T["conv_state"]
    small = {**T, "idx": torch.tensor([0, 1], dtype=torch.int32, device="cuda")}
    want = run_both(small)
    out = torch.empty_like(T["x"])
    ssu_conv_prefill(T["x"], T["weight"], T["bias"], state, out,
                     state_indices=torch.tensor([rows - 1, rows - 30], dtype=torch.int32,
                                                device="cuda"))
    assert_bitwise(out, want, "out")
    assert_bitwise(state[[rows - 1, rows - 30]], small["conv_state"], "rows")


def test_graph_and_other_stream():
    T = conv_inputs(71, batch=4, seq_len=9, channels=256, width=4, ctx=[9, 4, 0, 7])
    start = T["conv_state"].clone()
    eager = run_both(T)
    after = T["conv_state"].clone()
    side = torch.cuda.Stream()
    out, step = torch.empty_like(T["x"]), torch.empty_like(T["x"][:, 0])
    g = torch.cuda.CUDAGraph()

    def calls():
        ssu_conv_prefill(T["x"], T["weight"], T["bias"], T["conv_state"], out,
                         context_lengths=T["ctx"], state_indices=T["idx"])
        ssu_conv_decode(T["x"][:, 1], T["weight"], T["bias"], T["conv_state"], step,
                        state_indices=T["idx"])

    with torch.cuda.graph(g):
        calls()
    ref_state = after.clone()
    ref_step = torch.empty_like(step)
    ssu_conv_decode(T["x"][:, 1], T["weight"], T["bias"], ref_state, ref_step,
                    state_indices=T["idx"])
    for rep in range(3):
        T["conv_state"].copy_(start)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert_bitwise(out, eager, f"out, replay {rep}")
        assert_bitwise(step, ref_step, f"step, replay {rep}")
        assert_bitwise(T["conv_state"], ref_state, f"state, replay {rep}")
    T["conv_state"].copy_(start)
    side.wait_stream(torch.cuda.current_stream())
    ssu_conv_prefill(T["x"], T["weight"], T["bias"], T["conv_state"], out, context_lengths=T["ctx"],
                     state_indices=T["idx"], stream=side)
    side.synchronize()
    assert_bitwise(out, eager, "out on another stream")
