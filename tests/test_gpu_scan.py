"""The per-channel selective scan (prompts, single tokens) against the fp64 oracle."""
import numpy as np
import pytest
import torch

import oracle
from linear_rnn_recurrent_amd import ssu_scan_decode, ssu_scan_prefill
from gpu_helpers import assert_bitwise, untouched_rows
from sequence_helpers import check, f64, scan_bound, scan_inputs

pytestmark = pytest.mark.gpu


def call(T, out, *, update=True, softplus=True, step=False, state=None, stream=None):
    st = T["state"] if state is None else state
    if step:
        f = {k: None if T[k] is None else T[k][:, 0] for k in ("x", "B", "C", "dt", "z")}
        return ssu_scan_decode(f["x"], T["A"], f["B"], f["C"], f["dt"], st, out[:, 0],
                               dt_bias=T["dt_bias"], D=T["D"], z=f["z"], dt_softplus=softplus,
                               state_indices=T["idx"], stream=stream)
    return ssu_scan_prefill(T["x"], T["A"], T["B"], T["C"], T["dt"], st, out,
                            dt_bias=T["dt_bias"], D=T["D"], z=T["z"], dt_softplus=softplus,
                            context_lengths=T["ctx"], state_indices=T["idx"],
                            update_state=update, stream=stream)


def run_both(T, *, update=True, softplus=True, step=False, with_out=True):
    b, t, d = T["x"].shape
    n = T["B"].shape[-1]
    ref_state = f64(T["state"]).copy()
    ref, mag, smag = oracle.channel_scan(
        f64(T["x"]), f64(T["A"]), f64(T["B"]), f64(T["C"]), f64(T["dt"]), ref_state,
        dt_bias=f64(T["dt_bias"]), D=f64(T["D"]), z=f64(T["z"]), softplus=softplus,
        ctx=f64(T["ctx"]), idx=f64(T["idx"]), update=update)
    before = T["state"].clone()
    out = torch.full(T["x"].shape, float("nan"), dtype=T["x"].dtype, device="cuda")
    call(T, out if with_out else None, update=update, softplus=softplus, step=step)
    torch.cuda.synchronize()
    if with_out:
        check(out, ref, scan_bound(mag, t, n), out.dtype, "out")
        zero = (ref == 0) & (mag == 0)
        assert not np.signbit(f64(out)[zero]).any()  # +0.0 past a row's end
    idle = untouched_rows(T["idx"], T["state"].shape[0], b)
    if T["idx"] is None:
        idle = np.arange(b, T["state"].shape[0])
    assert_bitwise(T["state"][idle], before[idle], "rows of nobody")
    if not update:
        assert_bitwise(T["state"], before, "state read only")
        return out
    live = np.ones(T["state"].shape[0], bool)
    live[idle] = False
    check(T["state"][live], ref_state[live], scan_bound(smag[live], t, 0), T["state"].dtype, "state")
    return out


@pytest.mark.parametrize("io,dt,bc,st", [
    ("bf16", "bf16", "bf16", "f32"), ("f16", "f32", "f16", "f16"), ("f32", "f32", "f32", "f32"),
    ("bf16", "f32", "f32", "bf16"), ("f32", "f16", "bf16", "f32"), ("f16", "bf16", "f32", "bf16")])
@pytest.mark.parametrize("dstate", [4, 16, 24, 64])
def test_types_and_states(io, dt, bc, st, dstate):
    run_both(scan_inputs(dstate, batch=3, seq_len=19, dim=72, dstate=dstate, io=io, dt=dt, bc=bc,
                         st=st, ctx=[19, 7, 1]))


@pytest.mark.parametrize("dstate", [4, 8, 12, 16, 20, 32, 40, 64, 100, 128, 200, 256])
def test_every_lane_split(dstate):
    run_both(scan_inputs(1, batch=2, seq_len=37, dim=50, dstate=dstate, io="f32"))


@pytest.mark.parametrize("dim", [1, 3, 16, 63, 64, 65, 130, 514])
@pytest.mark.parametrize("seq_len", [1, 2, 8, 31, 64, 65, 129, 300])
def test_sizes(dim, seq_len):
    run_both(scan_inputs(dim + seq_len, batch=2, seq_len=seq_len, dim=dim, dstate=16, io="f32"))


@pytest.mark.parametrize("groups,dim", [(2, 64), (3, 51), (4, 260), (8, 8), (5, 500)])
@pytest.mark.parametrize("dstate", [8, 16, 64])
def test_groups(groups, dim, dstate):
    run_both(scan_inputs(groups, batch=2, seq_len=11, dim=dim, dstate=dstate, groups=groups))


@pytest.mark.parametrize("wide", [1, 3, 16, 64])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_strides(wide, io):
    run_both(scan_inputs(wide, batch=3, seq_len=70, dim=96, dstate=16, io=io, dt=io, wide=wide,
                         row_pad=32, ctx=[70, 33, 5]))


@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("D", [True, False])
@pytest.mark.parametrize("bias,softplus", [(True, True), (False, True), (True, False)])
def test_optional_inputs(gate, D, bias, softplus):
    T = scan_inputs(7, batch=2, seq_len=33, dim=40, dstate=16, gate=gate, D=D, bias=bias)
    if not softplus:
        T["dt"] = T["dt"].abs() * 0.2
        T["dt_bias"] = T["dt_bias"].abs() * 0.01
    run_both(T, softplus=softplus)


def test_lengths_empty_negative_too_long_and_nothing_read_past_them():
    T = scan_inputs(3, batch=7, seq_len=66, dim=80, dstate=16, ctx=[0, 1, -4, 66, 1000, 40, 63])
    for b, n in enumerate([0, 1, 0, 66, 66, 40, 63]):
        for k in ("x", "z", "dt", "B", "C"):
            T[k][b, n:] = float("nan")
    run_both(T)


def test_padding_rows_touch_nothing():
    T = scan_inputs(4, batch=4, seq_len=5, dim=64, dstate=16, idx=[3, -1, 0, -9], pool=6)
    for k in ("x", "z", "dt", "B", "C"):
        T[k][1], T[k][3] = float("nan"), float("inf")
    T["state"][[1, 2, 4, 5]] = float("nan")
    run_both(T)


def test_no_indices():
    run_both(scan_inputs(5, batch=3, seq_len=17, dim=48, dstate=16, idx="none", pool=5))


@pytest.mark.parametrize("scale", [0.0, 3.0, 40.0, 400.0])
def test_weak_and_strong_decay(scale):
    """dt' up to several hundred: decays from 1 to 0, dt' above softplus's linear
    range, states that collapse to the last token's term."""
    T = scan_inputs(6, batch=2, seq_len=70, dim=64, dstate=16, io="f32", dt_scale=1.0)
    T["dt"] *= scale
    if scale == 0.0:
        T["dt"] -= 200.0  # dt' = 0: the state stays
    run_both(T)


def test_window_is_read_only_and_commit_takes_the_accepted_tokens():
    T = scan_inputs(8, batch=4, seq_len=5, dim=320, dstate=16)
    run_both(T, update=False)
    T["ctx"] = torch.tensor([3, 0, 5, 1], dtype=torch.int32, device="cuda")
    run_both({**T, "state": T["state"].clone()})
    T["C"] = torch.full_like(T["C"], float("nan"))
    ref = scan_inputs(8, batch=4, seq_len=5, dim=320, dstate=16)
    ref["ctx"], full = T["ctx"], torch.empty_like(T["x"])
    call(ref, full)
    call(T, None)
    torch.cuda.synchronize()
    assert_bitwise(T["state"], ref["state"], "commit without outputs")


def test_long_prompt():
    run_both(scan_inputs(9, batch=1, seq_len=2048, dim=256, dstate=16, dt="bf16"))


@pytest.mark.parametrize("batch,seq_len,dim,dstate", [(8, 130, 2560, 16), (1, 200, 5120, 16),
                                                      (40, 33, 512, 16), (2, 77, 1536, 64),
                                                      (64, 5, 1030, 16), (3, 40, 600, 128)])
def test_many_workgroups(batch, seq_len, dim, dstate):
    run_both(scan_inputs(10, batch=batch, seq_len=seq_len, dim=dim, dstate=dstate))


# The library picks one of three evaluations by sizes. These reach, in order: rows
# of many and of few tokens; sweeping workgroups of 4, 8 and 16 waves, with one
# and several tiles of 16 states; chunks with one and several tiles, in teams of
# 4, 2 and 1, and one chunk to a row.
EVALUATIONS = [(64, 20, 640, 16), (64, 17, 600, 16), (2, 16, 70, 40), (64, 60, 48, 16), (6, 70, 500, 16), (3, 120, 90, 16),
               (4, 200, 33, 16), (70, 33, 40, 8), (20, 40, 130, 20), (2, 129, 64, 48), (1, 250, 48, 100),
               (1, 1900, 40, 16), (2, 2000, 90, 12), (1, 1850, 3, 16), (1, 600, 70, 64), (2, 300, 48, 128),
               (1, 290, 33, 256), (1, 280, 20, 200), (1, 70, 48, 40), (1, 200, 48, 40), (64, 20, 4000, 16),
               (64, 17, 600, 100), (32, 17, 600, 100)]


@pytest.mark.parametrize("batch,seq_len,dim,dstate", EVALUATIONS)
@pytest.mark.parametrize("kind", ["f32", "mixed", "commit", "window"])
def test_every_evaluation(batch, seq_len, dim, dstate, kind):
    """Uneven lengths (0, 1, all, too many among them), padding rows, strided
    views at odd offsets, padded pool rows; outputs and states; nothing read past
    a row's end."""
    g = np.random.default_rng(seq_len)
    ctx = g.integers(0, seq_len + 1, batch)
    ctx[0] = seq_len if batch < 3 else seq_len + 7
    if batch > 2:
        ctx[1], ctx[2] = 0, 1
    idx = g.permutation(batch + 2)[:batch]
    if batch > 3:
        idx[3] = -4
    T = scan_inputs(seq_len + dim, batch=batch, seq_len=seq_len, dim=dim, dstate=dstate,
                    io="f32" if kind == "f32" else "bf16", dt="f32" if kind == "f32" else "bf16",
                    st="f16" if kind == "mixed" else "f32", ctx=ctx.tolist(), idx=idx.tolist(),
                    wide=3 if kind == "mixed" else 4, row_pad=16, gate=kind != "f32")
    for b in range(batch):
        n = 0 if idx[b] < 0 else min(int(ctx[b]), seq_len)
        for k in ("x", "z", "dt", "B", "C"):
            if T[k] is not None:
                T[k][b, n:] = float("nan")
    run_both(T, update=kind != "window", with_out=kind != "commit")


@pytest.mark.parametrize("batch,seq_len,dim,groups,dstate", [(8, 64, 320, 4, 16), (1, 1900, 45, 3, 16),
                                                             (2, 300, 50, 2, 128), (40, 20, 60, 5, 16),
                                                             (1, 200, 96, 6, 32)])
def test_groups_in_every_evaluation(batch, seq_len, dim, groups, dstate):
    run_both(scan_inputs(5, batch=batch, seq_len=seq_len, dim=dim, groups=groups, dstate=dstate, io="f16"))


@pytest.mark.parametrize("batch,seq_len,dim,dstate", [(1, 1900, 40, 16), (6, 70, 500, 16), (2, 300, 48, 128)])
def test_infinite_state_entries_stay_where_they_are(batch, seq_len, dim, dstate):
    """An infinite entry of one channel's state touches that channel alone, and
    tokens past a row's end leave every entry, finite or not."""
    T = scan_inputs(6, batch=batch, seq_len=seq_len, dim=dim, dstate=dstate, io="f32", gate=False,
                    ctx=[seq_len - 5] * batch)
    row = int(T["idx"][0])
    clean = {**T, "state": T["state"].clone()}
    want = run_both(clean)
    T["A"][7, 2] = 0.0  # a decay of exactly 1
    T["state"][row, 7, 2] = float("inf")
    out = torch.empty_like(T["x"])
    call(T, out)
    torch.cuda.synchronize()
    assert torch.isinf(T["state"][row, 7, 2])
    keep = [c for c in range(dim) if c != 7]
    assert_bitwise(out[0][:, keep].contiguous(), want[0][:, keep].contiguous(), "other channels")
    assert not torch.isnan(T["state"][row][keep]).any()


@pytest.mark.parametrize("dstate", [4, 16, 24, 64, 256])
@pytest.mark.parametrize("io,dt,st", [("bf16", "bf16", "f32"), ("f32", "f32", "f16"),
                                      ("f16", "f32", "bf16")])
@pytest.mark.parametrize("batch,dim", [(1, 64), (5, 333), (64, 1024)])
def test_single_token(dstate, io, dt, st, batch, dim):
    if dstate == 256 and batch == 64:
        dim = 128
    run_both(scan_inputs(11, batch=batch, seq_len=1, dim=dim, dstate=dstate, io=io, dt=dt, st=st),
             step=True)


def test_single_token_padding_groups_strides():
    T = scan_inputs(12, batch=5, seq_len=1, dim=120, dstate=16, groups=3, wide=5, row_pad=16,
                    idx=[4, -1, 0, 7, -2], pool=8)
    run_both(T, step=True)


def test_single_token_in_place():
    for name in ("x", "z"):
        T = scan_inputs(13, batch=3, seq_len=1, dim=200, dstate=16)
        want = run_both({**T, "state": T["state"].clone()}, step=True)
        call(T, T[name], step=True)
        assert_bitwise(T[name], want, f"out in {name}'s place")


def test_prompt_is_its_tokens_one_by_one():
    T = scan_inputs(14, batch=2, seq_len=40, dim=96, dstate=16, io="f32")
    start = T["state"].clone()
    run_both(T)
    whole = T["state"]
    one = start.clone()
    for t in range(40):
        S = {k: (v[:, t:t + 1] if k in ("x", "z", "dt", "B", "C") else v) for k, v in T.items()}
        call(S, torch.empty(2, 1, 96, device="cuda"), step=True, state=one)
    ref = f64(one)
    check(whole, ref, scan_bound(np.abs(ref) + 8.0, 2 * 40, 0), torch.float32, "states")


def test_rows_far_into_a_large_pool():
    """Row offsets past 2^31 elements."""
    dim, n = 4096, 64
    rows = (1 << 31) // (dim * n) + 9
    T = scan_inputs(15, batch=2, seq_len=3, dim=dim, dstate=n, st="bf16", pool=2)
    big = torch.zeros(rows, dim, n, dtype=torch.bfloat16, device="cuda")
    big[[rows - 1, rows - 5]] = T["state"]
    out, want = torch.empty_like(T["x"]), torch.empty_like(T["x"])
    T["idx"] = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    call(T, want)
    far = torch.tensor([rows - 1, rows - 5], dtype=torch.int32, device="cuda")
    call({**T, "idx": far}, out, state=big)
    torch.cuda.synchronize()
    assert_bitwise(out, want, "out")
    assert_bitwise(big[[rows - 1, rows - 5]], T["state"], "rows")


def test_same_call_twice_is_bitwise_the_same():
    T = scan_inputs(16, batch=3, seq_len=150, dim=300, dstate=16)
    a, b = torch.empty_like(T["x"]), torch.empty_like(T["x"])
    s = T["state"].clone()
    call(T, a)
    call(T, b, state=s)
    assert_bitwise(a, b, "out")
    assert_bitwise(T["state"], s, "state")


def test_graph_and_other_stream():
    T = scan_inputs(17, batch=3, seq_len=70, dim=128, dstate=16, ctx=[70, 3, 41])
    start = T["state"].clone()
    out, step = torch.empty_like(T["x"]), torch.empty_like(T["x"])
    ref, ref_step, ref_state = torch.empty_like(out), torch.empty_like(step), start.clone()
    S = {k: (v[:, :1] if k in ("x", "z", "dt", "B", "C") else v) for k, v in T.items()}
    call(T, ref, state=ref_state)
    call(S, ref_step[:, :1], step=True, state=ref_state)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(T, out)
        call(S, step[:, :1], step=True)
    for rep in range(3):
        T["state"].copy_(start)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert_bitwise(out, ref, f"out, replay {rep}")
        assert_bitwise(step[:, 0].contiguous(), ref_step[:, 0].contiguous(), f"step, replay {rep}")
        assert_bitwise(T["state"], ref_state, f"state, replay {rep}")
    side = torch.cuda.Stream()
    T["state"].copy_(start)
    side.wait_stream(torch.cuda.current_stream())
    call(T, out, stream=side)
    side.synchronize()
    assert_bitwise(out, ref, "out on another stream")


@pytest.mark.parametrize("batch,seq_len,dim,dstate", [(1, 1900, 40, 16), (2, 300, 48, 128), (3, 40, 2000, 16),
                                                      (1, 600, 70, 64), (2, 129, 64, 48)])
def test_prompts_of_every_evaluation_in_a_graph(batch, seq_len, dim, dstate):
    """Several launches and a workspace of the call's own among them; the commit
    (no outputs) too."""
    T = scan_inputs(18, batch=batch, seq_len=seq_len, dim=dim, dstate=dstate)
    T["ctx"] = torch.full((batch,), seq_len - 3, dtype=torch.int32, device="cuda")
    start = T["state"].clone()
    ref, out = torch.empty_like(T["x"]), torch.empty_like(T["x"])
    ref_state = start.clone()
    call(T, ref, state=ref_state)
    call(T, None, state=ref_state)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(T, out)
        call(T, None)
    for rep in range(3):
        T["state"].copy_(start)
        out.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        junk = [torch.full((1 << 20,), float("nan"), device="cuda") for _ in range(4)]
        torch.cuda.synchronize()
        assert_bitwise(out, ref, f"out, replay {rep}")
        assert_bitwise(T["state"], ref_state, f"state, replay {rep}")
        del junk


def test_two_streams_at_once_with_workspaces_of_their_own():
    A = [scan_inputs(19 + i, batch=1, seq_len=1900, dim=200, dstate=16) for i in range(2)]
    want, outs = [], [torch.empty_like(a["x"]) for a in A]
    for a in A:
        o = torch.empty_like(a["x"])
        call(a, o, state=a["state"].clone())
        want.append(o)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in A]
    for _ in range(3):
        states = [a["state"].clone() for a in A]
        torch.cuda.synchronize()
        for a, o, st, s in zip(A, outs, states, streams):
            call(a, o, state=st, stream=s)
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert_bitwise(o, w, "out")


@pytest.mark.parametrize("batch,seq_len,dim,dstate", [(2, 1, 40, 16), (64, 17, 600, 16), (6, 70, 500, 16),
                                                      (4, 200, 33, 16), (1, 200, 48, 40), (1, 1900, 40, 16),
                                                      (2, 300, 48, 128)])
def test_infinite_decay_leaves_the_last_token_alone(batch, seq_len, dim, dstate):
    """Entries of A at -inf (or at -inf once scaled to powers of two) forget all but
    a token's own term, and tokens past a row's end do not touch them."""
    T = scan_inputs(8, batch=batch, seq_len=seq_len, dim=dim, dstate=dstate, io="f32",
                    ctx=[max(seq_len - 5 - b % 3, 1) for b in range(batch)])
    T["A"][:, 1] = -float("inf")
    T["A"][5, 3] = -3e38
    run_both(T)


def test_stream_by_object_and_by_handle():
    T = scan_inputs(4, batch=1, seq_len=1900, dim=40, dstate=16)
    s, outs = torch.cuda.Stream(), []
    for stream in (None, 0, s.cuda_stream, s):
        out, state = torch.empty_like(T["x"]), T["state"].clone()
        torch.cuda.synchronize()
        call(T, out, state=state, stream=stream)
        torch.cuda.synchronize()
        outs.append(out)
    for out in outs[1:]:
        assert_bitwise(out, outs[0], "out")
