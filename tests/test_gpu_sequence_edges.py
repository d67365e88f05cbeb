"""Calls of the convolution, scan and draft verification at the edges of what the
header allows: empty batches, streams, layouts."""
import numpy as np
import pytest
import torch

import linear_rnn_recurrent_amd as L
import oracle
from gpu_helpers import assert_bitwise, gpu
from linear_rnn_recurrent_amd import inputs
from sequence_helpers import check, conv_inputs, f64, scan_bound, scan_inputs, verify_inputs

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


def _spy(monkeypatch, kept):
    """Keeps (address, stream current at the allocation) of every torch.empty."""
    empty = torch.empty

    def spied(*a, **k):
        t = empty(*a, **k)
        kept.append((t.data_ptr(), torch.cuda.current_stream(t.device).cuda_stream))
        return t

    monkeypatch.setattr(torch, "empty", spied)


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("op", ["scan", "verify"])
def test_scratch_of_a_call_on_another_stream(monkeypatch, op, handle):
    """A block freed on the current stream, where work on it may be pending, does not
    become the scratch of a call on another stream; the results are those of the
    current stream with no wait for the device between."""
    side, kept = torch.cuda.Stream(), []
    stream = side.cuda_stream if handle else side
    if op == "scan":
        T = scan_inputs(71, batch=1, seq_len=1900, dim=200, dstate=16)
        need = L.scan_workspace_bytes(1, 1900, 200, 16)

        def call(stream=None):
            out, state = torch.zeros_like(T["x"]), T["state"].clone()
            go = (lambda: L.ssu_scan_prefill(T["x"], T["A"], T["B"], T["C"], T["dt"], state, out,
                                             dt_bias=T["dt_bias"], D=T["D"], z=T["z"],
                                             state_indices=T["idx"], stream=stream))
            return go, (out, state)
    else:
        T = verify_inputs(72, batch=3, tokens=4, vocab=70001)
        need = L.verify_workspace_bytes(3, 70001)

        def call(stream=None):
            acc, nxt = (torch.full((3,), -7, dtype=torch.int32, device="cuda") for _ in range(2))
            go = (lambda: L.ssu_draft_verify(T["tokens"], T["target"], T["uniforms"], acc, nxt,
                                             draft_probs=T["draft"], stream=stream))
            return go, (acc, nxt)
    assert need > 0
    go, want = call()
    go()
    for _ in range(3):
        go, got = call(stream)
        side.wait_stream(torch.cuda.current_stream())
        block = torch.zeros(need, dtype=torch.uint8, device="cuda")  # in use on the current stream ..
        address = block.data_ptr()
        del block                                                    # .. and free to be handed out there
        with monkeypatch.context() as m:
            _spy(m, kept)
            go()
        assert [s for _, s in kept] == [side.cuda_stream] and kept.pop()[0] != address
        torch.cuda.current_stream().wait_stream(side)
        for a, b in zip(got, want):
            assert_bitwise(a, b, op)


@pytest.mark.parametrize("handle", [False, True])
def test_tensors_made_by_the_other_calls_on_another_stream(monkeypatch, handle):
    """The workspace of a tree verify, workspace and output of a gated-delta-rule step
    and the rows that a pool captures: allocated under the call's stream, with the
    results of the current stream."""
    side, kept = torch.cuda.Stream(), []
    stream = side.cuda_stream if handle else side
    w = inputs.tree_workload(batch=3, num_nodes=24, nheads=2, dim=32, dstate=32, ngroups=1,
                             pool_rows=5, seed=31)
    T = {k: gpu(v) for k, v in w.tensors.items()}
    g = inputs.gdn_workload(batch=5, hidden=256, num_q_heads=2, num_v_heads=4, head_dim=64,
                            conv_width=4, pool_rows=8, seed=32)
    G = {k: gpu(v) for k, v in g.tensors.items()}
    start = {k: G[k].clone() for k in ("conv_state", "ssm_state")}
    pool = L.SsuPool([(0, 0, (3, 40), torch.float32), (1, 0, (7,), torch.bfloat16)], 3)

    def calls(stream=None):
        out = torch.zeros_like(T["x"])
        conv, ssm = start["conv_state"].clone(), start["ssm_state"].clone()
        if stream is not None:
            side.wait_stream(torch.cuda.current_stream())
        L.ssu_tree_verify(T["x"], T["A"], T["B"], T["C"], T["dt"], T["state"], out, T["parent_ids"],
                          depths=T["depths"], dt_bias=T["dt_bias"], D=T["D"], z=T["z"],
                          state_indices=T["state_indices"], stream=stream)
        y = L.ssu_gdn_decode(G["hidden_states"], G["w_ba"], G["mixed_qkv"], G["conv_weight"],
                             G["conv_bias"], conv, G["A_log"], G["dt_bias"], g.dims["scale"], ssm,
                             G["state_indices"], num_q_heads=2, stream=stream)
        rows = pool.capture(1, stream=stream)
        if stream is not None:
            torch.cuda.current_stream().wait_stream(side)
        return [out, y, conv, ssm, *rows]

    want = calls()
    for _ in range(3):
        kept.clear()
        with monkeypatch.context() as m:
            _spy(m, kept)
            got = calls(stream)
        assert [s for _, s in kept] == [side.cuda_stream] * 5
        for a, b in zip(got, want):
            assert_bitwise(a, b, "result")


@pytest.mark.parametrize("order", [(0, 1, 2), (0, 2, 1), (1, 0, 2), (1, 2, 0), (2, 0, 1), (2, 1, 0)])
@pytest.mark.parametrize("io,channels,width", [("bf16", 72, 4), ("f32", 33, 3), ("f16", 16, 8)])
def test_pools_with_their_axes_in_any_order(order, io, channels, width):
    T = conv_inputs(81, batch=5, seq_len=9, channels=channels, width=width, io=io,
                    ctx=[9, 0, 2, 7, 1], idx=[6, 1, -1, 0, 3], pool=8)
    want = torch.empty_like(T["x"])
    dense = T["conv_state"].clone()
    pool = dense.permute(order).clone(memory_format=torch.contiguous_format)
    pool = pool.permute([order.index(i) for i in range(3)])
    assert pool.shape == dense.shape and torch.equal(pool, dense)
    kw = dict(context_lengths=T["ctx"], state_indices=T["idx"])
    L.ssu_conv_prefill(T["x"], T["weight"], T["bias"], dense, want, **kw)
    out = torch.empty_like(T["x"])
    L.ssu_conv_prefill(T["x"], T["weight"], T["bias"], pool, out, **kw)
    assert_bitwise(out, want, "out")
    assert_bitwise(pool, dense, "conv_state")
    one, ref = torch.empty_like(T["x"][:, 0]), torch.empty_like(T["x"][:, 0])
    L.ssu_conv_decode(T["x"][:, 1], T["weight"], T["bias"], dense, ref, state_indices=T["idx"])
    L.ssu_conv_decode(T["x"][:, 1], T["weight"], T["bias"], pool, one, state_indices=T["idx"])
    assert_bitwise(one, ref, "step")
    assert_bitwise(pool, dense, "conv_state after a step")


def sequence_major(t):
    """The same values with the token axis outside the batch axis."""
    return None if t is None else t.transpose(0, 1).contiguous().transpose(0, 1)


# Rows, sweeps of 4, 8 and 16 waves, chunks with one and several tiles, one chunk to a row.
@pytest.mark.parametrize("batch,seq_len,dim,dstate", [
    (3, 1, 40, 16), (64, 17, 600, 16), (8, 64, 2560, 16), (3, 40, 2000, 16), (2, 300, 33, 16), (2, 2000, 90, 12),
    (2, 300, 48, 128), (64, 20, 4000, 16)])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_sequence_major_scan(batch, seq_len, dim, dstate, io):
    T = scan_inputs(91, batch=batch, seq_len=seq_len, dim=dim, dstate=dstate, io=io, dt=io,
                    ctx=[seq_len - b % 3 for b in range(batch)])
    M = {k: sequence_major(v) if k in ("x", "z", "dt", "B", "C") else v for k, v in T.items()}
    got = []
    for src, out in ((T, torch.full_like(T["x"], 7.0)), (M, sequence_major(torch.full_like(T["x"], 7.0)))):
        state = T["state"].clone()
        L.ssu_scan_prefill(src["x"], T["A"], src["B"], src["C"], src["dt"], state, out,
                           dt_bias=T["dt_bias"], D=T["D"], z=src["z"], context_lengths=T["ctx"],
                           state_indices=T["idx"])
        got.append((out, state))
    assert batch == 1 or seq_len == 1 or got[1][0].stride() == (dim, batch * dim, 1)
    assert_bitwise(got[1][0], got[0][0], "out")
    assert_bitwise(got[1][1], got[0][1], "state")


@pytest.mark.parametrize("batch,seq_len,channels", [(4, 19, 128), (3, 2, 77), (8, 100, 1030)])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_sequence_major_conv(batch, seq_len, channels, io):
    T = conv_inputs(92, batch=batch, seq_len=seq_len, channels=channels, width=4, io=io,
                    ctx=[max(seq_len - 4 * b, 0) for b in range(batch)])
    got = []
    for f in (lambda t: t, sequence_major):
        pool, out = T["conv_state"].clone(), f(torch.full_like(T["x"], 7.0))
        L.ssu_conv_prefill(f(T["x"]), T["weight"], T["bias"], pool, out, context_lengths=T["ctx"],
                           state_indices=T["idx"])
        got.append((out, pool))
    assert_bitwise(got[1][0], got[0][0], "out")
    assert_bitwise(got[1][1], got[0][1], "conv_state")


@pytest.mark.parametrize("vocab", [2500, 70001])
def test_sequence_major_verification(vocab):
    T = verify_inputs(93, batch=5, tokens=6, vocab=vocab, sharp=6.0)
    got = []
    for f in (lambda t: t, sequence_major):
        acc, nxt = (torch.full((5,), -7, dtype=torch.int32, device="cuda") for _ in range(2))
        ids = torch.full((5, 6), -7, dtype=torch.int32, device="cuda")
        L.ssu_draft_verify(T["tokens"], f(T["target"]), T["uniforms"], acc, nxt, draft_probs=f(T["draft"]),
                           accepted_node_ids=ids)
        got.append((acc, nxt, ids))
    for a, b in zip(got[1], got[0]):
        assert_bitwise(a, b, "result")


@pytest.mark.parametrize("batch,seq_len,dim,dstate", [
    (64, 17, 600, 16), (8, 64, 2560, 16), (2, 300, 33, 16), (1, 512, 1536, 16), (1, 1900, 40, 16), (2, 300, 48, 128)])
def test_growth_past_fp32_leaves_a_state_of_zero(batch, seq_len, dim, dstate):
    """A positive entry of A over tokens without input: token by token a state of 0
    stays 0, although the growth over all of them is beyond fp32. Five tokens of
    input at the end. The exponent 12 is known to 2 u relative (A log2 e and its
    product with dt'), a factor of 24 u a token, over the five 120 u of the term:
    within the 6 u a token of the bound at 32 tokens or more, and within its 32 u
    more at 17."""
    T = scan_inputs(94, batch=batch, seq_len=seq_len, dim=dim, dstate=dstate, io="f32", gate=False, bias=False)
    T["A"][:, 2] = 12.0
    T["dt"][:] = 1.0
    T["x"][:, :-5] = 0.0
    T["state"].zero_()
    A, x, B, C, dt = (f64(T[k]) for k in ("A", "x", "B", "C", "dt"))
    state = np.zeros(T["state"].shape)
    ref, mag, smag = oracle.channel_scan(x, A, B, C, dt, state, D=f64(T["D"]), softplus=False, idx=f64(T["idx"]))
    assert np.abs(ref).max() < 1e30
    out = torch.full_like(T["x"], float("nan"))
    L.ssu_scan_prefill(T["x"], T["A"], T["B"], T["C"], T["dt"], T["state"], out, D=T["D"], dt_softplus=False,
                       state_indices=T["idx"])
    check(out, ref, scan_bound(mag, seq_len, dstate), torch.float32, "out")
    check(T["state"], state, scan_bound(smag, seq_len, 0), torch.float32, "state")


@pytest.mark.parametrize("batch,seq_len,dim,dstate", [(16, 5, 1100, 16), (8, 40, 1000, 24), (3, 2000, 90, 12)])
def test_several_windows_on_one_state(batch, seq_len, dim, dstate):
    """Read-only calls may name a pool row more than once: each window's outputs are
    those of the window alone."""
    T = scan_inputs(95, batch=batch, seq_len=seq_len, dim=dim, dstate=dstate, idx=[2] * batch)
    c = conv_inputs(96, batch=batch, seq_len=seq_len, channels=dim, width=4, idx=[1] * batch)
    pools = T["state"].clone(), c["conv_state"].clone()
    spread = T["state"][2:3].repeat(batch, 1, 1), c["conv_state"][1:2].repeat(batch, 1, 1)
    got = []
    for scan_pool, conv_pool, scan_idx, conv_idx in ((T["state"], c["conv_state"], T["idx"], c["idx"]),
                                                     (*spread, None, None)):
        out, u = torch.full_like(T["x"], 7.0), torch.full_like(c["x"], 7.0)
        L.ssu_scan_prefill(T["x"], T["A"], T["B"], T["C"], T["dt"], scan_pool, out, dt_bias=T["dt_bias"],
                           D=T["D"], z=T["z"], state_indices=scan_idx, update_state=False)
        L.ssu_conv_prefill(c["x"], c["weight"], c["bias"], conv_pool, u, state_indices=conv_idx,
                           update_state=False)
        got.append((out, u))
    for a, b in zip(*got):
        assert_bitwise(a, b, "window")
    assert_bitwise(T["state"], pools[0], "state")
    assert_bitwise(c["conv_state"], pools[1], "conv_state")


@pytest.mark.parametrize("fork", [False, True])
def test_calls_on_a_stream_of_their_own_in_a_graph(fork):
    """Captured with stream=, the capture's own or one that forks off it: the scratch
    stays the graph's, whatever is allocated and freed between replays."""
    T = scan_inputs(97, batch=1, seq_len=1900, dim=200, dstate=16)
    V = verify_inputs(98, batch=3, tokens=4, vocab=70001)
    start, out = T["state"].clone(), torch.zeros_like(T["x"])
    acc, nxt = (torch.full((3,), -7, dtype=torch.int32, device="cuda") for _ in range(2))
    side = torch.cuda.Stream()

    def calls(stream=None):
        L.ssu_scan_prefill(T["x"], T["A"], T["B"], T["C"], T["dt"], T["state"], out, dt_bias=T["dt_bias"],
                           D=T["D"], z=T["z"], state_indices=T["idx"], stream=stream)
        L.ssu_draft_verify(V["tokens"], V["target"], V["uniforms"], acc, nxt, draft_probs=V["draft"],
                           stream=stream)

    calls()
    want = [t.clone() for t in (out, T["state"], acc, nxt)]
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        here = torch.cuda.current_stream()
        stream = side if fork else here
        if fork:
            side.wait_stream(here)
        calls(stream)
        if fork:
            here.wait_stream(side)
    for rep in range(3):
        junk = [torch.full((n,), float("nan"), device="cuda") for n in (1 << 14, 1 << 18, 1 << 20, 1 << 22)]
        with torch.cuda.stream(side):
            junk += [torch.full((n,), float("nan"), device="cuda") for n in (1 << 14, 1 << 18, 1 << 20, 1 << 22)]
        T["state"].copy_(start)
        out.zero_(), acc.zero_(), nxt.zero_()
        torch.cuda.synchronize()
        kept = [t.clone() for t in junk]
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip((out, T["state"], acc, nxt), want):
            assert_bitwise(a, b, f"replay {rep}")
        for a, b in zip(junk, kept):
            assert_bitwise(a, b, "memory of others")
        del junk, kept


def test_commit_of_more_blocks_than_a_launch_holds():
    """A group of each channel, so that every channel is a block of its own: 2,252,800
    blocks, above the 2^21 that one launch of the last states takes. The reference is
    the recurrence in 64 bits."""
    batch, seq_len, dim, dstate = 2200, 17, 1024, 16
    g = torch.Generator(device="cuda").manual_seed(99)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x, dt = r(batch, seq_len, dim).bfloat16(), r(batch, seq_len, dim).bfloat16()
    B = r(batch, seq_len, dim, dstate).bfloat16()
    A, state = -torch.exp(r(dim, dstate)), r(batch, dim, dstate)
    h, mag = state.double(), state.double().abs()
    for t in range(seq_len):
        v = torch.nn.functional.softplus(dt[:, t].double())[..., None]
        decay, u = torch.exp(v * A.double()), B[:, t].double() * v * x[:, t].double()[..., None]
        h, mag = h * decay + u, mag * decay + u.abs()
    assert L.scan_workspace_bytes(batch, seq_len, dim, dstate, dim) > 0
    L.ssu_scan_prefill(x, A, B, None, dt, state, None)
    assert bool(((state.double() - h).abs() <= (32 + 6 * seq_len) * 2.0 ** -24 * mag + 1e-37).all())


def test_older_calls_on_a_forked_stream_in_a_graph():
    """What a tree verify and a gated-delta-rule step allocate for a stream that forks
    off a capture stays the graph's."""
    side = torch.cuda.Stream()
    w = inputs.tree_workload(batch=3, num_nodes=24, nheads=2, dim=32, dstate=32, ngroups=1, pool_rows=5, seed=33)
    T = {k: gpu(v) for k, v in w.tensors.items()}
    d = inputs.gdn_workload(batch=5, hidden=256, num_q_heads=2, num_v_heads=4, head_dim=64, conv_width=4,
                            pool_rows=8, seed=34)
    G = {k: gpu(v) for k, v in d.tensors.items()}
    start = {k: G[k].clone() for k in ("conv_state", "ssm_state")}
    out = torch.zeros_like(T["x"])

    def calls(stream=None):
        L.ssu_tree_verify(T["x"], T["A"], T["B"], T["C"], T["dt"], T["state"], out, T["parent_ids"],
                          depths=T["depths"], dt_bias=T["dt_bias"], D=T["D"], z=T["z"],
                          state_indices=T["state_indices"], stream=stream)
        return L.ssu_gdn_decode(G["hidden_states"], G["w_ba"], G["mixed_qkv"], G["conv_weight"], G["conv_bias"],
                                G["conv_state"], G["A_log"], G["dt_bias"], d.dims["scale"], G["ssm_state"],
                                G["state_indices"], num_q_heads=2, stream=stream)

    def reset():
        for k, v in start.items():
            G[k].copy_(v)
        out.zero_()

    y = calls()
    want = [t.clone() for t in (out, y, G["conv_state"], G["ssm_state"])]
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        y = calls(side)
        here.wait_stream(side)
    for rep in range(3):
        reset()
        junk = [torch.full((n,), float("nan"), device="cuda") for n in (1 << 8, 1 << 14, 1 << 18)]
        with torch.cuda.stream(side):
            junk += [torch.full((n,), float("nan"), device="cuda") for n in (1 << 8, 1 << 14, 1 << 18)]
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip((out, y, G["conv_state"], G["ssm_state"]), want):
            assert_bitwise(a, b, f"replay {rep}")
        assert all(bool(torch.isnan(t).all()) for t in junk)
