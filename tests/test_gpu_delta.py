"""Gated delta rule on given q, k and v against the fp64 oracle."""
import numpy as np
import pytest
import torch

import linear_rnn_recurrent_amd as L
from gpu_helpers import assert_bitwise
from sequence_helpers import DT, check, f64
from serving_helpers import delta_inputs, delta_reference, norm_error

pytestmark = pytest.mark.gpu


def call(T, *, step=False, update=True, scale=None, l2=True, out=True, workspace=None):
    y = torch.full_like(T["v"], float("nan")) if out else None
    if not y is None and not y.is_contiguous():
        y = torch.full(T["v"].shape, float("nan"), dtype=T["v"].dtype, device="cuda")
    kw = dict(A_log=T["A_log"], dt_bias=T["dt_bias"], scale=scale, use_qk_l2norm=l2, state_indices=T["idx"])
    if step:
        L.ssu_delta_decode(T["q"], T["k"], T["v"], T["a"], T["b"], T["state"], y, **kw)
    else:
        L.ssu_delta_prefill(T["q"] if out else None, T["k"], T["v"], T["a"], T["b"], T["state"], y,
                            context_lengths=T["ctx"], update_state=update, workspace=workspace, **kw)
    torch.cuda.synchronize()
    return y


def verify(T, *, step=False, update=True, scale=None, l2=True):
    out, bound, state, sbound = delta_reference(T, step=step, scale=scale, l2=l2, update=update)
    before = T["state"].clone()
    y = call(T, step=step, update=update, scale=scale, l2=l2)
    check(y, out, bound, T["v"].dtype, "out")
    if not update:
        assert_bitwise(T["state"], before, "state")
        return y
    check(T["state"], state, sbound, T["state"].dtype, "state")
    # in the 2-norm roundings of either sign partly cancel: of d + 64 in each of n steps
    # (whose errors the decays and I - beta k k^T do not grow) remains the root
    n = 1 if step else T["v"].shape[1]
    lim = (8 + 4 * np.sqrt(T["v"].shape[-1] + 64) * np.sqrt(n)) * 2.0 ** -24
    lim += torch.finfo(T["state"].dtype).eps / 2 if T["state"].dtype != torch.float32 else 0.0
    assert norm_error(T["state"], state) <= lim
    return y


@pytest.mark.parametrize("io,gate,st", [("bf16", "f32", "f32"), ("f16", "f16", "f16"), ("f32", "f32", "f32"),
                                        ("bf16", "bf16", "bf16"), ("f32", "bf16", "f16"), ("f16", "f32", "bf16")])
@pytest.mark.parametrize("d", [32, 64, 128, 256])
def test_decode(io, gate, st, d):
    T = delta_inputs(1, batch=3, seq_len=1, hq=2, hv=4, d=d, io=io, gate=gate, st=st, step=True)
    T["idx"][1] = -1
    y = verify(T, step=True)
    assert_bitwise(y[1], torch.zeros_like(y[1]), "padding")


@pytest.mark.parametrize("hq,hv", [(1, 1), (3, 3), (1, 8), (2, 6), (5, 20)])
def test_head_layouts(hq, hv):
    verify(delta_inputs(2, batch=2, seq_len=1, hq=hq, hv=hv, d=64, step=True), step=True)
    verify(delta_inputs(3, batch=2, seq_len=9, hq=hq, hv=hv, d=64))


@pytest.mark.parametrize("io", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("seq_len", [1, 2, 5, 17])
def test_windows(io, d, seq_len):
    """A window with the state read only, then the commit of a part of it without outputs."""
    T = delta_inputs(4, batch=3, seq_len=seq_len, d=d, io=io)
    T["idx"][2] = -1
    verify(T, update=False)
    T["ctx"] = torch.tensor([seq_len // 2, seq_len, 1], dtype=torch.int32).cuda()
    _, _, state, sbound = delta_reference(T)
    before = T["state"].clone()
    call(T, out=False)
    check(T["state"], state, sbound, torch.float32, "committed")
    if seq_len == 1:
        assert_bitwise(T["state"][int(T["idx"][0])], before[int(T["idx"][0])], "nothing accepted")


@pytest.mark.parametrize("io", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("seq_len", [18, 31, 32, 33, 63, 64, 65, 97, 200, 331])
def test_prompts(io, d, seq_len):
    verify(delta_inputs(5, batch=2, seq_len=seq_len, d=d, io=io))


@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("st", ["f16", "bf16"])
def test_prompts_with_16_bit_states(d, st):
    verify(delta_inputs(6, batch=2, seq_len=150, d=d, st=st, gate="bf16"))


@pytest.mark.parametrize("io", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 128, 256])
def test_uneven_prompts(io, d):
    """Lengths from none to past the end, a padding row, NaN in every place that is not read, and
    zeros behind the ends."""
    T = delta_inputs(7, batch=7, seq_len=201, d=d, io=io, ctx=[201, 0, 1, 130, -4, 500, 64],
                     idx=[5, 2, 7, 0, 1, -1, 3], pool=9)
    live = [201, 0, 1, 130, 0, 0, 64]
    for i, n in enumerate(live):
        for name in ("q", "k", "v", "a", "b"):
            T[name][i, n:] = float("nan")
    T["state"][[1, 2, 4, 6, 8]] = float("nan")  # no one's, or of rows without tokens
    before = T["state"].clone()
    clean = {n: torch.nan_to_num(t, nan=0.0) if t is not None and t.is_floating_point() else t for n, t in T.items()}
    out, bound, state, sbound = delta_reference(clean)
    y = call(T)
    check(y, out, bound, DT[io], "out")
    for i, n in enumerate(live):
        assert_bitwise(y[i, n:], torch.zeros_like(y[i, n:]), "behind the end")
    for r in (1, 2, 4, 6, 8):
        assert_bitwise(T["state"][r], before[r], "untouched row")
    for r in (5, 7, 0, 3):
        check(T["state"][r], state[r], sbound[r], torch.float32, "state")


@pytest.mark.parametrize("io", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("l2", [True, False])
@pytest.mark.parametrize("seq_len", [3, 140])
def test_given_decays_and_betas(io, l2, seq_len):
    verify(delta_inputs(8, batch=2, seq_len=seq_len, d=64, io=io, raw=False, l2=l2), l2=l2, scale=0.3)


@pytest.mark.parametrize("io", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("seq_len", [4, 150])
@pytest.mark.parametrize("wide", [16, 6, 3])
def test_slices_of_wider_tensors(io, seq_len, wide):
    """Aligned to eight entries and not; pool rows with padding."""
    verify(delta_inputs(9, batch=2, seq_len=seq_len, d=64, io=io, wide=wide, row_pad=8))


@pytest.mark.parametrize("seq_len", [1, 6, 150])
def test_sequence_major_activations(seq_len):
    T = delta_inputs(10, batch=3, seq_len=seq_len, d=64)
    want = call({**T, "state": T["state"].clone()})
    for n in ("q", "k", "v", "a", "b"):
        T[n] = T[n].transpose(0, 1).contiguous().transpose(0, 1)
    assert_bitwise(call(T), want, "out")


@pytest.mark.parametrize("seq_len", [1, 7, 190])
@pytest.mark.parametrize("kind", ["reset", "strong", "none", "mixed"])
def test_decays(seq_len, kind):
    """Decays of 0 (a log of -inf), of nothing, far apart and near 1 next to far ones."""
    T = delta_inputs(11, batch=2, seq_len=seq_len, d=64, raw=False, gate="f32")
    g = torch.Generator().manual_seed(3)
    pick = torch.rand(T["a"].shape, generator=g).cuda()
    if kind == "reset":
        T["a"][pick < 0.05] = float("-inf")
    elif kind == "strong":
        T["a"].fill_(-1e4)
    elif kind == "none":
        T["a"].zero_()
    else:
        T["a"][pick < 0.2] = -90.0
        T["a"][pick > 0.6] = -1e-4
    if kind == "reset":  # the bound's factor |g| belongs to a decay of nothing: 0 there
        A = dict(T)
        A["a"] = T["a"].clamp_min(-750.0)
        out, _, state, _ = delta_reference(A)
        A["a"] = T["a"].clamp_min(-1.0)
        _, bound, _, sbound = delta_reference(A)
        y = call(T)
        # larger than the states of the real decays: those with a decay of e^-1 instead
        check(y, out, bound + 1e-5, torch.bfloat16, "out")
        check(T["state"], state, sbound + 1e-5, torch.float32, "state")
        return
    verify(T)


@pytest.mark.parametrize("io", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("seq_len", [2, 130])
@pytest.mark.parametrize("size", [1e-6, 1e4])
def test_small_and_large_values(io, seq_len, size):
    T = delta_inputs(12, batch=2, seq_len=seq_len, d=64, io=io)
    if io != "f16" or size < 1:
        T["v"] = (T["v"].float() * size).to(DT[io])
    T["state"] *= size
    T["k"][:, ::3] *= 0.01
    T["q"][:, 1::3] *= 30.0
    T["k"][:, 1] = 0.0
    verify(T)


@pytest.mark.parametrize("seq_len", [3, 135])
def test_equal_keys(seq_len):
    """The same key again and again with beta 1: every token writes over the one before."""
    T = delta_inputs(13, batch=2, seq_len=seq_len, d=64, raw=False, gate="f32")
    T["k"][:] = T["k"][:, :1]
    T["b"].fill_(1.0)
    T["a"].fill_(0.0)
    verify(T)


@pytest.mark.parametrize("io,seq_len,at", [("bf16", 150, 77), ("f16", 150, 64), ("bf16", 150, 127), ("bf16", 5, 2),
                                           ("f32", 150, 77)])
@pytest.mark.parametrize("where", ["q", "k", "v", "a", "b"])
def test_a_nan_reaches_no_earlier_token_and_no_other_row(io, seq_len, at, where):
    T = delta_inputs(14, batch=2, seq_len=seq_len, d=64, io=io)
    want = call({**T, "state": T["state"].clone()})
    T[where] = T[where].clone()
    T[where][1, at] = float("nan")
    y = call(T)
    assert torch.isfinite(y[0].float()).all() and torch.isfinite(y[1, :at].float()).all()
    assert torch.isnan(y[1, at].float()).all()
    assert torch.equal(y[0], want[0])
    near = (y[1, :at].float() - want[1, :at].float()).abs().max()
    assert near <= 4 * torch.finfo(DT[io]).eps * want.abs().max()


@pytest.mark.parametrize("seq_len", [3, 90])
def test_betas_up_to_two_and_growing_decays(seq_len):
    """beta of 2 reflects; a decay above 1 grows the state: followed as they are."""
    T = delta_inputs(15, batch=1, seq_len=seq_len, d=64, raw=False, gate="f32")
    T["b"] *= 2.0
    verify(T)
    T = delta_inputs(16, batch=1, seq_len=seq_len, d=64, raw=False, gate="f32")
    T["a"].fill_(0.02)
    T["a"][:, ::2] = -0.05
    verify(T)


def test_keys_longer_than_one_without_norm():
    """beta |k|^2 above 2 lets a state grow by every token; finite as long as it is, and the same
    in a prompt and token by token up to the rounding that grows with it."""
    T = delta_inputs(17, batch=1, seq_len=80, d=64, raw=False, gate="f32", l2=False)
    T["k"] = (T["k"].float() * 1.6).to(torch.bfloat16)
    T["b"].fill_(0.9)
    S = T["state"].clone()
    one = {**T, "state": S}
    steps = []
    for t in range(80):
        o = {**one, **{n: T[n][:, t] for n in ("q", "k", "v", "a", "b")}}
        steps.append(call(o, step=True, l2=False).float())
    y = call(T, l2=False).float()
    want = torch.stack(steps, 1)
    assert torch.isfinite(want).all() and torch.isfinite(y).all()
    # |1 - 0.9 * 1.58^2| = 1.25 a token at most; two evaluations, each off by (d + 64) roundings a token
    growth = 80 * 2 * (64 + 64) * 2.0 ** -24 * 1.25 ** 8
    assert (y - want).norm() <= (growth + 2 * 2.0 ** -8) * want.norm()


def test_prompt_as_two_prompts():
    T = delta_inputs(18, batch=2, seq_len=300, d=128)
    whole = {**T, "state": T["state"].clone()}
    verify(whole)
    first = {**T, **{n: T[n][:, :170] for n in ("q", "k", "v", "a", "b")}}
    call(first)
    second = {**T, **{n: T[n][:, 170:] for n in ("q", "k", "v", "a", "b")}}
    call(second)
    d = (T["state"] - whole["state"]).norm() / whole["state"].norm()
    assert d <= 2 * (8 + 4 * np.sqrt(192 * 300)) * 2.0 ** -24


@pytest.mark.parametrize("io,d", [("bf16", 128), ("f32", 64)])
def test_many_rows_as_rows_alone(io, d):
    """So many that their chunks are handed over in several segments and that a workgroup takes
    a whole head: as each row by itself, up to the rounding of either."""
    batch, seq_len, hq, hv = 24, 420, 8, 16
    ctx = [seq_len - 17 * (i % 5) - (400 if i == 7 else 0) for i in range(batch)]
    T = delta_inputs(24, batch=batch, seq_len=seq_len, hq=hq, hv=hv, d=d, io=io, ctx=ctx)
    rows = {**T, "state": T["state"].clone()}
    y = call(T)
    for i in (0, 7, 23):
        one = {n: (t[i:i + 1] if n in ("q", "k", "v", "a", "b", "idx", "ctx") else t) for n, t in rows.items()}
        want = call(one)
        n = max(ctx[i], 0)  # row 7 has none
        lim = 2 * (8 + 4 * np.sqrt((d + 64) * n)) * 2.0 ** -24
        assert norm_error(y[i].float(), f64(want[0].float())) <= lim + (2 * 2.0 ** -9 if io == "bf16" else 0.0)
        r = int(T["idx"][i])
        assert norm_error(T["state"][r], f64(rows["state"][r])) <= lim


@pytest.mark.parametrize("io,d,hq,hv", [("bf16", 128, 16, 32), ("f32", 64, 16, 32), ("f32", 256, 8, 16)])
def test_rows_in_several_segments(io, d, hq, hv):
    """A workspace that holds a part of the chunks at a time: as each row by itself, which fits."""
    batch, seq_len = 40, 420
    ctx = [seq_len - 61 * (i % 4) - (300 if i == 39 else 0) for i in range(batch)]
    T = delta_inputs(25, batch=batch, seq_len=seq_len, hq=hq, hv=hv, d=d, io=io, ctx=ctx)
    io_dtype = T["q"].dtype
    carry = 4 * batch * hv * d * d  # the states between segments, which a whole row's does not have
    assert (L.delta_workspace_bytes(batch, seq_len, hq, hv, d, io_dtype) - carry
            < 0.9 * L.delta_workspace_bytes(1, seq_len, hq, hv, d, io_dtype) * batch)
    rows = {**T, "state": T["state"].clone()}
    y = call(T)
    for i in (0, 17, 39):
        one = {n: (t[i:i + 1] if n in ("q", "k", "v", "a", "b", "idx", "ctx") else t) for n, t in rows.items()}
        want = call(one)
        lim = 2 * (8 + 4 * np.sqrt((d + 64) * max(ctx[i], 0))) * 2.0 ** -24
        assert norm_error(y[i].float(), f64(want[0].float())) <= lim + (2 * 2.0 ** -9 if io == "bf16" else 0.0)
        r = int(T["idx"][i])
        assert norm_error(T["state"][r], f64(rows["state"][r])) <= lim


def test_same_state_in_several_windows():
    T = delta_inputs(19, batch=3, seq_len=4, d=64)
    T["idx"][:] = 1
    verify(T, update=False)


def test_output_in_the_place_of_v():
    T = delta_inputs(20, batch=3, seq_len=1, d=128, step=True)
    want = call({**T, "state": T["state"].clone()}, step=True)
    v = T["v"].clone()
    L.ssu_delta_decode(T["q"], T["k"], v, T["a"], T["b"], T["state"], v, A_log=T["A_log"],
                       dt_bias=T["dt_bias"], state_indices=T["idx"])
    assert_bitwise(v, want, "out")


def test_agrees_with_the_fused_step():
    """The same layer's single token through ssu_gdn_decode with a convolution that passes its
    input through, and through ssu_delta_decode."""
    from linear_rnn_recurrent_amd import inputs
    w = inputs.gdn_workload(batch=4, hidden=64, num_q_heads=2, num_v_heads=4, head_dim=64, conv_width=4,
                            pool_rows=6, seed=5)
    G = {k: v.cuda() for k, v in w.tensors.items()}
    state = G["ssm_state"].clone()
    conv = G["conv_state"].clone()
    want = L.ssu_gdn_decode(G["hidden_states"], G["w_ba"], G["mixed_qkv"], G["conv_weight"], G["conv_bias"],
                            G["conv_state"], G["A_log"], G["dt_bias"], None, G["ssm_state"], G["state_indices"],
                            num_q_heads=2)
    y = torch.empty_like(G["mixed_qkv"], dtype=torch.float32)
    L.ssu_conv_decode(G["mixed_qkv"].float(), G["conv_weight"], G["conv_bias"], conv, y, state_indices=G["state_indices"])
    ba = G["hidden_states"].float() @ G["w_ba"].float()
    q, k, v = y[:, :128].unflatten(1, (2, 64)), y[:, 128:256].unflatten(1, (2, 64)), y[:, 256:].unflatten(1, (4, 64))
    out = torch.empty(4, 4, 64, device="cuda")
    L.ssu_delta_decode(q, k, v, ba[:, 4:], ba[:, :4], state, out, A_log=G["A_log"], dt_bias=G["dt_bias"],
                       state_indices=G["state_indices"])
    torch.cuda.synchronize()
    assert (out - want[:, 0].float()).abs().max() <= 2.0 ** -7 * (1 + want.float().abs().max())
    assert norm_error(state, f64(G["ssm_state"])) <= 1e-4


@pytest.mark.parametrize("seq_len", [5, 150])
def test_capture_and_streams(seq_len):
    """Captured on a stream of its own and replayed with eager work between, each replay against
    the eager call."""
    T = delta_inputs(21, batch=3, seq_len=seq_len, d=128, ctx=[seq_len, seq_len // 2, seq_len])
    start = T["state"].clone()
    want = call(T)
    after = T["state"].clone()
    y = torch.empty_like(want)
    need = L.delta_workspace_bytes(3, seq_len, 2, 4, 128)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    go = lambda **kw: L.ssu_delta_prefill(T["q"], T["k"], T["v"], T["a"], T["b"], T["state"], y, A_log=T["A_log"],  # noqa: E731
                                          dt_bias=T["dt_bias"], context_lengths=T["ctx"], state_indices=T["idx"],
                                          workspace=ws, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    T["state"].copy_(start)
    torch.cuda.synchronize()
    go(stream=side)
    side.synchronize()
    assert_bitwise(y, want, "side stream")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        go()
    for _ in range(3):
        T["state"].copy_(start)
        y.fill_(7.0)
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert_bitwise(y, want, "replay")
        assert_bitwise(T["state"], after, "replayed state")


def test_empty_calls():
    for batch, seq_len in ((0, 5), (2, 0), (0, 0)):
        T = delta_inputs(22, batch=batch, seq_len=seq_len, d=64)
        before = T["state"].clone()
        call(T)
        assert_bitwise(T["state"], before, "state")


def test_far_pool_rows():
    """A pool row whose offset passes 2^32 bytes and 2^31 elements."""
    hv, d = 8, 128
    row = hv * d * d
    pool = torch.empty((1 << 31) // row + 2, hv, d, d, dtype=torch.bfloat16, device="cuda")
    T = delta_inputs(23, batch=1, seq_len=130, hq=2, hv=hv, d=d, st="bf16")
    last = pool.shape[0] - 1
    pool[last] = T["state"][0]
    small = {**T, "state": T["state"][:1].clone(), "idx": torch.zeros(1, dtype=torch.int32, device="cuda")}
    want = call(small)
    T["state"], T["idx"] = pool, torch.tensor([last], dtype=torch.int32, device="cuda")
    assert_bitwise(call(T), want, "out")
    assert_bitwise(pool[last], small["state"][0], "state")
