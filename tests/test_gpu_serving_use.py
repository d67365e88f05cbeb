"""The gated delta rule, the norm and the log probabilities as a program uses them: states of a pool,
two streams at once, two graphs in turn over one workspace, and the calls that are refused."""
import pytest
import torch

import linear_rnn_recurrent_amd as L
from gpu_helpers import assert_bitwise
from linear_rnn_recurrent_amd import SsuError, SsuPool
from serving_helpers import delta_inputs

pytestmark = pytest.mark.gpu


def prefill(T, out, **kw):
    return L.ssu_delta_prefill(T["q"], T["k"], T["v"], T["a"], T["b"], kw.pop("state", T["state"]), out,
                               A_log=T["A_log"], dt_bias=T["dt_bias"], state_indices=kw.pop("idx", T["idx"]), **kw)


@pytest.mark.parametrize("seq_len", [4, 70])
def test_states_of_a_pool(seq_len):
    hv, d = 4, 64
    T = delta_inputs(41, batch=2, seq_len=seq_len, hv=hv, d=d)
    pool = SsuPool([(0, 0, (hv, d, d), torch.float32), (0, 1, (hv, d, d), torch.float32)], 5)
    idx = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    zero = torch.zeros(5, hv, d, d, device="cuda")
    want, got = torch.empty_like(T["v"]), torch.empty_like(T["v"])
    prefill(T, want, state=zero, idx=idx)
    prefill(T, got, state=pool.state(1), idx=idx)
    assert_bitwise(got, want, "out")
    for slot in range(5):
        first, second = pool.capture(slot)
        assert torch.count_nonzero(first) == 0
        assert_bitwise(second.view(torch.float32).reshape(-1), zero[slot].reshape(-1), f"slot {slot}")
    # a single token behind it
    S = {n: T[n][:, 0].contiguous() for n in ("q", "k", "v", "a", "b")}
    y = [torch.empty_like(S["v"]) for _ in range(2)]
    for out, state in zip(y, (zero, pool.state(1))):
        L.ssu_delta_decode(S["q"], S["k"], S["v"], S["a"], S["b"], state, out, A_log=T["A_log"],
                           dt_bias=T["dt_bias"], state_indices=idx)
    assert_bitwise(y[1], y[0], "step")


def test_two_streams_at_once():
    """Workspaces that the calls allocate belong to their streams."""
    sets = [delta_inputs(50 + i, batch=3, seq_len=200, d=128) for i in range(2)]
    g = torch.Generator().manual_seed(6)
    logits = [torch.randn(4, 60000, generator=g).cuda() for _ in range(2)]
    tokens = torch.arange(4, dtype=torch.int32).cuda()
    x = [torch.randn(64, 2048, generator=g).cuda().bfloat16() for _ in range(2)]
    w = torch.ones(2048).cuda()

    def all_of(i, stream=None):
        T = {**sets[i], "state": states[i]}
        y, lp = torch.empty_like(T["v"]), torch.empty(4, device="cuda")
        ids, best = torch.empty(4, 5, dtype=torch.int32, device="cuda"), torch.empty(4, 5, device="cuda")
        n = torch.empty_like(x[i])
        made = [y, lp, ids, best, n, states[i]]
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
            for t in made:
                t.record_stream(stream)
        for _ in range(3):
            prefill(T, y, stream=stream)
            L.ssu_token_logprobs(logits[i], tokens, lp, top_ids=ids, top_logprobs=best, stream=stream)
            L.ssu_rms_norm(x[i], w, n, stream=stream)
        return made

    states = [s["state"].clone() for s in sets]
    want = [all_of(i) for i in range(2)]
    states = [s["state"].clone() for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [all_of(i, streams[i]) for i in range(2)]
    torch.cuda.synchronize()
    for i in range(2):
        for a, b in zip(got[i], want[i]):
            assert torch.equal(a, b)


def test_two_graphs_over_one_workspace_in_turn():
    sets = [delta_inputs(60 + i, batch=2, seq_len=100 + 60 * i, d=64) for i in range(2)]
    need = max(L.delta_workspace_bytes(2, s["q"].shape[1], 2, 4, 64) for s in sets)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    starts = [s["state"].clone() for s in sets]
    want = [prefill(s, torch.empty_like(s["v"])) for s in sets]
    outs = [torch.empty_like(t) for t in want]
    graphs = []
    for s, y in zip(sets, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            prefill(s, y, workspace=ws)
    for order in ((0, 1), (1, 0), (0, 1)):
        for s, start in zip(sets, starts):
            s["state"].copy_(start)
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for y, t in zip(outs, want):
            assert_bitwise(y, t, "replay")
            y.zero_()


def test_delta_refusals():
    T = delta_inputs(70, batch=2, seq_len=40, d=64)
    y = torch.empty_like(T["v"])
    before = T["state"].clone()
    bad = [
        dict(q=T["q"].float()), dict(k=T["k"][:, :39]), dict(k=T["k"][..., :32]), dict(v=T["v"].cpu()),
        dict(a=T["a"][..., :3]), dict(b=T["b"].half()), dict(q=None), dict(out=None, update_state=False),
        dict(out=T["k"]), dict(out=T["v"]), dict(state=T["state"].transpose(2, 3)), dict(state=T["state"][:, :3]),
        dict(state_indices=T["idx"].long()), dict(state_indices=T["idx"][:1]), dict(A_log=T["A_log"].half()),
        dict(A_log=None), dict(context_lengths=T["idx"].float()),
        dict(workspace=torch.empty(64, dtype=torch.uint8, device="cuda")),
        dict(q=T["q"][:, :, :1].expand(-1, -1, 2, -1)), dict(out=y[:, :1].expand(-1, 40, -1, -1)),
        dict(q=T["q"][..., 1:], k=T["k"][..., 1:], v=T["v"][..., 1:], out=y[..., 1:], state=T["state"][..., 1:, 1:]),
        dict(q=T["q"].repeat(1, 1, 2, 1)[:, :, :3], k=T["k"].repeat(1, 1, 2, 1)[:, :, :3]),
    ]
    for kw in bad:
        full = {**{n: T[n] for n in ("q", "k", "v", "a", "b", "state", "A_log", "dt_bias")}, "out": y,
                "state_indices": T["idx"], **kw}
        args = [full.pop(n) for n in ("q", "k", "v", "a", "b", "state", "out")]
        with pytest.raises((ValueError, SsuError)):
            L.ssu_delta_prefill(*args, **full)
    torch.cuda.synchronize()
    assert_bitwise(T["state"], before, "state")


def test_norm_refusals():
    x = torch.randn(6, 256, device="cuda")
    w, y = torch.ones(256, device="cuda"), torch.empty(6, 256, device="cuda")
    code = torch.empty(6, 256, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty(6, 2, device="cuda")
    bad = [
        dict(x=x.cpu()), dict(x=x.double()), dict(x=x.t()), dict(x=x[0]), dict(weight=w[:100]), dict(weight=w.cpu()),
        dict(out=y[:5]), dict(out=code), dict(scales=s), dict(out=code, scales=s[:5]), dict(out=code, scales=s.half()),
        dict(out=code, scales=torch.empty(6, 3, device="cuda")), dict(group_size=100), dict(group_size=0),
        dict(residual=x), dict(residual=y), dict(residual=x[:, :128]), dict(z=x.half()), dict(eps=-1.0),
        dict(eps=float("nan")), dict(out=y[:1].expand(6, -1)),
        dict(out=code, scales=torch.empty(6, 64, device="cuda")),  # blocks of four
    ]
    for kw in bad:
        full = {"x": x, "weight": w, "out": y, **kw}
        with pytest.raises((ValueError, SsuError)):
            L.ssu_rms_norm(full.pop("x"), full.pop("weight"), full.pop("out"), **full)


def test_logprob_refusals():
    x = torch.randn(5, 300, device="cuda")
    tok, lp = torch.zeros(5, dtype=torch.int32, device="cuda"), torch.empty(5, device="cuda")
    ids = lambda k: torch.empty(5, k, dtype=torch.int32, device="cuda")  # noqa: E731
    top = lambda k: torch.empty(5, k, device="cuda")  # noqa: E731
    bad = [
        dict(logits=x.cpu()), dict(logits=x.double()), dict(logits=x.t()), dict(logits=x[:, ::2]), dict(logits=x[0]),
        dict(tokens=tok.long()), dict(tokens=tok[:4]), dict(logprobs=lp.half()), dict(entropy=lp[:4]),
        dict(top_ids=ids(3)), dict(top_logprobs=top(3)), dict(top_ids=ids(3), top_logprobs=top(4)),
        dict(top_ids=ids(33), top_logprobs=top(33)), dict(top_ids=ids(0), top_logprobs=top(0)),
        dict(context_lengths=tok[:2]), dict(state_indices=tok.long()),
        dict(workspace=torch.empty(8, dtype=torch.uint8)),
    ]
    for kw in bad:
        full = {"logits": x, "tokens": tok, "logprobs": lp, **kw}
        with pytest.raises((ValueError, SsuError)):
            L.ssu_token_logprobs(full.pop("logits"), full.pop("tokens"), full.pop("logprobs"), **full)
