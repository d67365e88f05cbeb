"""Log probabilities, entropy and alternatives against the fp64 oracle."""
import numpy as np
import pytest
import torch

import linear_rnn_recurrent_amd as L
from oracle import serving
from sequence_helpers import DT, U, f64, strided

pytestmark = pytest.mark.gpu


def run(logits, tokens, top=0, ctx=None, idx=None, entropy=True, **kw):
    lead = logits.shape[:-1]
    new = lambda *s, **k: torch.full(lead + s, -77, device="cuda", **k)  # noqa: E731
    lp, ent = new(dtype=torch.float32), new(dtype=torch.float32) if entropy else None
    ids = new(top, dtype=torch.int32) if top else None
    best = new(top, dtype=torch.float32) if top else None
    L.ssu_token_logprobs(logits, tokens, lp, entropy=ent, top_ids=ids, top_logprobs=best, context_lengths=ctx,
                         state_indices=idx, **kw)
    torch.cuda.synchronize()
    return lp, ent, ids, best


def close(got, ref, bound, what):
    g = f64(got)
    assert (np.isnan(g) == np.isnan(ref)).all(), what
    inf = np.isinf(ref)
    assert (g[inf] == ref[inf]).all(), what
    ok = ~np.isnan(ref) & ~inf
    err = np.abs(g[ok] - ref[ok])
    assert (err <= (bound[ok] if np.ndim(bound) else bound)).all(), (what, err.max())


def verify(logits, tokens, top=0, ctx=None, idx=None, **kw):
    two = logits.dim() == 2
    x, tok = f64(logits), f64(tokens)
    if two:
        x, tok = x[:, None], tok[:, None]
    with np.errstate(invalid="ignore"):
        lp, ent, ids, best = serving.token_logprobs(x, tok, max(top, 1), ctx=None if ctx is None else f64(ctx),
                                                    idx=None if idx is None else f64(idx))
    g = run(logits, tokens, top, ctx, idx, **kw)
    lead = logits.shape[:-1]
    # a term's exp: its argument x - m (one rounding, |x - m| <= R where it counts: e^-R V < u) and
    # itself, 4 + R u; a lane's sum rescaled and joined adds at most V / 1024 + 32 roundings of
    # positive terms, log's argument is off by that much and its value by 2; x - m and its
    # difference from log s round once each
    v = logits.shape[-1]
    R = np.log(v) + 24 * np.log(2)
    rel = (v / 256 + 40 + R) * U
    size = lambda r: rel + 4 * U * (np.abs(np.where(np.isfinite(r), r, 0.0)) + np.log(v))  # noqa: E731
    close(g[0], lp.reshape(lead), size(lp.reshape(lead)), "logprobs")
    if g[1] is not None:  # sum of p (x - m): its terms' sizes add up to at most log s + entropy
        close(g[1], ent.reshape(lead), 2 * rel * (1 + 2 * np.log(v)), "entropy")
    if top:
        want = ids.reshape(lead + (top,))
        got = f64(g[2])
        said = want != -2
        assert (got[said] == want[said]).all()
        assert ((got[~said] >= -1) & (got[~said] < v)).all()
        ref = best.reshape(lead + (top,))
        bad = np.isnan(ref)
        close(g[3][torch.from_numpy(~bad).cuda()], ref[~bad], size(ref[~bad]), "top")
        assert np.isnan(f64(g[3])[bad]).all()
    return g


def logits_of(seed, *shape, io="f32", std=3.0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(*shape, generator=g) * std).to(DT[io]).cuda()
    tok = torch.randint(0, shape[-1], shape[:-1], generator=g).int().cuda()
    return x, tok


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,vocab", [(1, 1), (3, 2), (2, 63), (5, 1000), (1, 4096), (2, 4097), (3, 32000), (2, 70001),
                                        (1, 262147), (700, 1031), (2050, 513)])
def test_sizes(io, rows, vocab):
    x, tok = logits_of(1, rows, vocab, io=io)
    verify(x, tok, min(vocab, 5))


@pytest.mark.parametrize("top", [1, 2, 17, 32])
@pytest.mark.parametrize("io,std", [("f32", 3.0), ("bf16", 0.01), ("bf16", 8.0), ("f16", 1.0)])
@pytest.mark.parametrize("rows,vocab", [(2, 40000), (1100, 3000)])
def test_alternatives(top, io, std, rows, vocab):
    """Among them types with many equal logits."""
    verify(*logits_of(2, rows, vocab, io=io, std=std), top)


@pytest.mark.parametrize("order", ["up", "down", "equal", "last", "zeros"])
@pytest.mark.parametrize("rows", [1, 1500])
def test_ordered_and_equal_logits(order, rows):
    v = 6000
    x = torch.arange(v, device="cuda", dtype=torch.float32) / 700
    x = {"up": x, "down": x.flip(0), "equal": torch.full_like(x, 2.5), "last": torch.where(x < x[-1], -5.0, 3.0),
         "zeros": torch.where(torch.arange(v, device="cuda") % 2 == 0, 0.0, -0.0)}[order]
    verify(x.repeat(rows, 1).contiguous(), torch.full((rows,), v - 1, dtype=torch.int32, device="cuda"), 32)


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,vocab", [(8, 9000), (1030, 1500)])
def test_masked_logits(io, rows, vocab):
    """Rows of which a mask (of -inf, or of the type's lowest value) leaves some, one, or none."""
    x, tok = logits_of(3, rows, vocab, io=io)
    low = torch.finfo(x.dtype).min
    x[0] = float("-inf")
    x[1] = low
    x[2, :] = float("-inf")
    x[2, vocab - 3] = 1.0
    x[3, 100:] = low
    x[4, 1:] = float("-inf")
    x[5, ::2] = float("-inf")
    x[6] = float("-inf")
    x[6, 7:15] = low
    verify(x, tok, 9)


def test_rows_with_nan_and_infinities():
    x, tok = logits_of(4, 6, 20000)
    x[1, 77] = float("nan")
    x[2, 19999] = float("inf")
    x[3] = float("nan")
    x[4, 0] = -float("nan")
    verify(x, tok, 4)
    tok[1], tok[2] = -1, 20000
    verify(x, tok, 4)


def test_large_logits():
    x, tok = logits_of(5, 4, 5000)
    x[0] += 1e4
    x[1] *= 1e6
    x[2] -= 3e4
    x[3] *= 1e37
    g = run(x, tok, 3)
    ref = serving.token_logprobs(f64(x)[:, None], f64(tok)[:, None], 3)
    for a, b in ((g[0], ref[0][:, 0]), (g[3], ref[3][:, 0])):
        assert (np.abs(f64(a) - b) <= 1e-4 + 4 * U * np.abs(b)).all()
    assert (f64(g[2]) == ref[2][:, 0]).all() and (np.abs(f64(g[1]) - ref[1][:, 0]) <= 1e-4).all()


def test_tokens_outside_the_vocabulary():
    x, tok = logits_of(6, 5, 800)
    tok[:] = torch.tensor([-1, 800, 799, 0, 1 << 30], dtype=torch.int32)
    g = verify(x, tok, 2)
    assert torch.isinf(g[0][[0, 1, 4]]).all()


@pytest.mark.parametrize("vocab", [900, 50000])
def test_padded_batches(vocab):
    """Lengths from none to past the end, a padding row, NaN in what is not read."""
    x, tok = logits_of(7, 5, 4, vocab, io="bf16")
    ctx = torch.tensor([4, 0, 2, 9, -3], dtype=torch.int32).cuda()
    idx = torch.tensor([0, 1, 2, -1, 4], dtype=torch.int32).cuda()
    for b, n in enumerate([4, 0, 2, 0, 0]):
        x[b, n:] = float("nan")
    g = verify(x, tok, 3, ctx=ctx, idx=idx)
    assert (g[0][1] == 0).all() and (g[1][3] == 0).all() and (g[2][4] == -1).all() and (g[3][2, 2:] == 0).all()


@pytest.mark.parametrize("wide", [8, 3])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [(4,), (2, 3), (1200,)])
def test_slices_of_wider_tensors(wide, io, rows):
    x, tok = logits_of(8, *rows, 2001, io=io)
    verify(strided(x, wide, len(rows)), tok, 4)
    if len(rows) == 2:
        verify(x.transpose(0, 1).contiguous().transpose(0, 1), tok, 4)


def test_optional_outputs():
    x, tok = logits_of(9, 3, 30000)
    want = run(x, tok, 4)
    assert torch.equal(run(x, tok, 0, entropy=False)[0], want[0])
    assert torch.equal(run(x, tok, 4, entropy=False)[2], want[2])


@pytest.mark.parametrize("rows,vocab", [(1, 100000), (64, 32000), (1100, 2000)])
def test_capture_and_streams(rows, vocab):
    x, tok = logits_of(10, rows, vocab)
    want = run(x, tok, 6)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [torch.empty_like(t) for t in want]
    ws = torch.empty(max(16, L.logprobs_workspace_bytes(1, rows, vocab, 6)), dtype=torch.uint8, device="cuda")
    go = lambda **kw: L.ssu_token_logprobs(x, tok, outs[0], entropy=outs[1], top_ids=outs[2], top_logprobs=outs[3], **kw)  # noqa: E731
    torch.cuda.synchronize()
    go(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        go(workspace=ws)
    for _ in range(3):
        for t in outs:
            t.zero_()
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_empty():
    run(torch.empty(0, 500, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda"), 3)
    run(torch.empty(3, 0, 500, device="cuda"), torch.empty(3, 0, dtype=torch.int32, device="cuda"), 3)
