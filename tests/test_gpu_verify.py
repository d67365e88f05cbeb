"""Draft verification against the fp64 oracle: every result is an integer and
has to be equal. A draw differs only if u times the total falls within the
rounding of an fp64 sum (about 1e-15 relative) of a step of the distribution
function; the seeds below are fixed, and none does."""
import numpy as np
import pytest
import torch

import oracle
from linear_rnn_recurrent_amd import (inputs, ssu_draft_verify, ssu_prefill, ssu_replay,
                                      ssu_tree_verify, verify_workspace_bytes)
from gpu_helpers import assert_bitwise, gpu
from sequence_helpers import f64, verify_inputs

pytestmark = pytest.mark.gpu


def call(T, most=None, path=True, workspace=None, stream=None):
    b, t = T["tokens"].shape
    acc = torch.full((b,), -77, dtype=torch.int32, device="cuda")
    nxt = torch.full((b,), -77, dtype=torch.int32, device="cuda")
    ids = torch.full((b, most or t), -77, dtype=torch.int32, device="cuda") if path else None
    ssu_draft_verify(T["tokens"], T["target"], T["uniforms"], acc, nxt, draft_probs=T["draft"],
                     parent_ids=T["parents"], context_lengths=T["ctx"], state_indices=T["idx"],
                     accepted_node_ids=ids, workspace=workspace, stream=stream)
    return acc, nxt, ids


def run_both(T, most=None, path=True):
    acc, nxt, ids = call(T, most, path)
    torch.cuda.synchronize()
    want = oracle.draft_verify(f64(T["tokens"]), f64(T["target"]), f64(T["uniforms"]),
                               draft=f64(T["draft"]), parents=f64(T["parents"]), ctx=f64(T["ctx"]),
                               idx=f64(T["idx"]), max_accept=most)
    np.testing.assert_array_equal(f64(acc), want[0], "accepted")
    np.testing.assert_array_equal(f64(nxt), want[1], "next")
    if path:
        np.testing.assert_array_equal(f64(ids), want[2], "path")
    return want


@pytest.mark.parametrize("probs", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("kind", ["draft", "given", "tree"])
@pytest.mark.parametrize("vocab", [1, 2, 7, 300, 2047, 2048, 2049, 5000, 32000])
def test_types_kinds_and_vocabularies(probs, kind, vocab):
    want = run_both(verify_inputs(vocab, batch=7, tokens=6, vocab=vocab, probs=probs,
                                  tree=kind == "tree", draft=kind == "draft"))
    if vocab == 5000 and probs == "f32":
        assert len(set(want[0].tolist())) > 1  # not all rows stop at the same place


@pytest.mark.parametrize("tokens", [1, 2, 3, 63, 64, 65, 66, 127, 128])
@pytest.mark.parametrize("kind", ["draft", "given", "tree"])
def test_numbers_of_tokens(tokens, kind):
    run_both(verify_inputs(tokens, batch=5, tokens=tokens, vocab=600, tree=kind == "tree",
                           draft=kind == "draft", sharp=8.0))


@pytest.mark.parametrize("kind", ["draft", "given"])
def test_long_chains_are_accepted_past_a_wave(kind):
    """Drafts equal to the target: with q = p every token stands (u q < p), so
    the lengths are the context lengths, over 64 tokens among them."""
    T = verify_inputs(3, batch=6, tokens=128, vocab=40, draft=True, ctx=[128, 64, 65, 66, 1, 100])
    if kind == "draft":
        T["draft"] = T["target"][:, :-1].contiguous()
        T["tokens"][:, 1:] = T["target"][:, :-1].argmax(-1).int()
        want = run_both(T)
        assert want[0].tolist() == [128, 64, 65, 66, 1, 100]
    else:
        T["draft"] = None
        T["target"] = torch.zeros_like(T["target"])
        T["target"].scatter_(2, T["tokens"].roll(-1, 1).long()[..., None], 1.0)
        want = run_both(T)
        assert want[0].tolist() == [128, 64, 65, 66, 1, 100]


def test_lengths_and_padding_rows():
    for kind in ("draft", "tree"):
        T = verify_inputs(5, batch=8, tokens=9, vocab=3000, tree=kind == "tree",
                          draft=kind == "draft", ctx=[9, 0, -3, 1, 2, 50, 5, 9],
                          idx=[3, 1, 2, 0, -1, 4, 9, 8])
        for b, n in enumerate([9, 0, 0, 1, 0, 9, 5, 9]):
            T["target"][b, n:] = float("nan")  # never read
            T["uniforms"][b, max(n, 1):] = float("nan")
            T["tokens"][b, n:] = 1 << 30
            if T["draft"] is not None:
                T["draft"][b, max(n - 1, 0):] = float("nan")
            else:
                T["parents"][b, n:] = 0
        run_both(T)


@pytest.mark.parametrize("most", [1, 2, 3, 9, 20])
@pytest.mark.parametrize("kind", ["draft", "given", "tree"])
def test_bounded_paths(most, kind):
    run_both(verify_inputs(17, batch=9, tokens=9, vocab=50, tree=kind == "tree",
                           draft=kind == "draft", sharp=9.0), most=most)


def test_without_a_path():
    run_both(verify_inputs(18, batch=4, tokens=5, vocab=100), path=False)


@pytest.mark.parametrize("wide", [1, 8, 64])
def test_strides(wide):
    run_both(verify_inputs(19, batch=3, tokens=4, vocab=2500, probs="bf16", wide=wide))
    run_both(verify_inputs(20, batch=3, tokens=8, vocab=2500, probs="f32", tree=True, wide=wide))


def test_trees_with_bad_parents_repeated_and_foreign_tokens():
    T = verify_inputs(21, batch=6, tokens=24, vocab=500, tree=True)
    T["parents"][0, 5:] = -1
    T["parents"][1, 3] = 3
    T["parents"][1, 4] = 20
    T["tokens"][2, 1:] = T["tokens"][2, 1]   # one token over and over
    T["parents"][2, 1:] = 0
    T["tokens"][3, 2:9] = -5
    T["tokens"][4, 2:9] = 500
    T["parents"][5, 1:] = 0                  # a star: every rejected child is taken out
    run_both(T)


def test_star_with_all_mass_on_the_children():
    """Children that hold all of the distribution: the last one stands whatever
    its number says, since nothing else is left."""
    T = verify_inputs(22, batch=2, tokens=5, vocab=64, tree=True)
    T["parents"][:, 1:] = 0
    T["target"][:] = 0.0
    for k in range(1, 5):
        T["tokens"][:, k] = 7 * k
        T["target"][:, 0, 7 * k] = 0.25
    T["target"][:, 1:, 3] = 1.0
    T["uniforms"][:, 1:] = 0.9990234375
    want = run_both(T)
    assert want[0].tolist() == [2, 2] and want[2][:, 1].tolist() == [4, 4]


def test_residual_without_mass_and_rows_without_mass():
    T = verify_inputs(23, batch=4, tokens=3, vocab=4100)
    T["draft"] = (T["target"][:, :-1] * 2).contiguous()  # q above p everywhere: no residual
    T["uniforms"][:, 1:] = 0.75                          # u q = 1.5 p: rejected
    T["target"][1] = 0.0
    T["target"][2] = float("nan")
    T["target"][3] = -1.0
    want = run_both(T)
    assert want[0].tolist() == [1, 1, 1, 1]
    assert want[1][0] >= 0 and want[1][1:].tolist() == [-1, -1, -1]


def test_large_vocabularies_take_two_launches():
    """Over 65536 entries: the sums in a launch of their own; residuals without
    mass, rows without mass, bounded paths and padding there too."""
    for probs, wide in (("f32", 0), ("bf16", 3)):
        T = verify_inputs(33, batch=6, tokens=4, vocab=70001, probs=probs, wide=wide,
                          ctx=[4, 0, 4, 4, 4, 1], idx=[0, 1, -1, 2, 3, 4])
        T["draft"][3] = T["target"][3, :-1] * 2
        T["uniforms"][3, 1:] = 0.75
        T["target"][4] = 0.0
        run_both(T)
        run_both(T, most=2)
    T = verify_inputs(34, batch=3, tokens=20, vocab=66000, tree=True)
    T["parents"][1, 1:] = 0
    run_both(T)
    run_both(T, most=2)
    run_both(verify_inputs(35, batch=2, tokens=100, vocab=65537, draft=False, sharp=9.0))


def test_large_vocabulary_in_a_graph():
    T = verify_inputs(36, batch=4, tokens=5, vocab=90000)
    want = run_both(T)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        acc, nxt, ids = call(T)
    for rep in range(3):
        acc.fill_(9), nxt.fill_(9), ids.fill_(9)
        g.replay()
        torch.cuda.synchronize()
        for got, ref in zip((acc, nxt, ids), want):
            np.testing.assert_array_equal(f64(got), ref)


def test_numbers_at_the_ends():
    """u = 0 draws the first entry with mass, u just below 1 the last with any."""
    T = verify_inputs(24, batch=4, tokens=1, vocab=9000, draft=False)
    T["target"][:, :, :100] = 0.0
    T["target"][:, :, 8000:] = 0.0
    T["target"][2:, :, :] = 0.0
    T["target"][2:, :, 4321] = 0.25
    T["uniforms"][:, 0] = torch.tensor([0.0, 1 - 2.0 ** -24, 0.0, 1 - 2.0 ** -24])
    want = run_both(T)
    assert want[1].tolist()[0] == 100 and want[1].tolist()[2:] == [4321, 4321]


def test_large_vocabularies_and_offsets_past_32_bits():
    run_both(verify_inputs(25, batch=3, tokens=2, vocab=300001, probs="bf16"))
    # 17 rows of 2^27 bf16 entries apart: offsets past 2^31
    vocab, tokens = 1000, 18
    T = verify_inputs(26, batch=1, tokens=tokens, vocab=vocab, probs="bf16", draft=False, sharp=9.0)
    far = torch.zeros(1, tokens, 1 << 27, dtype=torch.bfloat16, device="cuda")[..., :vocab]
    far.copy_(T["target"])
    T["tokens"][0, 1:] = T["target"][0, :-1].argmax(-1).int()
    T["uniforms"][:, 1:] = 0.0
    T["target"] = far
    want = run_both(T)
    assert want[0].tolist() == [tokens]


def test_the_drawn_tokens_follow_the_target():
    """Draft and target over 8 tokens: over 60,000 rows the first token after
    token 0 (the accepted draft or the drawn one) has the target's frequencies.
    The standard deviation of a frequency is at most sqrt(1/4/60000) = 0.00204;
    5 of them over 8 cells are 0.0102."""
    g = torch.Generator().manual_seed(27)
    n, v = 60000, 8
    p = torch.tensor([0.30, 0.02, 0.18, 0.05, 0.25, 0.00, 0.15, 0.05])
    q = torch.tensor([0.05, 0.20, 0.18, 0.15, 0.10, 0.22, 0.05, 0.05])
    T = {"target": p.expand(n, 2, v).contiguous().cuda(), "parents": None, "ctx": None, "idx": None,
         "uniforms": torch.rand(n, 2, generator=g).cuda(),
         "draft": q.expand(n, 1, v).contiguous().cuda(),
         "tokens": torch.cat([torch.zeros(n, 1), torch.multinomial(q, n, True, generator=g)[:, None]],
                             1).int().cuda()}
    tree = {**T, "draft": None, "tokens": torch.tensor([0, 4, 2, 0]).int().repeat(n, 1).cuda(),
            "parents": torch.tensor([-1, 0, 0, 0]).int().repeat(n, 1).cuda(),
            "target": p.expand(n, 4, v).contiguous().cuda(),
            "uniforms": torch.rand(n, 4, generator=g).cuda()}
    for case in (T, tree):
        acc, nxt, ids = call(case)
        tok = torch.where(acc > 1, case["tokens"].gather(1, ids[:, 1:2].clamp_min(0).long())[:, 0],
                          nxt)
        freq = torch.bincount(tok.long(), minlength=v).cpu().double() / n
        assert float((freq - p.double()).abs().max()) < 0.0102


def test_workspace_graph_and_other_stream():
    T = verify_inputs(28, batch=6, tokens=5, vocab=7000)
    want = run_both(T)
    ws = torch.full((verify_workspace_bytes(6, 7000),), 255, dtype=torch.uint8, device="cuda")
    b, t = T["tokens"].shape
    acc, nxt = (torch.zeros(b, dtype=torch.int32, device="cuda") for _ in range(2))

    def run(stream=None):
        ssu_draft_verify(T["tokens"], T["target"], T["uniforms"], acc, nxt, draft_probs=T["draft"],
                         workspace=ws, stream=stream)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for rep in range(3):
        acc.fill_(9), nxt.fill_(9), ws.fill_(rep)
        g.replay()
        torch.cuda.synchronize()
        np.testing.assert_array_equal(f64(acc), want[0])
        np.testing.assert_array_equal(f64(nxt), want[1])
    side = torch.cuda.Stream()
    acc.fill_(9)
    side.wait_stream(torch.cuda.current_stream())
    run(side)
    side.synchronize()
    np.testing.assert_array_equal(f64(acc), want[0])


def test_chain_window_verify_and_replay_without_the_host():
    """The heads' path: window with the stash, verification, replay of the
    accepted tokens, all on device results; the state is the one of a prefill of
    exactly the accepted tokens."""
    w = inputs.prefill_workload(batch=5, seq_len=6, nheads=4, dim=32, dstate=32, ngroups=1,
                                pool_rows=7, seed=29, ctx=("none",), io_dtype="f32",
                                bc_dtype="f32", bc_std=0.2)
    T = {k: gpu(v) for k, v in w.tensors.items()}
    b, t, h, d = T["x"].shape
    V = verify_inputs(30, batch=b, tokens=t, vocab=300, sharp=6.0)
    S = dict(replay_dA=torch.empty(b, t, h, device="cuda"), replay_dt=torch.empty(b, t, h, device="cuda"),
             replay_u=torch.empty(b, t, h, d, device="cuda"),
             replay_B=torch.empty(tuple(T["B"].shape), device="cuda"))
    ref = T["state"].clone()
    out = torch.empty_like(T["x"])
    kw = dict(dt_bias=T["dt_bias"], D=T["D"], z=T["z"], state_indices=T["state_indices"])
    ssu_prefill(T["x"], T["A"], T["B"], T["C"], T["dt"], T["state"], out, **kw, **S)
    acc, _, _ = call({**V, "idx": T["state_indices"]})
    ssu_replay(T["state"], S["replay_dA"], S["replay_u"], S["replay_B"], S["replay_dt"], acc,
               state_indices=T["state_indices"])
    ssu_prefill(T["x"], T["A"], T["B"], T["C"], T["dt"], ref, out, context_lengths=acc, **kw)
    torch.cuda.synchronize()
    assert acc.min() >= 1 and acc.max() > 1
    # replay and prefill run the same recurrence: t steps, three roundings each, either side
    diff = (T["state"] - ref).abs().max().item()
    assert diff <= 2 * 3 * t * 2.0 ** -24 * ref.abs().max().item()


def test_tree_verify_and_path_commit_without_the_host():
    w = inputs.tree_workload(batch=3, num_nodes=24, nheads=2, dim=32, dstate=32, ngroups=1,
                             pool_rows=5, seed=31, io_dtype="f32", bc_dtype="f32", bc_std=0.2)
    T = {k: gpu(v) for k, v in w.tensors.items()}
    b, m, h, d = T["x"].shape
    V = verify_inputs(32, batch=b, tokens=m, vocab=200, tree=True, sharp=6.0)
    T["parent_ids"] = V["parents"]
    S = dict(replay_dA=torch.empty(b, m, h, device="cuda"), replay_dt=torch.empty(b, m, h, device="cuda"),
             replay_u=torch.empty(b, m, h, d, device="cuda"),
             replay_B=torch.empty(tuple(T["B"].shape), device="cuda"))
    start = T["state"].clone()
    out = torch.empty_like(T["x"])
    ssu_tree_verify(T["x"], T["A"], T["B"], T["C"], T["dt"], T["state"], out, T["parent_ids"],
                    dt_bias=T["dt_bias"], D=T["D"], state_indices=T["state_indices"], **S)
    acc, nxt, ids = call({**V, "idx": T["state_indices"]}, most=8)
    ssu_replay(T["state"], S["replay_dA"], S["replay_u"], S["replay_B"], S["replay_dt"], acc,
               state_indices=T["state_indices"], accepted_node_ids=ids)
    torch.cuda.synchronize()
    assert acc.max() > 1
    for r in range(b):  # the path's tokens through a prefill of their own
        n = int(acc[r])
        path = ids[r, :n].long()
        row = T["state_indices"][r:r + 1]
        st = start.clone()
        pick = lambda k: T[k][r:r + 1, path].contiguous()  # noqa: E731
        ssu_prefill(pick("x"), T["A"], pick("B"), pick("C"), pick("dt"), st,
                    torch.empty_like(pick("x")), dt_bias=T["dt_bias"], D=T["D"], state_indices=row)
        got, want = T["state"][row.long()], st[row.long()]
        assert (got - want).abs().max().item() <= 2 * 3 * n * 2.0 ** -24 * want.abs().max().item()
    assert_bitwise(T["state"][[i for i in range(5) if i not in f64(T["state_indices"])]],
                   start[[i for i in range(5) if i not in f64(T["state_indices"])]], "other rows")
