"""The most rows of one call of the log probabilities: the size query, the call and the header agree."""
import pytest
import torch

import linear_rnn_recurrent_amd as L
from test_abi_serving import err, lib, logprob_dims, logprobs  # noqa: F401


@pytest.mark.parametrize("batch,tokens", [(1 << 25, 1), (1 << 12, 1 << 13), ((1 << 24) + 5, 1), (1, 1 << 24)])
def test_rows_that_the_query_admits(lib, batch, tokens):  # noqa: F811
    assert lib.ssu_logprobs_workspace_bytes(logprob_dims(batch=batch, num_tokens=tokens)) == 0


@pytest.mark.parametrize("batch,tokens", [((1 << 25) + 1, 1), ((1 << 13) + 1, 1 << 12), (1 << 30, 1 << 30)])
def test_rows_that_query_and_call_refuse(lib, batch, tokens):  # noqa: F811
    d = logprob_dims(batch=batch, num_tokens=tokens)
    assert lib.ssu_logprobs_workspace_bytes(d) == -1
    assert logprobs(lib, d) == 2 and "2^25" in err(lib)


@pytest.mark.gpu
@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
def test_more_rows_than_a_launch_has_workgroups(io):
    """2^24 rows of 256 threads each would be 2^32 of them. In fp64 against the formula: lse of three
    logits and its difference from one, 12 roundings of values up to |x| + log 3 beside 4 of exp and log."""
    rows, vocab = (1 << 24) + 5, 3
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(rows, vocab, generator=g, device="cuda").to(io)
    tok = torch.randint(0, vocab, (rows,), generator=g, device="cuda", dtype=torch.int32)
    lp, ent = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    ids, best = torch.empty(rows, 2, dtype=torch.int32, device="cuda"), torch.empty(rows, 2, device="cuda")
    L.ssu_token_logprobs(x, tok, lp, entropy=ent, top_ids=ids, top_logprobs=best)
    ref = x.double() - x.double().logsumexp(1, keepdim=True)
    lim = 16 * 2.0 ** -24 * (8 + 1.1)  # |x| < 8 of 5e7 normal values
    assert x.abs().max() < 8
    assert (lp - ref.gather(1, tok.long()[:, None])[:, 0]).abs().max() <= lim
    assert (ent + (ref.exp() * ref).sum(1)).abs().max() <= lim
    order = x.double().sort(dim=1, descending=True, stable=True).indices[:, :2]
    assert torch.equal(ids.long(), order)
    assert (best - ref.gather(1, order)).abs().max() <= lim
