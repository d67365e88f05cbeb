"""Gated delta rule: values at which a prompt in chunks could lose digits or leave a range that the
token-by-token recurrence keeps. Against the fp64 oracle."""
import numpy as np
import pytest
import torch

from sequence_helpers import DT, U, check, f64
from serving_helpers import delta_inputs, norm_error
from test_gpu_delta import call

pytestmark = pytest.mark.gpu


def lost(d):
    """What the end of fp32's range costs a step. The matrix cores take parts below 2^-126 as 0, so an
    entry of the state or of u, whose parts go down to 2^-17 of it, is off by less than 2 x 2^-126 in each
    of the products with k, q, L and P (of at most 1, d + 64 of them)."""
    return 4 * (d + 64) * 2.0 ** -126


def reference(T, *, l2=True):
    """(out, its bound, state, its bound) of given decays and betas, for every beta and length of k.

    With S' = alpha S + u k^T, u = beta (v - alpha S k), |.| the 2-norm of a value row: an error e of S
    becomes alpha e max(1, |1 - beta k.k|), and a step adds roundings of alpha S (and of alpha's
    argument), of u, whose terms are beta v and beta alpha S k, times |k|, and of the sum. Each counts
    as often as in the oracle's own bound, which holds for 0 <= beta <= 1 and |k| <= 1.
    """
    A = {n: f64(t) for n, t in T.items()}
    q, k, v, a, b, S = (A[n] for n in ("q", "k", "v", "a", "b", "state"))
    S = S.copy()
    nb, t, hv, d = v.shape
    heads = np.arange(hv) // (hv // k.shape[2])
    c = (2 * d + 64 + 48 + 12) * U
    out, bound, sbound = np.zeros(v.shape), np.zeros(v.shape), np.zeros(S.shape)
    row_norm = lambda x: np.sqrt((x ** 2).sum(-1))  # noqa: E731
    for i in range(nb):
        r = int(A["idx"][i])
        e = np.zeros((hv, d))
        for s in range(t):
            ks, qs = k[i, s][heads], q[i, s][heads]
            if l2:
                ks, qs = (x / np.sqrt((x ** 2).sum(-1, keepdims=True) + 1e-6) for x in (ks, qs))
            qs = qs * d ** -0.5
            g = np.maximum(a[i, s], -1e300)
            alpha, beta, kn = np.exp(g)[:, None], b[i, s][:, None], row_norm(ks)[:, None]
            size = np.where(alpha > 0, 1 + np.abs(g)[:, None], 0.0)
            old = row_norm(S[r]) * alpha
            S[r] *= alpha[..., None]
            u = beta * (v[i, s] - np.einsum("hvk,hk->hv", S[r], ks))
            S[r] += u[..., None] * ks[:, None]
            e = (e * alpha * np.maximum(1, np.abs(1 - beta * kn ** 2))
                 + c * (old * size * (1 + np.abs(beta) * kn ** 2) + kn * (np.abs(u) + np.abs(beta * v[i, s])))
                 + lost(d))
            out[i, s] = np.einsum("hvk,hk->hv", S[r], qs)
            bound[i, s] = row_norm(qs)[:, None] * (e + c * row_norm(S[r])) + lost(d)
        sbound[r] = e[..., None]
    return out, bound, S, sbound


def near(got, ref, n, d, what, io=torch.float32):
    """The difference's 2-norm over the reference's. Roundings of either sign leave the root of their
    number: of an entry, three a step and step after step (sqrt(9 n)), and of the sums of products and
    functions of the last one (sqrt(d + 64)); a dot product with q has the ratio that its entries have.
    Beside it what lies below fp32's range (lost) over the n steps, for every entry."""
    lim = (np.sqrt(d + 64) + 3 * np.sqrt(n)) * U + (torch.finfo(io).eps / 2 if io != torch.float32 else 0.0)
    err = norm_error(got, ref)
    lim += np.sqrt(ref.size) * n * lost(d) / max(np.linalg.norm(ref), 1e-300)
    assert err <= lim, (what, err, lim)


def given(seed, *, batch=1, seq_len, d=64, io="f32", l2=True, zero=False, **kw):
    T = delta_inputs(seed, batch=batch, seq_len=seq_len, d=d, io=io, raw=False, gate="f32", l2=l2, **kw)
    if zero:
        T["state"].zero_()
    return T


def verify(T, *, l2=True, span=slice(None)):
    """Every entry within its bound, and the outputs of `span` and the state by their own norms."""
    out, bound, state, sbound = reference(T, l2=l2)
    n, d, io = T["v"].shape[1], T["v"].shape[-1], T["v"].dtype
    y = call(T, l2=l2)
    check(y, out, bound, io, "out")
    check(T["state"], state, sbound, torch.float32, "state")
    near(y[:, span].float(), out[:, span], n, d, "out", io)
    rows = T["idx"].long().tolist()
    near(T["state"][rows], state[rows], n, d, "state")
    return y


@pytest.mark.parametrize("keys", ["equal", "positive"])
@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("beta,seq_len", [(-0.25, 18), (-0.25, 64), (-0.25, 130), (-0.5, 64), (-0.5, 130), (-1.0, 64),
                                          (-3.0, 18), (2.0, 130), (2.05, 64), (2.099, 130), (3.0, 64)])
def test_betas_outside_zero_to_one(beta, seq_len, io, keys):
    """No decay: a negative beta, or one above 2, grows what stands along a key with every token."""
    T = given(101, seq_len=seq_len, io=io)
    T["a"].zero_()
    T["b"].fill_(beta)
    T["k"] = T["k"][:, :1].repeat(1, seq_len, 1, 1) if keys == "equal" else T["k"].abs()
    T["v"][:, 1::2] = -T["v"][:, 1::2].abs()
    T["v"][:, ::2] = T["v"][:, ::2].abs()
    out, bound, state, sbound = reference(T)
    y = call(T)
    if io == "f16" and np.abs(out).max() > 6e4:
        keep = np.abs(out) < 6e4
        assert torch.isfinite(y.float()[torch.from_numpy(keep).cuda()]).all()
    else:
        check(y, out, bound, DT[io], "out")
    check(T["state"], state, sbound, torch.float32, "state")


@pytest.mark.parametrize("io,small", [("f32", 1e-36), ("bf16", 1e-36), ("f32", 1e-20), ("f16", 1e-6)])
@pytest.mark.parametrize("seq_len,turn", [(130, 64), (130, 70), (90, 32), (40, 20)])
def test_values_that_turn_ordinary(io, small, seq_len, turn):
    T = given(102, seq_len=seq_len, io=io, zero=True)
    v = T["v"].float()
    v[:, :turn] *= small
    v[:, turn:] *= 10
    T["v"] = v.to(DT[io])
    before = {n: t[:, :turn] if n in ("q", "k", "v", "a", "b") else t for n, t in T.items()}
    out = reference(before)[0]
    y = verify(T, span=slice(turn, None))
    if io == "f32":
        near(y[:, :turn], out, turn, 64, "out before")


def test_values_behind_a_long_silence():
    """A state that fades by e^-5.5 in 64 tokens without a value, then values of up to 20."""
    T = given(103, seq_len=1100, io="bf16")
    T["a"].fill_(-5.5 / 64)
    T["v"][:, :1024] = 0.0
    T["v"][:, 1024:] = (T["v"][:, 1024:].float() * 6).clamp(-20, 20).to(torch.bfloat16)
    verify(T, span=slice(1024, None))


@pytest.mark.parametrize("large", [1e4, 1e6, 1e8])
@pytest.mark.parametrize("seq_len,at", [(64, 50), (150, 100), (40, 20)])
@pytest.mark.parametrize("d", [32, 64, 128, 256])
def test_a_large_token_leaves_those_before_it(large, seq_len, at, d):
    T = given(104, seq_len=seq_len, d=d)
    T["v"][:, at] *= large
    verify(T, span=slice(0, at))


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_a_large_token_in_every_tile_under_strong_decays(io):
    """Outputs of the other tokens by their own norm: the decays leave nothing of the large ones."""
    T = given(105, seq_len=128, io=io)
    T["a"].fill_(-9.0)
    T["v"][:, ::16] *= 1e4
    out, bound, state, sbound = reference(T)
    y = call(T)
    check(y, out, bound, DT[io], "out")
    check(T["state"], state, sbound, torch.float32, "state")
    others = [t for t in range(128) if t % 16 > 3]
    near(y[:, others].float(), out[:, others], 16, 64, "out", DT[io])


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("seq_len", [64, 150])
@pytest.mark.parametrize("shift", [-10.0, -17.0, -25.0])
def test_small_betas(io, seq_len, shift):
    T = given(106, seq_len=seq_len, io=io, zero=True)
    T["b"] = torch.sigmoid(torch.logit(T["b"].double()) + shift).float()
    out, _, state, _ = reference(T)
    y = call(T)
    if io != "f16":  # below fp16's range
        near(y.float(), out, seq_len, 64, "out", DT[io])
    rows = T["idx"].long().tolist()
    near(T["state"][rows], state[rows], seq_len, 64, "state")


@pytest.mark.parametrize("io,size", [("f32", 1e-2), ("f32", 1e-5), ("f32", 1e-8), ("f32", 1e-18), ("bf16", 1e-5),
                                     ("bf16", 1e-8), ("f16", 1e-4), ("f32", 30.0), ("bf16", 30.0)])
@pytest.mark.parametrize("seq_len", [64, 150])
def test_short_and_long_keys_without_norm(io, size, seq_len):
    T = given(107, seq_len=seq_len, io=io, l2=False, zero=True)
    T["k"] = (T["k"].float() * size).to(DT[io])
    T["b"] /= max(1.0, size * size)
    out, _, state, _ = reference(T, l2=False)
    y = call(T, l2=False)
    if io != "f16":
        near(y.float(), out, seq_len, 64, "out", DT[io])
    rows = T["idx"].long().tolist()
    near(T["state"][rows], state[rows], seq_len, 64, "state")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("seq_len", [40, 72, 100])
@pytest.mark.parametrize("small", [1e-3, 1e-5, 1e-9])
def test_small_values_behind_a_reset(io, seq_len, small):
    """Nothing is left of the old state (a decay of 0 at the first token of a chunk)."""
    at = 64 if seq_len > 64 else 32
    T = given(108, seq_len=seq_len, io=io)
    T["a"][:, at] = float("-inf")
    T["v"][:, at:] = (T["v"][:, at:].float() * small).to(DT[io])
    verify(T, span=slice(at, None))


@pytest.mark.parametrize("size", [1e-25, 1e20])
def test_queries_of_any_size_without_norm(size):
    """Their squares leave fp32's range, their products with the state do not."""
    T = given(109, seq_len=70, l2=False)
    T["q"] *= size
    verify(T, l2=False)


@pytest.mark.parametrize("at", [3, 40, 69])
def test_an_overflow_reaches_no_earlier_token(at):
    """A value that leaves fp32's range with its token's beta, and one that is infinite."""
    for v, beta in ((3e38, 1.9), (float("inf"), 0.5)):
        T = given(110, seq_len=70)
        want = call({**T, "state": T["state"].clone()})
        T["v"][0, at, 1, 7], T["b"][0, at, 1] = v, beta
        y = call(T)
        assert torch.isfinite(y[0, :at]).all() and not torch.isfinite(y[0, at, 1, 7])
        near(y[0, :at], f64(want[0, :at]), 2 * 70, 64, "before")
        others = [c for c in range(64) if c != 7]
        assert torch.isfinite(y[0, at:, 1, others]).all()


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_a_query_that_is_not_finite_reaches_no_other_token(io, value):
    T = given(111, seq_len=70, io=io, l2=False)
    twin = {**T, "state": T["state"].clone()}
    want = call(twin, l2=False)
    T["q"] = T["q"].clone()
    T["q"][0, 33, 0, 5] = value
    y = call(T, l2=False)
    assert not torch.isfinite(y[0, 33, :2].float()).any() and torch.isfinite(y[0, 33, 2:].float()).all()
    others = [t for t in range(70) if t != 33]
    assert torch.equal(y[0, others], want[0, others]) and torch.equal(T["state"], twin["state"])
