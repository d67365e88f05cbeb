"""fp64 oracle of the gated delta rule on given q, k and v, the RMS norm and the
tokens' log probabilities: plain numpy from the definitions in include/ssu.h.

TEST INFRASTRUCTURE ONLY. Arrays are float64 (int32 for index arrays); pools
are updated in place.
"""
import numpy as np

EPS = 1e-6
U = 2.0 ** -24


def _silu(v):
    return v / (1.0 + np.exp(-v))


def _lengths(batch, seq_len, ctx, idx):
    out = []
    for b in range(batch):
        n = seq_len if ctx is None else int(min(max(int(ctx[b]), 0), seq_len))
        out.append(0 if idx is not None and idx[b] < 0 else n)
    return out


def gated_delta(q, k, v, a, b, state, *, A_log=None, dt_bias=None, scale=None, l2=True, ctx=None,
                idx=None, update=True):
    """q, k [b,t,hq,d], v [b,t,hv,d], a, b [b,t,hv], state [rows,hv,d,d] -> (out, its error
    bound, the state's error bound per value row [rows,hv,d]).

    The bound counts roundings. A step from a state row of norm |S| off by e (2-norm) with
    |k| <= 1 and 0 <= beta <= 1 leaves e no larger (I - beta k k^T shrinks), decays it by
    alpha, and adds its own: products of d terms and their sums, the norms of q and k, exp,
    softplus and sigmoid and their arguments (d + 48 roundings of the row and of u), the same
    again where a chunk of 64 tokens is summed in another order from operands in three parts, whose
    products leave out what is below 24 bits (4 roundings each of the three products).
    """
    nb, t, hv, d = v.shape
    hq = k.shape[2]
    heads = np.arange(hv) // (hv // hq)
    sc = d ** -0.5 if scale is None or not scale > 0 else scale
    out, bound = np.zeros(v.shape), np.zeros(v.shape)
    sbound = np.zeros(state.shape[:3])
    c = (2 * d + 64 + 48 + 12) * U
    for i, n in enumerate(_lengths(nb, t, ctx, idx)):
        if n == 0:
            continue
        row = i if idx is None else int(idx[i])
        S = state[row].copy()
        e = np.zeros((hv, d))
        for s in range(n):
            if A_log is not None:
                bias = 0.0 if dt_bias is None else dt_bias
                g = -np.exp(A_log) * np.logaddexp(0.0, a[i, s] + bias)
                beta = 1.0 / (1.0 + np.exp(-b[i, s]))
            else:
                g, beta = a[i, s], b[i, s]
            alpha = np.exp(g)
            ks = k[i, s][heads]
            if l2:
                ks = ks / np.sqrt((ks ** 2).sum(-1, keepdims=True) + EPS)
            old = np.sqrt((S ** 2).sum(-1)) * alpha[:, None]
            S = S * alpha[:, None, None]
            u = beta[:, None] * (v[i, s] - np.einsum("hvk,hk->hv", S, ks))
            S = S + u[..., None] * ks[:, None]
            e = (e * alpha[:, None]
                 + c * (old * (1 + np.abs(g))[:, None] + np.abs(u) + np.abs(beta[:, None] * v[i, s])))
            if q is not None:
                qs = q[i, s][heads]
                if l2:
                    qs = qs / np.sqrt((qs ** 2).sum(-1, keepdims=True) + EPS)
                norm = np.sqrt((qs ** 2).sum(-1, keepdims=True)) * sc
                out[i, s] = np.einsum("hvk,hk->hv", S, qs) * sc
                bound[i, s] = norm * (e + c * np.sqrt((S ** 2).sum(-1)))
        if update:
            state[row] = S
            sbound[row] = e
    return out, bound, sbound


def rms_norm(x, weight, *, residual=None, z=None, group=None, eps=EPS, unit=False,
             gate_first=False):
    """x [.., n] -> (y before its rounding, the residual's sum or None)."""
    h = x if residual is None else x + residual
    left = None if residual is None else h
    n = x.shape[-1]
    g = n if group is None else group
    if z is not None and gate_first:
        h = h * _silu(z)
    p = h.reshape(h.shape[:-1] + (n // g, g))
    y = p / np.sqrt((p ** 2).mean(-1, keepdims=True) + eps)
    w = np.broadcast_to(weight if weight.shape[0] == n else np.tile(weight, n // g), (n,))
    y = y.reshape(h.shape) * (w + 1.0 if unit else w)
    if z is not None and not gate_first:
        y = y * _silu(z)
    return y, left


def token_logprobs(logits, tokens, top, *, ctx=None, idx=None):
    """logits [b,t,v], tokens [b,t] -> (logprobs, entropy, ids, top logprobs)."""
    nb, t, v = logits.shape
    lp, ent = np.zeros((nb, t)), np.zeros((nb, t))
    ids, best = np.full((nb, t, top), -1, np.int64), np.zeros((nb, t, top))
    for i, n in enumerate(_lengths(nb, t, ctx, idx)):
        for s in range(n):
            x, tok = logits[i, s], int(tokens[i, s])
            order = np.argsort(-x, kind="stable")[:top]
            inside = 0 <= tok < v
            if np.isnan(x).any() or (x == np.inf).any():
                lp[i, s] = np.nan if inside else -np.inf
                ent[i, s] = np.nan
                ids[i, s], best[i, s] = -2, np.nan  # not said
                continue
            m = x.max()
            if m == -np.inf:
                lp[i, s], best[i, s], ids[i, s] = -np.inf, -np.inf, order
                continue
            with np.errstate(divide="ignore"):
                e = np.exp(x - m)
            log_s = np.log(e.sum())  # x - m first: m may be larger than fp64 resolves log s beside
            p = e / e.sum()
            keep = p > 0
            ent[i, s] = -(p[keep] * (x[keep] - m - log_s)).sum()
            lp[i, s] = x[tok] - m - log_s if inside else -np.inf
            ids[i, s], best[i, s] = order, x[order] - m - log_s
    return lp, ent, ids, best
