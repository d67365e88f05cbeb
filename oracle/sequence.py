"""fp64 oracle of the causal convolution, the per-channel selective scan and
draft verification: plain numpy loops from the definitions in include/ssu.h.

TEST INFRASTRUCTURE ONLY. Arrays are float64 (int32 for index arrays); pools
are updated in place. Every function returns (out, magnitude) or what it says:
`magnitude` holds, for every output, the sum of the magnitudes of the terms it
is a sum of, the scale of the rounding of that sum in any order.
"""
import numpy as np


def _silu(v):
    return v / (1.0 + np.exp(-v))


def _lengths(batch, seq_len, ctx, idx):
    out = []
    for b in range(batch):
        n = seq_len if ctx is None else int(min(max(int(ctx[b]), 0), seq_len))
        out.append(0 if idx is not None and idx[b] < 0 else n)
    return out


def causal_conv(x, weight, bias, conv_state, *, silu=True, ctx=None, idx=None, update=True):
    """x [b,t,c], weight [c,W], conv_state [rows,c,W-1] -> (out, magnitude)."""
    nb, t, c = x.shape
    w = weight.shape[1]
    out, mag = np.zeros(x.shape), np.zeros(x.shape)
    for b, n in enumerate(_lengths(nb, t, ctx, idx)):
        if n == 0:
            continue
        row = b if idx is None else int(idx[b])
        win = np.concatenate([conv_state[row].T, x[b, :n]]) if w > 1 else x[b, :n]
        for k in range(n):
            acc = np.zeros(c) if bias is None else bias.copy()
            m = np.abs(acc)
            for j in range(w):
                acc = acc + weight[:, j] * win[k + j]
                m = m + np.abs(weight[:, j] * win[k + j])
            out[b, k] = _silu(acc) if silu else acc
            mag[b, k] = m
        if update and w > 1:
            conv_state[row] = win[n:n + w - 1].T
    return out, mag


def channel_scan(x, A, B, C, dt, state, *, dt_bias=None, D=None, z=None, softplus=True, ctx=None,
                 idx=None, update=True):
    """x, z, dt [b,t,d], A [d,n], B, C [b,t,g,n], state [rows,d,n] ->
    (out, magnitude, state magnitude [rows,d,n] of the rows' new states)."""
    nb, t, d = x.shape
    per = d // B.shape[2]
    out, mag = np.zeros(x.shape), np.zeros(x.shape)
    smag = np.abs(state)
    for b, n in enumerate(_lengths(nb, t, ctx, idx)):
        if n == 0:
            continue
        row = b if idx is None else int(idx[b])
        h, hm = state[row].copy(), np.abs(state[row])
        for k in range(n):
            v = dt[b, k] + (0.0 if dt_bias is None else dt_bias)
            if softplus:
                v = np.logaddexp(0.0, v)
            Bk, Ck = np.repeat(B[b, k], per, 0), np.repeat(C[b, k], per, 0)
            decay = np.exp(A * v[:, None])
            u = Bk * (v * x[b, k])[:, None]
            h = h * decay + u
            hm = hm * decay + np.abs(u)
            skip = 0.0 if D is None else D * x[b, k]
            y = (h * Ck).sum(1) + skip
            m = (hm * np.abs(Ck)).sum(1) + np.abs(skip)
            if z is not None:
                y, m = y * _silu(z[b, k]), m * np.abs(_silu(z[b, k]))
            out[b, k], mag[b, k] = y, m
        if update:
            state[row] = h
            smag[row] = hm
    return out, mag, smag


def _draw(w, u):
    w = np.where(w > 0, w, 0.0)  # negative and NaN count as 0
    if not w.sum() > 0:
        return -1
    c = np.cumsum(w)
    hit = np.nonzero((c > u * c[-1]) & (w > 0))[0]
    return int(hit[0]) if hit.size else int(np.nonzero(w)[0][-1])


def draft_verify(tokens, target, uniforms, *, draft=None, parents=None, ctx=None, idx=None,
                 max_accept=None):
    """-> (accepted [b], next [b], path [b, max_accept])."""
    nb, t, v = target.shape
    most = t if max_accept is None else max_accept
    acc, nxt = np.zeros(nb, np.int32), np.full(nb, -1, np.int32)
    path = np.full((nb, most), -1, np.int32)
    for b, n in enumerate(_lengths(nb, t, ctx, idx)):
        if n == 0:
            continue
        chain = [0]

        def prob(row, x):
            p = row[x] if 0 <= x < v else 0.0
            return p if p > 0 else 0.0

        if draft is not None:
            w = target[b, 0]
            for k in range(1, n):
                if len(chain) == most:
                    break
                x = int(tokens[b, k])
                q = draft[b, k - 1]
                if uniforms[b, k] * (q[x] if 0 <= x < v else 0.0) < prob(target[b, k - 1], x):
                    chain.append(k)
                    w = target[b, k]
                else:
                    w = target[b, k - 1] - q
                    break
        else:
            at, left, w = 0, 1.0, target[b, 0].copy()
            for k in range(1, n):
                par = k - 1 if parents is None else int(parents[b, k])
                if len(chain) == most:
                    break
                if par != at or not 0 <= par < k:
                    continue
                x = int(tokens[b, k])
                if uniforms[b, k] * left < prob(w, x):
                    chain.append(k)
                    at, left, w = k, 1.0, target[b, k].copy()
                elif 0 <= x < v:
                    left -= prob(w, x)
                    w[x] = 0.0
        got = _draw(w, uniforms[b, 0])
        if got < 0:
            got = _draw(target[b, chain[-1]], uniforms[b, 0])
        acc[b], nxt[b] = len(chain), got
        path[b, :len(chain)] = chain
    return acc, nxt, path
