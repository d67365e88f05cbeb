"""Inputs and tolerances of the convolution, scan and draft-verification tests
(not a test module).

Tolerances count roundings. u = 2^-24 is half a step of fp32; a value stored in
type t is off by at most eps(t)/2 relative, and by half the smallest subnormal.
"""
import numpy as np
import torch

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = 2.0 ** -24


def f64(t):
    if t is None:
        return None
    t = t.detach().cpu()
    return t.double().numpy() if t.is_floating_point() else t.numpy()


def store_error(ref, dtype):
    """Half a step of `dtype` at ref, and half its smallest subnormal."""
    fi = torch.finfo(dtype)
    return np.abs(ref) * fi.eps / 2 + fi.smallest_normal * fi.eps / 2


def check(got, ref, bound, dtype, what):
    """|got - ref| <= bound + the rounding to dtype. The value that is rounded
    may itself be off by `bound`, hence the rounding of |ref| + bound."""
    err = np.abs(f64(got) - ref)
    lim = bound + store_error(np.abs(ref) + bound, dtype)
    bad = ~(err <= lim)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, err / lim, 0)), err.shape)
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} off; worst at {i}: got "
                             f"{f64(got)[i]!r} ref {ref[i]!r} limit {lim[i]!r}")


def conv_bound(ref, mag, width):
    """W products and sums and the bias: W + 1 roundings of a partial sum of at
    most mag. silu has a slope of at most 1.1 and its own exp, reciprocal and
    product: 8 roundings of the result, counting the exp's argument (|v| u
    relative, and |v| silu'(v) stays below 1.1 (1 + |v|))."""
    return 1.1 * (width + 1) * U * mag + 8 * U * (np.abs(ref) + 1.1 * mag)


def scan_bound(mag, steps, dstate):
    """Every step rounds the state three times (product with the decay, the new
    term, their sum), softplus, exp and their arguments add at most 16 roundings
    to each term (exp's argument error |a| c u is damped by exp(-|a|), so its sum
    over any number of steps stays below c u / e of the term), and a work split
    over time doubles the rounding of the carried state. dstate sums, the skip,
    the gate: dstate + 16 more."""
    return (32 + 6 * steps + dstate) * U * mag


def strided(t, extra, lead):
    """t as a slice of a wider tensor: `extra` more entries in the last axis of
    its 2-D or 3-D (rows of `lead` leading axes) form, filled with NaN."""
    shape = list(t.shape)
    row = int(np.prod(shape[lead:]))
    wide = torch.full(shape[:lead] + [row + extra], float("nan"), dtype=t.dtype, device=t.device)
    v = wide[..., extra // 2: extra // 2 + row]
    v = v.unflatten(-1, shape[lead:]) if len(shape) > lead + 1 else v
    v.copy_(t)
    return v


def conv_inputs(seed, *, batch, seq_len, channels, width, io="bf16", wt=None, st=None, pool=None,
                idx="perm", ctx=None, layout="chan", bias=True, wide=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    pool = batch + 3 if pool is None else pool
    T = {"x": r(batch, seq_len, channels).to(DT[io]).cuda(),
         "weight": (r(channels, width) * width ** -0.5).to(DT[wt or io]).cuda(),
         "bias": (r(channels) * 0.3).to(DT[wt or io]).cuda() if bias else None}
    if wide:
        T["x"] = strided(T["x"], wide, 2)
    s = r(pool, channels, width - 1).to(DT[st or io]).cuda()
    if layout == "tap":
        s = s.transpose(1, 2).contiguous().transpose(1, 2)
    elif layout == "padded":  # row stride and channel stride larger than dense
        big = torch.full((pool, channels + 1, width + 1), float("nan"), dtype=s.dtype, device="cuda")
        big[:, :channels, 1:width] = s
        s = big[:, :channels, 1:width]
    T["conv_state"] = s
    if isinstance(idx, str):
        T["idx"] = None if idx == "none" else torch.randperm(pool, generator=g)[:batch].int().cuda()
    else:
        T["idx"] = torch.tensor(idx, dtype=torch.int32).cuda()
    T["ctx"] = None if ctx is None else torch.tensor(ctx, dtype=torch.int32).cuda()
    return T


def scan_inputs(seed, *, batch, seq_len, dim, dstate, groups=1, io="bf16", dt="f32", bc=None,
                st="f32", pool=None, idx="perm", ctx=None, gate=True, D=True, bias=True, wide=0,
                row_pad=0, dt_scale=0.5):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    pool = batch + 3 if pool is None else pool
    T = {"x": r(batch, seq_len, dim).to(DT[io]).cuda(),
         "z": r(batch, seq_len, dim).to(DT[io]).cuda() if gate else None,
         "dt": (r(batch, seq_len, dim) * dt_scale).to(DT[dt]).cuda(),
         "B": r(batch, seq_len, groups, dstate).to(DT[bc or io]).cuda(),
         "C": r(batch, seq_len, groups, dstate).to(DT[bc or io]).cuda(),
         "A": -torch.exp(torch.rand(dim, dstate, generator=g) * np.log(16.0)).cuda(),
         "D": r(dim).cuda() if D else None,
         "dt_bias": torch.log(torch.expm1(torch.rand(dim, generator=g) * 0.099 + 0.001)).cuda()
         if bias else None}
    if wide:
        for k in ("x", "z", "dt", "B", "C"):
            if T[k] is not None:
                T[k] = strided(T[k], wide, 2)
    s = r(pool, dim, dstate).to(DT[st]).cuda()
    if row_pad:
        big = torch.full((pool, dim * dstate + row_pad), float("nan"), dtype=s.dtype, device="cuda")
        big[:, :dim * dstate] = s.flatten(1)
        s = big[:, :dim * dstate].unflatten(1, (dim, dstate))
    T["state"] = s
    if isinstance(idx, str):
        T["idx"] = None if idx == "none" else torch.randperm(pool, generator=g)[:batch].int().cuda()
    else:
        T["idx"] = torch.tensor(idx, dtype=torch.int32).cuda()
    T["ctx"] = None if ctx is None else torch.tensor(ctx, dtype=torch.int32).cuda()
    return T


def verify_inputs(seed, *, batch, tokens, vocab, probs="f32", tree=False, draft=True, ctx=None,
                  idx=None, sharp=4.0, wide=0):
    """Drafts sampled from (chains with draft) or ranked by a noisy copy of the
    target, so that several tokens in a row are accepted."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    logits = r(batch, tokens, vocab) * sharp
    p = logits.softmax(-1).to(DT[probs])
    T = {"target": p, "uniforms": torch.rand(batch, tokens, generator=g), "draft": None,
         "parents": None}
    tok = torch.randint(0, vocab, (batch, tokens), generator=g)
    noisy = logits + r(batch, tokens, vocab)
    if tree:
        par = (torch.rand(batch, tokens, generator=g) * torch.arange(tokens)).long()
        par[:, 0] = -1
        T["parents"] = par.int()
        order = noisy.argsort(-1, descending=True)
        for b in range(batch):
            seen = {}
            for k in range(1, tokens):
                q = int(par[b, k])
                tok[b, k] = order[b, q, min(seen.get(q, 0), vocab - 1)]
                seen[q] = seen.get(q, 0) + 1
    elif tokens > 1:
        q = noisy[:, :-1].softmax(-1)
        tok[:, 1:] = torch.multinomial(q.reshape(-1, vocab), 1, generator=g).reshape(batch, -1)
        if draft:
            T["draft"] = q.to(DT[probs])
    elif draft:
        T["draft"] = p[:, :0]
    T["tokens"] = tok.int()
    T["ctx"] = None if ctx is None else torch.tensor(ctx, dtype=torch.int32)
    T["idx"] = None if idx is None else torch.tensor(idx, dtype=torch.int32)
    T = {k: None if v is None else v.cuda() for k, v in T.items()}
    if wide:
        T["target"] = strided(T["target"], wide, 2)
        if T["draft"] is not None:
            T["draft"] = strided(T["draft"], wide, 2)
    return T
