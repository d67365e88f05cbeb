"""Inputs of the gated delta rule, norm and log probability tests (not a test module)."""
import numpy as np
import torch

from sequence_helpers import DT, f64, strided


def delta_inputs(seed, *, batch, seq_len, hq=2, hv=4, d=64, io="bf16", gate="f32", st="f32", pool=None,
                 idx="perm", ctx=None, raw=True, l2=True, wide=0, row_pad=0, a_scale=1.0,
                 step=False):
    """raw: a and b with A_log and dt_bias; otherwise decays' logarithms and betas."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    pool = batch + 3 if pool is None else pool
    T = {"q": r(batch, seq_len, hq, d), "k": r(batch, seq_len, hq, d), "v": r(batch, seq_len, hv, d)}
    if not l2:  # keys of at most unit length: rounding one up by a step of bf16 stays below 1
        T["k"] = T["k"] / T["k"].norm(dim=-1, keepdim=True) * 0.99
    T = {n: t.to(DT[io]).cuda() for n, t in T.items()}
    a, b = r(batch, seq_len, hv) * a_scale, r(batch, seq_len, hv)
    if not raw:
        a, b = -torch.nn.functional.softplus(a - 2.0) * 2.0, torch.sigmoid(b)
    T["a"], T["b"] = a.to(DT[gate]).cuda(), b.to(DT[gate]).cuda()
    T["A_log"] = torch.log(torch.rand(hv, generator=g) * 15 + 1).cuda() if raw else None
    T["dt_bias"] = (torch.rand(hv, generator=g) * 2 - 6).cuda() if raw else None
    if wide:
        for n in ("q", "k", "v", "a", "b"):
            T[n] = strided(T[n], wide, 2)
    s = (r(pool, hv, d, d) * 0.2).to(DT[st]).cuda()
    if row_pad:
        big = torch.full((pool, hv * d * d + row_pad), float("nan"), dtype=s.dtype, device="cuda")
        big[:, :hv * d * d] = s.flatten(1)
        s = big[:, :hv * d * d].unflatten(1, (hv, d, d))
    T["state"] = s
    if isinstance(idx, str):
        T["idx"] = None if idx == "none" else torch.randperm(pool, generator=g)[:batch].int().cuda()
    else:
        T["idx"] = torch.tensor(idx, dtype=torch.int32).cuda()
    T["ctx"] = None if ctx is None else torch.tensor(ctx, dtype=torch.int32).cuda()
    if step:
        T.update({n: T[n][:, 0] for n in ("q", "k", "v", "a", "b")})
    return T


def delta_reference(T, *, step=False, scale=None, l2=True, update=True):
    """(out, its bound, state, its bound), fp64."""
    from oracle import serving
    A = {n: f64(t) for n, t in T.items()}
    if step:
        A.update({n: A[n][:, None] for n in ("q", "k", "v", "a", "b")})
    state = A["state"].copy()
    out, bound, sbound = serving.gated_delta(A["q"], A["k"], A["v"], A["a"], A["b"], state,
                                             A_log=A["A_log"], dt_bias=A["dt_bias"], scale=scale,
                                             l2=l2, ctx=A["ctx"], idx=A["idx"], update=update)
    if step:
        out, bound = out[:, 0], bound[:, 0]
    return out, bound, state, np.broadcast_to(sbound[..., None], state.shape)


def norm_error(got, ref, floor=0.0):
    """2-norm of the difference over the reference's, both over finite entries."""
    g = f64(got)
    return float(np.linalg.norm(g - ref) / max(np.linalg.norm(ref), floor or 1e-300))
