"""Every evaluation of the per-channel scan, at sizes whose choice is checked on the
CPU (tests/test_scan_plan.py): outputs and states, the read-only window, the commit
without outputs, all pairs of types, against the fp64 oracle."""
import itertools

import numpy as np
import pytest
import torch

import oracle
from linear_rnn_recurrent_amd import ssu_scan_prefill
from gpu_helpers import assert_bitwise
from scan_evaluations import SIZES, TYPED
from sequence_helpers import check, f64, scan_bound, scan_inputs

pytestmark = pytest.mark.gpu

TYPES = [("bf16", "bf16", "bf16", "f32"), ("f32", "f32", "f32", "f32"), ("f16", "f32", "f16", "bf16"),
         ("bf16", "f32", "f32", "f16")]


def build(size, io, dt, bc, st, wide):
    """Uneven lengths (all, 0, 1, too many among them) where there are any, a padding
    row, views of wider tensors at offsets that are and are not multiples of four,
    padded pool rows; NaN in everything that may not be read."""
    batch, seq_len, dim, dstate, groups, lengths = size
    g = np.random.default_rng(seq_len + dim)
    ctx = None
    if lengths:
        ctx = g.integers(0, seq_len + 1, batch)
        ctx[0] = seq_len - 1 if batch == 1 else seq_len + 7
        if batch > 2:
            ctx[1], ctx[2] = 0, 1
        elif batch == 2:
            ctx[1] = max(seq_len - seq_len // 3, 1)
    idx = g.permutation(batch + 2)[:batch]
    if batch > 3:
        idx[3] = -4
    T = scan_inputs(seq_len + dim, batch=batch, seq_len=seq_len, dim=dim, dstate=dstate, groups=groups, io=io,
                    dt=dt, bc=bc, st=st, ctx=None if ctx is None else ctx.tolist(), idx=idx.tolist(), wide=wide,
                    row_pad=16, gate=wide != 3)
    counts = [0 if idx[b] < 0 else seq_len if ctx is None else min(int(ctx[b]), seq_len) for b in range(batch)]
    for b, n in enumerate(counts):
        for k in ("x", "z", "dt", "B", "C"):
            if T[k] is not None:
                T[k][b, n:] = float("nan")
    T["counts"] = counts
    return T


def run(T, state, out, update=True, C=True):
    ssu_scan_prefill(T["x"], T["A"], T["B"], T["C"] if C else None, T["dt"], state, out, dt_bias=T["dt_bias"],
                     D=T["D"], z=T["z"], context_lengths=T["ctx"], state_indices=T["idx"], update_state=update)


def compare(T):
    """The call, the window and the commit against one oracle run."""
    seq_len, dstate = T["x"].shape[1], T["B"].shape[-1]
    want = f64(T["state"]).copy()
    ref, mag, smag = oracle.channel_scan(
        f64(T["x"]), f64(T["A"]), f64(T["B"]), f64(T["C"]), f64(T["dt"]), want, dt_bias=f64(T["dt_bias"]),
        D=f64(T["D"]), z=f64(T["z"]), ctx=f64(T["ctx"]), idx=f64(T["idx"]))
    idx = f64(T["idx"])
    live = np.zeros(T["state"].shape[0], bool)
    live[idx[idx >= 0]] = True
    pool = T["state"]
    before = pool.clone()
    for kind in ("window", "commit", "both"):
        out = None if kind == "commit" else torch.full(T["x"].shape, float("nan"), dtype=T["x"].dtype,
                                                       device="cuda")
        run(T, pool, out, update=kind != "window", C=kind != "commit")
        torch.cuda.synchronize()
        if out is not None:
            check(out, ref, scan_bound(mag, seq_len, dstate), out.dtype, f"{kind}: out")
            for b, n in enumerate(T["counts"]):  # +0.0 past a row's end
                assert_bitwise(out[b, n:], torch.zeros_like(out[b, n:]), f"{kind}: row {b}'s end")
        if kind == "window":
            assert_bitwise(pool, before, "pool after a window")
            continue
        check(pool[live], want[live], scan_bound(smag[live], seq_len, 0), pool.dtype, f"{kind}: state")
        assert_bitwise(pool[~live], before[~live], "rows of nobody")
        pool.copy_(before)


@pytest.mark.parametrize("size", SIZES, ids=lambda s: "-".join(map(str, s)))
def test_listed_sizes(size):
    i = list(SIZES).index(size)
    compare(build(size, *TYPES[i % 4], wide=(4, 3, 16, 1)[(i // 4) % 4]))


@pytest.mark.parametrize("size", TYPED, ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("io,dt", list(itertools.product(("f32", "f16", "bf16"), repeat=2)))
def test_pairs_of_types(size, io, dt):
    """x, z and out by dt; B and C in each of the three types, read four at a time and
    one at a time."""
    for bc, wide in (("f32", 4), ("f16", 16), ("bf16", 3), (io, 4)):
        compare(build(size, io, dt, bc, "f32" if bc == io else "bf16", wide=wide))
