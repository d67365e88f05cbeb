"""RMS norm with residual, gate and e4m3 output against the fp64 oracle."""
import numpy as np
import pytest
import torch

import linear_rnn_recurrent_amd as L
from gpu_helpers import assert_bitwise
from oracle import serving
from sequence_helpers import DT, U, check, f64, store_error, strided

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


def inputs(seed, shape, *, io="bf16", wt=None, res=None, gate=None, group=None, wide=0, size=1.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    n = shape[-1]
    T = {"x": (r(*shape) * size).to(DT[io]).cuda(), "weight": (1 + 0.3 * r(group or n)).to(DT[wt or io]).cuda(),
         "residual": (r(*shape) * 2 * size).to(DT[res]).cuda() if res else None,
         "z": r(*shape).to(DT[io]).cuda() if gate else None}
    if wide:
        for k in ("x", "residual", "z"):
            if T[k] is not None:
                T[k] = strided(T[k], wide, len(shape) - 1)
    return T


def bounds(T, group, unit, gate):
    """(y, its bound, h): a group's sum of squares rounds n + 1 times (all terms positive), half of
    that reaches its root; then the division, the root, two products, the weight's offset, the
    residual's sum and a gate's exp, sum, division (with |z| u from its argument) are 16 more. A
    gate in front moves the root as it moves a square, by less than twice its own."""
    A = {k: f64(t) for k, t in T.items()}
    y, h = serving.rms_norm(A["x"], A["weight"], residual=A["residual"], z=A["z"], group=group, unit=unit,
                            gate_first=gate == "before")
    z = 0.0 if A["z"] is None else np.abs(A["z"])
    n = group or y.shape[-1]
    rel = (n / 2 + 24 + 3 * np.max(z) if gate == "before" else n / 2 + 24 + z) * U
    # what a sum with the residual loses against its parts, seen from the row's size
    loss = 0.0
    if h is not None:
        w = np.broadcast_to(np.abs(A["weight"] if A["weight"].shape[0] == y.shape[-1] else
                                   np.tile(A["weight"], y.shape[-1] // n)) + unit, y.shape)
        p = h.reshape(h.shape[:-1] + (-1, n))
        inv = np.repeat(1 / np.sqrt((p ** 2).mean(-1) + 1e-6), n, -1)
        loss = U * (np.abs(A["x"]) + np.abs(A["residual"])) * inv * w
    return y, rel * np.abs(y) + loss, h


def run(T, out_dtype, *, group=None, unit=False, gate=None, block=None, out=None):
    shape = T["x"].shape
    out = torch.full(shape, float("nan"), device="cuda").to(out_dtype) if out is None else out
    scales = torch.full(shape[:-1] + (shape[-1] // block,), float("nan"), device="cuda") if block else None
    L.ssu_rms_norm(T["x"], T["weight"], out, residual=T["residual"], z=T["z"], scales=scales, group_size=group,
                   unit_offset=unit, gate_first=gate == "before")
    torch.cuda.synchronize()
    return out, scales


def verify(T, out_dtype, *, group=None, unit=False, gate=None, block=None):
    y, bound, h = bounds(T, group, unit, gate)
    out, scales = run(T, out_dtype, group=group, unit=unit, gate=gate, block=block)
    if h is not None:
        check(T["residual"], h, U * np.abs(h), T["residual"].dtype, "residual")
    if not block:
        check(out, y, bound, out_dtype, "out")
        return
    p, pb = (a.reshape(a.shape[:-1] + (-1, block)) for a in (y, bound))
    most = np.abs(p).max(-1)
    s = np.maximum(most / 448, 2.0 ** -126)
    serr = np.where(most / 448 > 2.0 ** -126, pb.max(-1) / 448 + 2 * U * s, 0.0)
    assert (np.abs(f64(scales) - s) <= serr).all()
    # a code stands for y within half its step (2^-4 of the value, 2^-10 below 2^-6) of what was
    # divided, which is off by y's bound, the scale's and two roundings
    code = f64(out.float()).reshape(p.shape)
    v = p / s[..., None]
    off = pb / s[..., None] + np.abs(v) * (serr / s + 0.0)[..., None] + 3 * U * np.abs(v)
    assert np.isfinite(code).all()
    lim = np.maximum((np.abs(v) + off) * 2.0 ** -4, 2.0 ** -10) + off
    assert (np.abs(code - v) <= lim).all()
    # and all but those next to the middle of two codes are the nearest code
    lead = np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -6)))
    ulp = np.exp2(lead - 3)
    near = np.abs(np.abs(v / ulp - np.floor(v / ulp)) - 0.5) * ulp <= off
    assert (np.where(near, 0.0, code - np.round(v / ulp) * ulp) == 0).all()


@pytest.mark.parametrize("n", [1, 7, 8, 64, 96, 100, 128, 513, 1000, 2048, 5120, 16384, 20001, 32768])
@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
def test_columns(n, io):
    verify(inputs(1, (3, n), io=io), DT[io])


@pytest.mark.parametrize("io,wt,res,out", [("bf16", "f32", "f32", "bf16"), ("f16", "bf16", "f16", "f32"),
                                           ("f32", "f16", "bf16", "f16"), ("bf16", "bf16", "bf16", "f32")])
@pytest.mark.parametrize("unit", [False, True])
def test_types_and_residuals(io, wt, res, out, unit):
    verify(inputs(2, (5, 776), io=io, wt=wt, res=res), DT[out], unit=unit)


@pytest.mark.parametrize("gate", ["after", "before"])
@pytest.mark.parametrize("n,group", [(4096, 128), (1024, 64), (512, 512), (960, 96), (2048, 1024), (35, 7),
                                     (5120, 640), (8192, 4096), (40000, 20000)])
def test_groups_and_gates(n, group, gate):
    verify(inputs(3, (4, n), gate=gate, group=group), torch.bfloat16, group=group, gate=gate)
    verify(inputs(4, (4, n), gate=gate, io="f32"), torch.float32, group=group, gate=gate) if n <= 32768 else None


@pytest.mark.parametrize("n,group,block", [(2048, None, 2048), (2048, None, 128), (512, None, 8), (520, None, 520),
                                           (100, None, 100), (4096, 128, 4096), (1024, 128, 128), (1024, 64, 512),
                                           (5120, None, 64), (20480, None, 512), (24, 8, 24), (1001, None, 1001)])
@pytest.mark.parametrize("io,res", [("bf16", "bf16"), ("f16", "f32"), ("f32", None)])
def test_codes_and_scales(n, group, block, io, res):
    verify(inputs(5, (6, n), io=io, res=res, group=group), E4M3, group=group, block=block)


@pytest.mark.parametrize("wide", [16, 6, 3])
@pytest.mark.parametrize("n", [128, 2048])
def test_slices_of_wider_tensors(n, wide):
    verify(inputs(6, (3, 5, n), res="f32", gate="after", wide=wide), torch.bfloat16, gate="after")
    verify(inputs(7, (15, n), res="bf16", wide=wide), E4M3, block=n)


def test_token_major_rows():
    T = inputs(8, (3, 5, 256), gate="after")
    want, _ = run(T, torch.bfloat16, gate="after")
    for k in ("x", "z"):
        T[k] = T[k].transpose(0, 1).contiguous().transpose(0, 1)
    out = torch.empty(5, 3, 256, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    run(T, torch.bfloat16, gate="after", out=out)
    assert_bitwise(out.contiguous(), want, "out")


@pytest.mark.parametrize("n", [96, 2048, 20000])
@pytest.mark.parametrize("at", ["x", "z"])
def test_output_in_an_inputs_place(n, at):
    T = inputs(9, (4, n), gate="after")
    want, _ = run(T, torch.bfloat16, gate="after")
    run(T, torch.bfloat16, gate="after", out=T[at])
    assert_bitwise(T[at], want, at)


@pytest.mark.parametrize("n", [64, 2048])
def test_rows_of_zeros_small_and_large_values(n):
    T = inputs(10, (5, n), io="f32")
    T["x"][0] = 0.0
    T["x"][1] *= 1e-18   # squares below fp32's range: the epsilon is all of the mean
    T["x"][2] *= 1e15
    T["x"][3] *= 1e-3
    verify(T, torch.float32)
    verify(T, E4M3, block=n)
    out, scales = run(T, E4M3, block=n)
    assert (out[0].float() == 0).all() and scales[0, 0] == 2.0 ** -126


@pytest.mark.parametrize("n,block", [(64, 64), (2048, 2048), (2048, 128)])
def test_a_nan_stays_in_its_row(n, block):
    T = inputs(11, (4, n))
    want, ws = run(T, E4M3, block=block)
    T["x"][2, 5] = float("nan")
    out, scales = run(T, E4M3, block=block)
    keep = [0, 1, 3]
    assert torch.equal(out.view(torch.uint8)[keep], want.view(torch.uint8)[keep])
    assert torch.equal(scales[keep], ws[keep])
    assert torch.isnan(out[2].float()).all() and torch.isnan(scales[2]).all()


def test_empty_and_one_row():
    for shape in ((0, 64), (1, 64), (0, 3, 64), (2, 0, 64)):
        verify(inputs(12, shape), torch.bfloat16) if 0 not in shape else run(inputs(12, shape), torch.bfloat16)


def test_many_rows():
    verify(inputs(13, (3001, 128), gate="after"), torch.bfloat16, gate="after")


@pytest.mark.parametrize("n", [128, 4096])
def test_capture(n):
    T = inputs(14, (9, n), res="f32")
    start = T["residual"].clone()
    want, ws = run(T, E4M3, block=n)
    after = T["residual"].clone()
    out, scales = torch.empty_like(want), torch.empty_like(ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.ssu_rms_norm(T["x"], T["weight"], out, residual=T["residual"], scales=scales)
    for _ in range(3):
        T["residual"].copy_(start)
        scales.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.uint8), want.view(torch.uint8)) and torch.equal(scales, ws)
        assert_bitwise(T["residual"], after, "residual")


def test_store_error_of_the_helper():
    assert store_error(np.array([1.0]), torch.bfloat16)[0] >= 2.0 ** -8
