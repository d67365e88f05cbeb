"""Refusals of the gated delta rule, norm and log probability entry points (no
GPU: every path here returns before any HIP call) and the layout of their structs."""
import ctypes
import os
import subprocess

import pytest

from linear_rnn_recurrent_amd import ssu as S

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x100000  # a 16-byte aligned non-null pointer value, never dereferenced


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(S.LIB_PATH):
        from linear_rnn_recurrent_amd import build
        build.build()
    return S.load_library()


def err(lib):
    return lib.ssu_last_error().decode()


def test_struct_layouts_match_the_header(tmp_path):
    names = ("ssu_delta_dims", "ssu_norm_dims", "ssu_logprob_dims")
    fields = [(n, f[0]) for n in names for f in getattr(S, n)._fields_]
    src = tmp_path / "sz.c"
    src.write_text('#include "ssu.h"\n#include <stdio.h>\n#include <stddef.h>\nint main(void){'
                   + "".join(f'printf("%zu\\n", sizeof({n}));' for n in names)
                   + "".join(f'printf("%zu\\n", offsetof({n}, {f}));' for n, f in fields)
                   + 'printf("%d %d\\n", SSU_E4M3, SSU_MAX_TOP);return 0;}\n')
    exe = tmp_path / "sz"
    subprocess.run(["gcc", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"),
                    "-I", "/opt/rocm/include", str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True,
                                          check=True).stdout.split()]
    assert got == ([ctypes.sizeof(getattr(S, n)) for n in names]
                   + [getattr(getattr(S, n), f).offset for n, f in fields] + [S.SSU_E4M3, S.SSU_MAX_TOP])


def delta_dims(**kw):
    d = dict(batch=2, num_q_heads=2, num_v_heads=4, head_dim=64, pool_rows=4, use_qk_l2norm=1, state_dtype=0,
             io_dtype=2, gate_dtype=0, bias_dtype=0, state_row_stride=0)
    for k in ("q", "k", "v", "a", "b", "out"):
        d[k + "_batch_stride"] = d[k + "_token_stride"] = 0
    d.update(kw)
    return S.ssu_delta_dims(*d.values())


def delta(lib, d, seq_len=8, update=1, step=False, ws=FAKE, ws_bytes=1 << 50, **ptrs):
    p = dict(q=FAKE, k=FAKE + 64, v=FAKE + 128, a=FAKE + 192, b=FAKE + 256, A_log=None, dt_bias=None, state=FAKE,
             out=FAKE + 320, ctx=None, idx=None)
    p.update(ptrs)
    args = [p[n] for n in ("q", "k", "v", "a", "b", "A_log", "dt_bias")]
    if step:
        return lib.ssu_delta_decode(d, *args, 0.0, p["state"], p["out"], p["idx"], None)
    return lib.ssu_delta_prefill(d, seq_len, *args, 0.0, p["state"], p["out"], update, p["ctx"], p["idx"], ws,
                                 ws_bytes, None)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(batch=-1), 1, "batch"), (dict(num_q_heads=0), 1, "> 0"), (dict(num_v_heads=0), 1, "> 0"),
    (dict(pool_rows=0), 1, "> 0"), (dict(num_q_heads=3), 1, "multiple"), (dict(head_dim=96), 2, "head_dim"),
    (dict(head_dim=0), 2, "head_dim"), (dict(state_dtype=3), 2, "dtype"), (dict(io_dtype=4), 2, "dtype"),
    (dict(gate_dtype=-1), 2, "dtype"), (dict(bias_dtype=9), 2, "dtype"), (dict(batch=5), 1, "pool_rows"),
    (dict(state_row_stride=4 * 64 * 64 - 4), 1, "state_row_stride"), (dict(state_row_stride=4 * 64 * 64 + 2), 1, "16-byte"),
    (dict(q_token_stride=127), 1, "q token stride"), (dict(k_batch_stride=8), 1, "k batch stride"),
    (dict(v_token_stride=-256), 1, "v token stride"), (dict(a_token_stride=3), 1, "a token stride"),
    (dict(b_batch_stride=5), 1, "b batch stride"), (dict(out_token_stride=255), 1, "out token stride"),
    (dict(v_token_stride=(1 << 25) + 1), 2, "2^25"), (dict(num_q_heads=1 << 20, num_v_heads=1 << 20), 2, "2^25"),
])
def test_delta_rejects_bad_dims(lib, kw, status, needle):
    assert delta(lib, delta_dims(**kw)) == status
    assert needle in err(lib)


def test_delta_pointers(lib):
    assert lib.ssu_delta_prefill(None, 8, *([FAKE] * 7), 0.0, FAKE, FAKE, 1, None, None, None, 0, None) == 1
    for name in ("q", "k", "v", "a", "b", "state"):
        assert delta(lib, delta_dims(), **{name: None}) == 1 and f"'{name}'" in err(lib)
        assert delta(lib, delta_dims(), **{name: FAKE + 1}) == 1 and f"'{name}'" in err(lib)
    assert delta(lib, delta_dims(), state=FAKE + 8) == 1 and "'state'" in err(lib)
    assert delta(lib, delta_dims(), out=None, update=0) == 1 and "'out'" in err(lib)
    assert delta(lib, delta_dims(), step=True, out=None) == 1 and "'out'" in err(lib)
    assert delta(lib, delta_dims(), dt_bias=FAKE) == 1 and "A_log" in err(lib)
    assert delta(lib, delta_dims(), A_log=FAKE + 2) == 1 and "'A_log'" in err(lib)
    for at in (0, 64, 128, 192, 256):
        assert delta(lib, delta_dims(), out=FAKE + at) == 1 and "overlap" in err(lib)
    assert delta(lib, delta_dims(v_batch_stride=512), step=True, out=FAKE + 128) == 1 and "strides" in err(lib)
    assert delta(lib, delta_dims(), seq_len=-1) == 1 and "seq_len" in err(lib)
    assert delta(lib, delta_dims(), seq_len=(1 << 30) + 1) == 2 and "too large" in err(lib)
    assert delta(lib, delta_dims(), idx=FAKE + 2) == 1 and "'state_indices'" in err(lib)
    assert delta(lib, delta_dims(), ctx=FAKE + 1) == 1 and "'context_lengths'" in err(lib)
    for rc in (delta(lib, delta_dims(batch=0), k=None), delta(lib, delta_dims(), seq_len=0, k=None)):
        assert rc == 0 and err(lib) == ""


def test_delta_workspace(lib):
    for seq_len in (1, 7, 4096):
        need = lib.ssu_delta_workspace_bytes(delta_dims(), seq_len)
        assert need >= 0
        if need:
            assert delta(lib, delta_dims(), seq_len=seq_len, ws_bytes=need - 1) == 1 and "workspace_bytes" in err(lib)
            assert delta(lib, delta_dims(), seq_len=seq_len, ws=None) == 1 and "'workspace'" in err(lib)
            assert delta(lib, delta_dims(), seq_len=seq_len, ws=FAKE + 8) == 1 and "'workspace'" in err(lib)
    for bad in (dict(batch=-1), dict(head_dim=48), dict(num_q_heads=3), dict(io_dtype=7), dict(num_q_heads=0)):
        assert lib.ssu_delta_workspace_bytes(delta_dims(**bad), 8) == -1
    assert lib.ssu_delta_workspace_bytes(delta_dims(), -1) == -1
    assert lib.ssu_delta_workspace_bytes(None, 8) == -1
    assert lib.ssu_delta_workspace_bytes(delta_dims(batch=0), 4096) == 0
    assert lib.ssu_delta_workspace_bytes(delta_dims(), 0) == 0


def norm_dims(**kw):
    d = dict(batch=2, num_tokens=3, columns=256, group=256, scale_block=0, weight_columns=256, io_dtype=2,
             weight_dtype=2, residual_dtype=2, out_dtype=2, unit_offset=0, gate_first=0)
    for k in ("x", "z", "residual", "out"):
        d[k + "_batch_stride"] = d[k + "_token_stride"] = 0
    d.update(kw)
    return S.ssu_norm_dims(*d.values())


def norm(lib, d, eps=1e-6, **ptrs):
    p = dict(x=FAKE, weight=FAKE + 64, residual=None, z=None, out=FAKE + 128, scales=None)
    p.update(ptrs)
    return lib.ssu_rms_norm(d, p["x"], p["weight"], p["residual"], p["z"], p["out"], p["scales"], eps, None)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(batch=-1), 1, "batch"), (dict(num_tokens=-1), 1, "num_tokens"), (dict(columns=0), 1, "> 0"),
    (dict(group=0), 1, "> 0"), (dict(group=96), 1, "multiple"), (dict(weight_columns=64), 1, "weight_columns"),
    (dict(io_dtype=4), 2, "dtype"), (dict(weight_dtype=3), 2, "dtype"), (dict(residual_dtype=5), 2, "dtype"),
    (dict(out_dtype=3), 2, "dtype"), (dict(scale_block=128), 1, "scales"),
    (dict(out_dtype=4), 1, "scale_block"), (dict(out_dtype=4, scale_block=100), 1, "scale_block"),
    (dict(out_dtype=4, columns=288, group=288, weight_columns=288, scale_block=96), 2, "power of two"),
    (dict(out_dtype=4, columns=2048, group=2048, weight_columns=2048, scale_block=1024), 2, "power of two"),
    (dict(out_dtype=4, scale_block=4), 2, "power of two"),
    (dict(out_dtype=4, columns=192, group=96, weight_columns=96, scale_block=64), 2, "power of two"),
    (dict(columns=32769, group=32769, weight_columns=32769), 2, "32768"),
    (dict(x_token_stride=255), 1, "x token stride"), (dict(z_batch_stride=5), 1, "z batch stride"),
    (dict(residual_token_stride=-256), 1, "residual token stride"), (dict(out_batch_stride=-1), 1, "out batch stride"),
])
def test_norm_rejects_bad_dims(lib, kw, status, needle):
    assert norm(lib, norm_dims(**kw)) == status
    assert needle in err(lib)


def test_norm_pointers(lib):
    assert lib.ssu_rms_norm(None, *([FAKE] * 6), 1e-6, None) == 1
    for name in ("x", "weight", "out"):
        assert norm(lib, norm_dims(), **{name: None}) == 1 and f"'{name}'" in err(lib)
    for name in ("x", "weight", "out", "residual", "z"):
        assert norm(lib, norm_dims(), **{name: FAKE + 1}) == 1 and f"'{name}'" in err(lib)
    coded = norm_dims(out_dtype=4, scale_block=256)
    assert norm(lib, coded) == 1 and "'scales'" in err(lib)
    assert norm(lib, norm_dims(), scales=FAKE) == 1 and "scales" in err(lib)
    for at in (0, 128):
        assert norm(lib, norm_dims(), residual=FAKE + at) == 1 and "overlap" in err(lib)
    assert norm(lib, norm_dims(), residual=FAKE + 192, z=FAKE + 192) == 1 and "overlap" in err(lib)
    assert norm(lib, norm_dims(x_token_stride=512), out=FAKE) == 1 and "strides" in err(lib)
    assert norm(lib, norm_dims(out_dtype=0), z=FAKE + 192, out=FAKE + 192) == 1 and "type" in err(lib)
    assert norm(lib, coded, scales=FAKE, out=FAKE) == 1 and "type" in err(lib)
    assert norm(lib, norm_dims(), eps=-1.0) == 1 and "eps" in err(lib)
    assert norm(lib, norm_dims(), eps=float("nan")) == 1 and "eps" in err(lib)
    for kw in (dict(batch=0), dict(num_tokens=0)):
        assert norm(lib, norm_dims(**kw), x=None) == 0 and err(lib) == ""


def logprob_dims(**kw):
    d = dict(batch=2, num_tokens=3, vocab=1000, top=4, logit_dtype=0, reserved=0, logit_batch_stride=0,
             logit_row_stride=0)
    d.update(kw)
    return S.ssu_logprob_dims(*d.values())


def logprobs(lib, d, ws=FAKE, ws_bytes=1 << 50, **ptrs):
    p = dict(logits=FAKE, tokens=FAKE, ctx=None, idx=None, logprobs=FAKE, entropy=FAKE, ids=FAKE, top=FAKE)
    p.update(ptrs)
    return lib.ssu_token_logprobs(d, p["logits"], p["tokens"], p["ctx"], p["idx"], p["logprobs"], p["entropy"],
                                  p["ids"], p["top"], ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(reserved=1), 1, "reserved"), (dict(batch=-1), 1, "batch"), (dict(num_tokens=-2), 1, "num_tokens"),
    (dict(vocab=0), 1, "vocab"), (dict(vocab=(1 << 24) + 1), 1, "vocab"), (dict(logit_dtype=3), 2, "dtype"),
    (dict(top=0), 1, "top"), (dict(top=33), 1, "top"), (dict(vocab=3), 1, "top"),
    (dict(batch=1 << 13, num_tokens=1 << 13), 2, "2^25"), (dict(logit_row_stride=999), 1, "logits token stride"),
    (dict(logit_batch_stride=1), 1, "logits batch stride"),
])
def test_logprobs_reject_bad_dims(lib, kw, status, needle):
    assert logprobs(lib, logprob_dims(**kw)) == status
    assert needle in err(lib)


def test_logprobs_pointers_and_workspace(lib):
    assert lib.ssu_token_logprobs(None, *([FAKE] * 9), 0, None) == 1
    for name in ("logits", "tokens", "logprobs"):
        assert logprobs(lib, logprob_dims(), **{name: None}) == 1 and f"'{name}'" in err(lib)
    for name in ("ids", "top"):
        assert logprobs(lib, logprob_dims(), **{name: None}) == 1 and "together" in err(lib)
    for name in ("logits", "tokens", "ctx", "idx", "logprobs", "entropy", "ids", "top"):
        assert logprobs(lib, logprob_dims(), **{name: FAKE + 2}) == 1 and "aligned" in err(lib)
    d = logprob_dims(vocab=100000)
    need = lib.ssu_logprobs_workspace_bytes(d)
    assert need > 0
    assert logprobs(lib, d, ws_bytes=need - 1) == 1 and "workspace_bytes" in err(lib)
    assert logprobs(lib, d, ws=None) == 1 and "'workspace'" in err(lib)
    for kw in (dict(batch=0), dict(num_tokens=0)):
        assert logprobs(lib, logprob_dims(**kw), logits=None) == 0 and err(lib) == ""
        assert lib.ssu_logprobs_workspace_bytes(logprob_dims(**kw)) == 0
    for bad in (dict(batch=-1), dict(vocab=0), dict(top=33), dict(top=-1), dict(vocab=2), dict(batch=1 << 26, num_tokens=1)):
        assert lib.ssu_logprobs_workspace_bytes(logprob_dims(**bad)) == -1
    assert lib.ssu_logprobs_workspace_bytes(None) == -1
