"""Python binding of libssu (ctypes). Argument marshalling only.

Each function takes torch tensors that live on the GPU, checks that their
shapes agree (the C library cannot see shapes), and calls the C entry point of
the same name on torch's current stream. All computation happens in the HIP
kernels of libssu.so; there is no fallback. If the library has not been built
the first call raises RuntimeError (build it with
`python -m linear_rnn_recurrent_amd.build`).
"""
import contextlib
import ctypes
import os
from typing import Optional, Sequence

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libssu.so")

SSU_OK, SSU_EINVAL, SSU_ENOTSUP, SSU_EHIP, SSU_ENOMEM = 0, 1, 2, 3, 4
SSU_F32, SSU_F16, SSU_BF16, SSU_U8, SSU_E4M3 = 0, 1, 2, 3, 4
SSU_MAX_TOP = 32
_DT = {torch.float32: SSU_F32, torch.float16: SSU_F16, torch.bfloat16: SSU_BF16,
       torch.uint8: SSU_U8}

EXPORTS = ("ssu_decode", "ssu_prefill", "ssu_replay", "ssu_tree_verify",
           "ssu_tree_verify_noalloc", "ssu_replay_layers",
           "ssu_state_clear_layers", "ssu_state_gather", "ssu_state_scatter", "ssu_state_pack",
           "ssu_state_unpack", "ssu_conv_prefill", "ssu_conv_decode", "ssu_scan_prefill",
           "ssu_scan_decode", "ssu_scan_workspace_bytes", "ssu_draft_verify", "ssu_verify_workspace_bytes", "ssu_delta_prefill",
           "ssu_delta_decode", "ssu_delta_workspace_bytes", "ssu_rms_norm", "ssu_token_logprobs",
           "ssu_logprobs_workspace_bytes", "ssu_gdn_decode", "ssu_gdn_workspace_bytes", "ssu_tree_workspace_bytes",
           "ssu_pool_bytes_per_slot", "ssu_pool_slab_bytes", "ssu_pool_spec", "ssu_pool_specs",
           "ssu_pool_name", "ssu_pool_owns_memory",
           "ssu_pool_alloc", "ssu_pool_free", "ssu_pool_info", "ssu_pool_state_ptr",
           "ssu_pool_state_bytes_per_slot", "ssu_pool_find_state", "ssu_pool_clear",
           "ssu_pool_clear_slot", "ssu_pool_capture", "ssu_pool_restore",
           "ssu_pool_copy_slot_from", "ssu_last_error", "ssu_version")


class SsuError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__(f"[ssu status {status}] {msg}")
        self.status = status


class ssu_dims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("nheads", ctypes.c_int32), ("dim", ctypes.c_int32),
                ("dstate", ctypes.c_int32), ("ngroups", ctypes.c_int32),
                ("pool_rows", ctypes.c_int32), ("state_row_stride", ctypes.c_int64),
                ("state_dtype", ctypes.c_int32), ("io_dtype", ctypes.c_int32),
                ("bc_dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class ssu_replay_layer(ctypes.Structure):
    _fields_ = [("state", ctypes.c_void_p), ("replay_dA", ctypes.c_void_p),
                ("replay_u", ctypes.c_void_p), ("replay_B", ctypes.c_void_p),
                ("replay_dt", ctypes.c_void_p)]


class ssu_state_layer(ctypes.Structure):
    _fields_ = [("recurrent_state", ctypes.c_void_p), ("conv_state", ctypes.c_void_p)]


class ssu_gdn_dims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("hidden", ctypes.c_int32),
                ("num_q_heads", ctypes.c_int32), ("num_v_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("conv_width", ctypes.c_int32),
                ("pool_rows", ctypes.c_int32), ("use_qk_l2norm", ctypes.c_int32),
                ("ssm_row_stride", ctypes.c_int64), ("conv_slot_stride", ctypes.c_int64),
                ("conv_chan_stride", ctypes.c_int64), ("conv_tap_stride", ctypes.c_int64)]


class ssu_conv_dims(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("batch", "channels", "width", "pool_rows",
                                               "io_dtype", "weight_dtype", "state_dtype",
                                               "reserved")]
                + [(n, ctypes.c_int64) for n in ("x_batch_stride", "x_token_stride",
                                                 "out_batch_stride", "out_token_stride",
                                                 "state_row_stride", "state_chan_stride",
                                                 "state_tap_stride")])


class ssu_scan_dims(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("batch", "dim", "dstate", "ngroups", "pool_rows",
                                               "state_dtype", "io_dtype", "dt_dtype", "bc_dtype",
                                               "reserved")]
                + [(n, ctypes.c_int64) for n in ("state_row_stride",
                                                 "x_batch_stride", "x_token_stride",
                                                 "z_batch_stride", "z_token_stride",
                                                 "out_batch_stride", "out_token_stride",
                                                 "dt_batch_stride", "dt_token_stride",
                                                 "b_batch_stride", "b_token_stride",
                                                 "c_batch_stride", "c_token_stride")])


class ssu_verify_dims(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("batch", "num_tokens", "vocab", "max_accept_len",
                                               "prob_dtype", "reserved")]
                + [(n, ctypes.c_int64) for n in ("target_batch_stride", "target_row_stride",
                                                 "draft_batch_stride", "draft_row_stride")])


class ssu_delta_dims(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("batch", "num_q_heads", "num_v_heads", "head_dim",
                                               "pool_rows", "use_qk_l2norm", "state_dtype",
                                               "io_dtype", "gate_dtype", "bias_dtype")]
                + [(n, ctypes.c_int64) for n in ("state_row_stride",
                                                 "q_batch_stride", "q_token_stride",
                                                 "k_batch_stride", "k_token_stride",
                                                 "v_batch_stride", "v_token_stride",
                                                 "a_batch_stride", "a_token_stride",
                                                 "b_batch_stride", "b_token_stride",
                                                 "out_batch_stride", "out_token_stride")])


class ssu_norm_dims(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("batch", "num_tokens", "columns", "group",
                                               "scale_block", "weight_columns", "io_dtype",
                                               "weight_dtype", "residual_dtype", "out_dtype",
                                               "unit_offset", "gate_first")]
                + [(n, ctypes.c_int64) for n in ("x_batch_stride", "x_token_stride",
                                                 "z_batch_stride", "z_token_stride",
                                                 "residual_batch_stride", "residual_token_stride",
                                                 "out_batch_stride", "out_token_stride")])


class ssu_logprob_dims(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("batch", "num_tokens", "vocab", "top",
                                               "logit_dtype", "reserved")]
                + [(n, ctypes.c_int64) for n in ("logit_batch_stride", "logit_row_stride")])


class ssu_state_spec(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("layer", ctypes.c_int32), ("rank", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("shape", ctypes.c_int64 * 4)]


_LIB = None
_P = ctypes.c_void_p
_I32 = ctypes.c_int32


def load_library(path: Optional[str] = None):
    """Load libssu.so (once) and declare the C signatures."""
    global _LIB
    if _LIB is not None and path is None:
        return _LIB
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"libssu.so not found at {p}: build it with "
                           "`python -m linear_rnn_recurrent_amd.build`")
    lib = ctypes.CDLL(p)
    D = ctypes.POINTER(ssu_dims)
    S = ctypes.POINTER(ssu_state_spec)
    sig = {
        "ssu_decode": [D, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I32, _P, _P],
        "ssu_prefill": [D, _I32, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I32, _P, _P,
                        _P, _P, _P, _P, _P],
        "ssu_replay": [D, _I32, _P, _P, _P, _P, _P, _P, _P, _I32, _P, _I32, _P],
        "ssu_tree_verify": [D, _I32, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I32, _P, _P, _P,
                            _P, _P, _P, _P, _P, ctypes.c_int64, _P],
        "ssu_tree_verify_noalloc": [D, _I32, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I32, _P,
                                    _P, _P, _P, _P, _P, _P, _P],
        "ssu_replay_layers": [D, _I32, _P, _I32, _P, _P, _I32, _P, _I32, _P],
        "ssu_state_clear_layers": [_P, _I32, _I32, _I32, ctypes.c_int64, ctypes.c_int64, _P],
        "ssu_state_gather": [_P, _I32, ctypes.c_int64, _P, ctypes.c_int64, _P, _I32,
                             ctypes.c_int64, _P],
        "ssu_state_scatter": [_P, ctypes.c_int64, _P, _I32, ctypes.c_int64, _P, _I32,
                              ctypes.c_int64, _P],
        "ssu_state_pack": [_P, _I32, ctypes.c_int64, ctypes.c_int64, _P, _I32, _P, _I32, _P, _P],
        "ssu_gdn_decode": [ctypes.POINTER(ssu_gdn_dims), _P, _P, _P, _P, _P, _P, _P, _P,
                           ctypes.c_float, _P, _P, _P, _P, ctypes.c_int64, _P],
        "ssu_conv_prefill": [ctypes.POINTER(ssu_conv_dims), _I32, _P, _P, _P, _P, _P, _I32, _I32,
                             _P, _P, _P],
        "ssu_conv_decode": [ctypes.POINTER(ssu_conv_dims), _P, _P, _P, _P, _P, _I32, _P, _P],
        "ssu_scan_prefill": [ctypes.POINTER(ssu_scan_dims), _I32, _P, _P, _P, _P, _P, _P, _P, _P,
                             _P, _P, _I32, _I32, _P, _P, _P, ctypes.c_int64, _P],
        "ssu_scan_decode": [ctypes.POINTER(ssu_scan_dims), _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                            _I32, _P, _P],
        "ssu_draft_verify": [ctypes.POINTER(ssu_verify_dims), _P, _P, _P, _P, _P, _P, _P, _P, _P,
                             _P, _P, ctypes.c_int64, _P],
        "ssu_delta_prefill": [ctypes.POINTER(ssu_delta_dims), _I32, _P, _P, _P, _P, _P, _P, _P,
                              ctypes.c_float, _P, _P, _I32, _P, _P, _P, ctypes.c_int64, _P],
        "ssu_delta_decode": [ctypes.POINTER(ssu_delta_dims), _P, _P, _P, _P, _P, _P, _P,
                             ctypes.c_float, _P, _P, _P, _P],
        "ssu_rms_norm": [ctypes.POINTER(ssu_norm_dims), _P, _P, _P, _P, _P, _P, ctypes.c_float,
                         _P],
        "ssu_token_logprobs": [ctypes.POINTER(ssu_logprob_dims), _P, _P, _P, _P, _P, _P, _P, _P,
                               _P, ctypes.c_int64, _P],
        "ssu_state_unpack": [_P, _I32, ctypes.c_int64, ctypes.c_int64, _P, _I32, _P, _I32, _P, _P],
        "ssu_pool_bytes_per_slot": [S, _I32, ctypes.POINTER(ctypes.c_size_t)],
        "ssu_pool_slab_bytes": [S, _I32, _I32, ctypes.POINTER(ctypes.c_size_t)],
        "ssu_pool_alloc": [S, _I32, _I32, ctypes.c_char_p, _P, ctypes.c_size_t, _P,
                           ctypes.POINTER(_P)],
        "ssu_pool_spec": [_P, _I32, S],
        "ssu_pool_specs": [_P, S, _I32, ctypes.POINTER(_I32)],
        "ssu_pool_name": [_P, ctypes.POINTER(ctypes.c_char_p)],
        "ssu_pool_owns_memory": [_P, ctypes.POINTER(_I32)],
        "ssu_pool_free": [_P],
        "ssu_pool_info": [_P, ctypes.POINTER(_I32), ctypes.POINTER(_I32)],
        "ssu_pool_state_ptr": [_P, _I32, ctypes.POINTER(_P)],
        "ssu_pool_state_bytes_per_slot": [_P, _I32, ctypes.POINTER(ctypes.c_size_t)],
        "ssu_pool_find_state": [_P, _I32, _I32, ctypes.POINTER(_I32)],
        "ssu_pool_clear": [_P, _P],
        "ssu_pool_clear_slot": [_P, _I32, _P],
        "ssu_pool_capture": [_P, _I32, ctypes.POINTER(_P), ctypes.POINTER(ctypes.c_size_t),
                             _I32, _P],
        "ssu_pool_restore": [_P, _I32, ctypes.POINTER(_P), ctypes.POINTER(ctypes.c_size_t),
                             _I32, _P],
        "ssu_pool_copy_slot_from": [_P, _P, _I32, _I32, _P],
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = ctypes.c_int32
    lib.ssu_tree_workspace_bytes.argtypes = [D, _I32]
    lib.ssu_tree_workspace_bytes.restype = ctypes.c_int64
    lib.ssu_gdn_workspace_bytes.argtypes = [ctypes.POINTER(ssu_gdn_dims)]
    lib.ssu_gdn_workspace_bytes.restype = ctypes.c_int64
    lib.ssu_scan_workspace_bytes.argtypes = [ctypes.POINTER(ssu_scan_dims), _I32]
    lib.ssu_scan_workspace_bytes.restype = ctypes.c_int64
    lib.ssu_verify_workspace_bytes.argtypes = [ctypes.POINTER(ssu_verify_dims)]
    lib.ssu_verify_workspace_bytes.restype = ctypes.c_int64
    lib.ssu_delta_workspace_bytes.argtypes = [ctypes.POINTER(ssu_delta_dims), _I32]
    lib.ssu_delta_workspace_bytes.restype = ctypes.c_int64
    lib.ssu_logprobs_workspace_bytes.argtypes = [ctypes.POINTER(ssu_logprob_dims)]
    lib.ssu_logprobs_workspace_bytes.restype = ctypes.c_int64
    lib.ssu_last_error.argtypes = []
    lib.ssu_last_error.restype = ctypes.c_char_p
    lib.ssu_version.argtypes = []
    lib.ssu_version.restype = ctypes.c_int32
    if path is None:
        _LIB = lib
    return lib


def _check(status):
    if status != SSU_OK:
        raise SsuError(status, load_library().ssu_last_error().decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device, stream):
    if stream is not None:
        return ctypes.c_void_p(stream if isinstance(stream, int) else stream.cuda_stream)
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _need(cond, msg):
    if not cond:
        raise ValueError(msg)


def _dev(t, name, dtypes=None, shape=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if dtypes is not None and t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t


def _dense(t, name, dtypes=None, shape=None):
    _dev(t, name, dtypes, shape)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


_FLOAT = (torch.float32, torch.float16, torch.bfloat16)


def _on(stream, device):
    """A context in which new tensors belong to `stream` (None: to the current one). The
    allocator orders a block by the stream that is current at its allocation; one that was
    freed on another stream may still be in use by what is queued on that one."""
    if stream is None:
        return contextlib.nullcontext()
    return torch.cuda.stream(torch.cuda.ExternalStream(stream, device) if isinstance(stream, int)
                             else stream)


def _scratch(workspace, need, device, stream):
    """The caller's workspace, or one of `need` bytes that belongs to the call's stream;
    returns (tensor, address, bytes). The tensor has to live until the call is launched:
    freed before, its memory could go to another call at once."""
    if workspace is None:
        if need <= 0:
            return None, 0, 0
        if stream is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=device)
        else:
            with _on(stream, device):
                workspace = torch.empty(need, dtype=torch.uint8, device=device)
    else:
        _dense(workspace, "workspace", (torch.uint8,))
        if workspace.device != device:
            raise ValueError(f"workspace is on {workspace.device}, the call on {device}")
    return workspace, workspace.data_ptr(), workspace.numel()


def _result(shape, dtype, device, stream):
    """A new tensor that a call on `stream` writes and its caller may read on the current
    stream: it belongs to the first, and its free waits for the second."""
    with _on(stream, device):
        t = torch.empty(shape, dtype=dtype, device=device)
    if stream is not None:
        t.record_stream(torch.cuda.current_stream(device))
    return t


def _state_geometry(state, nheads, dim, dstate):
    """state: [rows, nheads, dim, dstate] with dense rows; stride(0) may be padded."""
    _dev(state, "state", _FLOAT)
    _need(state.dim() == 4 and tuple(state.shape[1:]) == (nheads, dim, dstate),
          f"state has shape {tuple(state.shape)}, expected [rows, {nheads}, {dim}, {dstate}]")
    st = state.stride()
    _need(st[3] == 1 and st[2] == dstate and st[1] == dim * dstate,
          "state rows must be dense ([nheads, dim, dstate] contiguous)")
    _need(st[0] >= nheads * dim * dstate or state.shape[0] == 1, "state row stride too small")
    stride = st[0] if state.shape[0] > 1 else nheads * dim * dstate
    return state.shape[0], stride


def _dims(batch, nheads, dim, dstate, ngroups, pool_rows, row_stride, state_dtype,
          io_dtype, bc_dtype):
    return ssu_dims(batch, nheads, dim, dstate, ngroups, pool_rows, row_stride,
                    _DT[state_dtype], _DT[io_dtype], _DT[bc_dtype], 0)


def _opt_idx(t, name, n):
    if t is None:
        return None
    return _dense(t, name, (torch.int32,), (n,))


def ssu_decode(x, A, B, C, dt, state, out, *, dt_bias=None, D=None, z=None,
               dt_softplus=True, state_indices=None, stream=None):
    """One decode step; updates `state` in place and writes `out`.

    x, z, out [batch, nheads, dim]; A, dt_bias, D [nheads] fp32; dt [batch, nheads] fp32;
    B, C [batch, ngroups, dstate]; state [rows, nheads, dim, dstate];
    state_indices [batch] int32 (negative = padding row).
    """
    lib = load_library()
    _dense(x, "x", _FLOAT)
    _need(x.dim() == 3, "x must be [batch, nheads, dim]")
    batch, nheads, dim = x.shape
    _dense(B, "B", _FLOAT)
    _need(B.dim() == 3 and B.shape[0] == batch, "B must be [batch, ngroups, dstate]")
    ngroups, dstate = B.shape[1], B.shape[2]
    _dense(C, "C", (B.dtype,), B.shape)
    _dense(A, "A", (torch.float32,), (nheads,))
    _dense(dt, "dt", (torch.float32,), (batch, nheads))
    if dt_bias is not None:
        _dense(dt_bias, "dt_bias", (torch.float32,), (nheads,))
    if D is not None:
        _dense(D, "D", (torch.float32,), (nheads,))
    if z is not None:
        _dense(z, "z", (x.dtype,), x.shape)
    _dense(out, "out", (x.dtype,), x.shape)
    rows, stride = _state_geometry(state, nheads, dim, dstate)
    _opt_idx(state_indices, "state_indices", batch)
    d = _dims(batch, nheads, dim, dstate, ngroups, rows, stride, state.dtype, x.dtype, B.dtype)
    with torch.cuda.device(x.device):
        _check(lib.ssu_decode(ctypes.byref(d), _ptr(x), _ptr(A), _ptr(B), _ptr(C), _ptr(dt),
                              _ptr(dt_bias), _ptr(D), _ptr(z), _ptr(state), _ptr(out),
                              1 if dt_softplus else 0, _ptr(state_indices),
                              _stream(x.device, stream)))
    return out


def ssu_prefill(x, A, B, C, dt, state, out, *, dt_bias=None, D=None, z=None,
                dt_softplus=True, context_lengths=None, state_indices=None,
                replay_dA=None, replay_u=None, replay_B=None, replay_dt=None, stream=None):
    """All seq_len tokens in one launch.

    x, z, out [batch, seq_len, nheads, dim]; dt [batch, seq_len, nheads];
    B, C [batch, seq_len, ngroups, dstate]; context_lengths [batch] int32.
    Replay stash (fp32, all four or none): replay_dA, replay_dt [batch, seq_len, nheads],
    replay_u [batch, seq_len, nheads, dim], replay_B [batch, seq_len, ngroups, dstate].
    """
    lib = load_library()
    _dense(x, "x", _FLOAT)
    _need(x.dim() == 4, "x must be [batch, seq_len, nheads, dim]")
    batch, seq_len, nheads, dim = x.shape
    _dense(B, "B", _FLOAT)
    _need(B.dim() == 4 and tuple(B.shape[:2]) == (batch, seq_len),
          "B must be [batch, seq_len, ngroups, dstate]")
    ngroups, dstate = B.shape[2], B.shape[3]
    _dense(C, "C", (B.dtype,), B.shape)
    _dense(A, "A", (torch.float32,), (nheads,))
    _dense(dt, "dt", (torch.float32,), (batch, seq_len, nheads))
    if dt_bias is not None:
        _dense(dt_bias, "dt_bias", (torch.float32,), (nheads,))
    if D is not None:
        _dense(D, "D", (torch.float32,), (nheads,))
    if z is not None:
        _dense(z, "z", (x.dtype,), x.shape)
    _dense(out, "out", (x.dtype,), x.shape)
    rows, stride = _state_geometry(state, nheads, dim, dstate)
    _opt_idx(state_indices, "state_indices", batch)
    _opt_idx(context_lengths, "context_lengths", batch)
    stash = (replay_dA, replay_u, replay_B, replay_dt)
    if any(s is not None for s in stash):
        _dense(replay_dA, "replay_dA", (torch.float32,), (batch, seq_len, nheads))
        _dense(replay_dt, "replay_dt", (torch.float32,), (batch, seq_len, nheads))
        _dense(replay_u, "replay_u", (torch.float32,), x.shape)
        _dense(replay_B, "replay_B", (torch.float32,), B.shape)
    d = _dims(batch, nheads, dim, dstate, ngroups, rows, stride, state.dtype, x.dtype, B.dtype)
    with torch.cuda.device(x.device):
        _check(lib.ssu_prefill(ctypes.byref(d), seq_len, _ptr(x), _ptr(A), _ptr(B), _ptr(C),
                               _ptr(dt), _ptr(dt_bias), _ptr(D), _ptr(z), _ptr(state),
                               _ptr(out), 1 if dt_softplus else 0, _ptr(context_lengths),
                               _ptr(state_indices), *[_ptr(s) for s in stash],
                               _stream(x.device, stream)))
    return out


def ssu_replay(state, replay_dA, replay_u, replay_B, replay_dt, accepted_lengths, *,
               state_indices=None, active_batch=None, accepted_node_ids=None, stream=None):
    """Apply accepted stashed tokens to the state, in place.

    replay_dA, replay_dt [batch, seq_len, nheads]; replay_u [batch, seq_len, nheads, dim];
    replay_B [batch, seq_len, ngroups, dstate]; accepted_lengths, state_indices [batch] int32.
    accepted_node_ids [batch, max_accept_len] int32: token t of row b is stash entry
    accepted_node_ids[b, t] (default: entry t). Rows b >= active_batch (default batch)
    are never read.
    """
    lib = load_library()
    _dense(replay_dA, "replay_dA", (torch.float32,))
    _need(replay_dA.dim() == 3, "replay_dA must be [batch, seq_len, nheads]")
    batch, seq_len, nheads = replay_dA.shape
    _dense(replay_u, "replay_u", (torch.float32,))
    _need(replay_u.dim() == 4 and tuple(replay_u.shape[:3]) == (batch, seq_len, nheads),
          "replay_u must be [batch, seq_len, nheads, dim]")
    dim = replay_u.shape[3]
    _dense(replay_B, "replay_B", (torch.float32,))
    _need(replay_B.dim() == 4 and tuple(replay_B.shape[:2]) == (batch, seq_len),
          "replay_B must be [batch, seq_len, ngroups, dstate]")
    ngroups, dstate = replay_B.shape[2], replay_B.shape[3]
    _dense(replay_dt, "replay_dt", (torch.float32,), (batch, seq_len, nheads))
    _dense(accepted_lengths, "accepted_lengths", (torch.int32,), (batch,))
    _opt_idx(state_indices, "state_indices", batch)
    max_accept = 0
    if accepted_node_ids is not None:
        _dense(accepted_node_ids, "accepted_node_ids", (torch.int32,))
        _need(accepted_node_ids.dim() == 2 and accepted_node_ids.shape[0] == batch,
              "accepted_node_ids must be [batch, max_accept_len]")
        max_accept = accepted_node_ids.shape[1]
    rows, stride = _state_geometry(state, nheads, dim, dstate)
    if active_batch is None:
        active_batch = batch
    d = _dims(batch, nheads, dim, dstate, ngroups, rows, stride, state.dtype, torch.float32,
              torch.float32)
    with torch.cuda.device(state.device):
        _check(lib.ssu_replay(ctypes.byref(d), seq_len, _ptr(state), _ptr(replay_dA),
                              _ptr(replay_u), _ptr(replay_B), _ptr(replay_dt),
                              _ptr(accepted_lengths), _ptr(state_indices), int(active_batch),
                              _ptr(accepted_node_ids), int(max_accept),
                              _stream(state.device, stream)))


def _tree_dims(x, A, B, C, dt, state, out, parent_ids, depths, dt_bias, D, z, state_indices,
               stash):
    """Shape checks of a tree-verify call; returns (dims, num_nodes)."""
    _dense(x, "x", _FLOAT)
    _need(x.dim() == 4, "x must be [batch, num_nodes, nheads, dim]")
    batch, num_nodes, nheads, dim = x.shape
    _dense(B, "B", _FLOAT)
    _need(B.dim() == 4 and tuple(B.shape[:2]) == (batch, num_nodes),
          "B must be [batch, num_nodes, ngroups, dstate]")
    ngroups, dstate = B.shape[2], B.shape[3]
    _dense(C, "C", (B.dtype,), B.shape)
    _dense(A, "A", (torch.float32,), (nheads,))
    _dense(dt, "dt", (torch.float32,), (batch, num_nodes, nheads))
    _dense(parent_ids, "parent_ids", (torch.int32,), (batch, num_nodes))
    if depths is not None:
        _dense(depths, "depths", (torch.int32,), (batch, num_nodes))
    if dt_bias is not None:
        _dense(dt_bias, "dt_bias", (torch.float32,), (nheads,))
    if D is not None:
        _dense(D, "D", (torch.float32,), (nheads,))
    if z is not None:
        _dense(z, "z", (x.dtype,), x.shape)
    _dense(out, "out", (x.dtype,), x.shape)
    rows, stride = _state_geometry(state, nheads, dim, dstate)
    _opt_idx(state_indices, "state_indices", batch)
    replay_dA, replay_u, replay_B, replay_dt = stash
    if any(s is not None for s in stash):
        _dense(replay_dA, "replay_dA", (torch.float32,), (batch, num_nodes, nheads))
        _dense(replay_dt, "replay_dt", (torch.float32,), (batch, num_nodes, nheads))
        _dense(replay_u, "replay_u", (torch.float32,), x.shape)
        _dense(replay_B, "replay_B", (torch.float32,), B.shape)
    return _dims(batch, nheads, dim, dstate, ngroups, rows, stride, state.dtype, x.dtype,
                 B.dtype), num_nodes


def ssu_tree_verify(x, A, B, C, dt, state, out, parent_ids, *, depths=None, dt_bias=None,
                    D=None, z=None, dt_softplus=True, state_indices=None, replay_dA=None,
                    replay_u=None, replay_B=None, replay_dt=None, workspace=None, stream=None):
    """Every node of a draft tree per batch row, from the read-only committed state.

    x, z, out [batch, num_nodes, nheads, dim]; dt [batch, num_nodes, nheads];
    B, C [batch, num_nodes, ngroups, dstate]; parent_ids, depths [batch, num_nodes] int32.
    Replay stash (fp32, all four or none) in the ssu_prefill layouts with the node axis.
    workspace: a uint8 GPU tensor of at least tree_workspace_bytes(...) bytes (allocated
    here when None).
    """
    lib = load_library()
    stash = (replay_dA, replay_u, replay_B, replay_dt)
    d, num_nodes = _tree_dims(x, A, B, C, dt, state, out, parent_ids, depths, dt_bias, D, z,
                              state_indices, stash)
    need = max(int(lib.ssu_tree_workspace_bytes(ctypes.byref(d), num_nodes)), 16)
    workspace, wp, wn = _scratch(workspace, need, x.device, stream)
    with torch.cuda.device(x.device):
        _check(lib.ssu_tree_verify(ctypes.byref(d), num_nodes, _ptr(x), _ptr(A), _ptr(B),
                                   _ptr(C), _ptr(dt), _ptr(dt_bias), _ptr(D), _ptr(z),
                                   _ptr(state), _ptr(out), 1 if dt_softplus else 0,
                                   _ptr(state_indices), _ptr(parent_ids), _ptr(depths),
                                   *[_ptr(s) for s in stash], wp, wn,
                                   _stream(x.device, stream)))
    return out


def ssu_tree_verify_noalloc(x, A, B, C, dt, state, out, parent_ids, *, depths=None,
                            dt_bias=None, D=None, z=None, dt_softplus=True, state_indices=None,
                            replay_dA=None, replay_u=None, replay_B=None, replay_dt=None,
                            stream=None):
    """ssu_tree_verify without a workspace: the library's per-GPU scratch of
    SSU_TREE_SCRATCH_BYTES holds the B.C dots, so nothing is allocated (for
    code under graph capture). Calls that overlap on one GPU race on it."""
    lib = load_library()
    stash = (replay_dA, replay_u, replay_B, replay_dt)
    d, num_nodes = _tree_dims(x, A, B, C, dt, state, out, parent_ids, depths, dt_bias, D, z,
                              state_indices, stash)
    with torch.cuda.device(x.device):
        _check(lib.ssu_tree_verify_noalloc(ctypes.byref(d), num_nodes, _ptr(x), _ptr(A), _ptr(B),
                                           _ptr(C), _ptr(dt), _ptr(dt_bias), _ptr(D), _ptr(z),
                                           _ptr(state), _ptr(out), 1 if dt_softplus else 0,
                                           _ptr(state_indices), _ptr(parent_ids), _ptr(depths),
                                           *[_ptr(s) for s in stash], _stream(x.device, stream)))
    return out


TREE_SCRATCH_BYTES = 4194304  # SSU_TREE_SCRATCH_BYTES of include/ssu.h


def tree_workspace_bytes(batch, ngroups, num_nodes):
    """Bytes of the workspace ssu_tree_verify needs (no GPU needed)."""
    return 4 * batch * ngroups * num_nodes * num_nodes


def _device_table(structs, device):
    """Pack ctypes structs into one device buffer (a uint8 tensor)."""
    n = len(structs)
    size = ctypes.sizeof(structs[0]) if n else 0
    raw = bytearray(size * n)
    for i, st in enumerate(structs):
        ctypes.memmove((ctypes.c_char * size).from_buffer(raw, i * size), ctypes.addressof(st), size)
    host = torch.frombuffer(raw, dtype=torch.uint8) if n else torch.empty(0, dtype=torch.uint8)
    return host.to(device)


class ReplayLayerTable:
    """Device array of per-layer replay buffers for ssu_replay_layers.

    states[i] [rows, nheads, dim, dstate]; dAs[i], dts[i] [batch, seq_len, nheads];
    us[i] [batch, seq_len, nheads, dim]; Bs[i] [batch, seq_len, ngroups, dstate] (fp32).
    Every layer has the same shapes and dtypes. Keeps the tensors alive."""

    def __init__(self, states, dAs, us, Bs, dts):
        n = len(states)
        _need(n > 0 and all(len(v) == n for v in (dAs, us, Bs, dts)), "one entry per layer")
        s0, a0, u0, b0 = states[0], dAs[0], us[0], Bs[0]
        for i in range(n):
            _need(states[i].dtype == s0.dtype and states[i].shape == s0.shape and
                  states[i].stride() == s0.stride(), "every layer's state has the same geometry")
            _dense(dAs[i], "replay_dA", (torch.float32,), a0.shape)
            _dense(dts[i], "replay_dt", (torch.float32,), a0.shape)
            _dense(us[i], "replay_u", (torch.float32,), u0.shape)
            _dense(Bs[i], "replay_B", (torch.float32,), b0.shape)
        _need(a0.dim() == 3 and u0.dim() == 4 and b0.dim() == 4, "stash shapes")
        self.batch, self.seq_len, self.nheads = a0.shape
        self.dim = u0.shape[3]
        self.ngroups, self.dstate = b0.shape[2], b0.shape[3]
        self.rows, self.stride = _state_geometry(s0, self.nheads, self.dim, self.dstate)
        self.state_dtype = s0.dtype
        self.keep = (states, dAs, us, Bs, dts)
        self.num_layers = n
        self.device = s0.device
        self.table = _device_table([ssu_replay_layer(states[i].data_ptr(), dAs[i].data_ptr(),
                                                     us[i].data_ptr(), Bs[i].data_ptr(),
                                                     dts[i].data_ptr()) for i in range(n)],
                                   self.device)


def ssu_replay_layers(table: ReplayLayerTable, accepted_lengths, *, state_indices=None,
                      active_batch=None, accepted_node_ids=None, stream=None):
    """ssu_replay for every layer of `table` in one launch (shared accepted
    lengths, state indices and node ids)."""
    lib = load_library()
    _dense(accepted_lengths, "accepted_lengths", (torch.int32,), (table.batch,))
    _opt_idx(state_indices, "state_indices", table.batch)
    max_accept = 0
    if accepted_node_ids is not None:
        _dense(accepted_node_ids, "accepted_node_ids", (torch.int32,))
        _need(accepted_node_ids.dim() == 2 and accepted_node_ids.shape[0] == table.batch,
              "accepted_node_ids must be [batch, max_accept_len]")
        max_accept = accepted_node_ids.shape[1]
    if active_batch is None:
        active_batch = table.batch
    d = _dims(table.batch, table.nheads, table.dim, table.dstate, table.ngroups, table.rows,
              table.stride, table.state_dtype, torch.float32, torch.float32)
    with torch.cuda.device(table.device):
        _check(lib.ssu_replay_layers(ctypes.byref(d), table.seq_len, _ptr(table.table),
                                     table.num_layers, _ptr(accepted_lengths),
                                     _ptr(state_indices), int(active_batch),
                                     _ptr(accepted_node_ids), int(max_accept),
                                     _stream(table.device, stream)))


class StateLayerTable:
    """Device array of per-layer {recurrent, conv} state buffers for
    ssu_state_clear_layers. Entries may be None (that buffer is skipped)."""

    def __init__(self, recurrent, conv):
        _need(len(recurrent) == len(conv) and len(recurrent) > 0, "one entry per layer")
        self.keep = (recurrent, conv)
        self.num_layers = len(recurrent)
        dev = next(t.device for t in list(recurrent) + list(conv) if t is not None)
        self.device = dev
        self.table = _device_table([ssu_state_layer(0 if r is None else r.data_ptr(),
                                                    0 if c is None else c.data_ptr())
                                    for r, c in zip(recurrent, conv)], dev)


def ssu_state_clear_layers(table: StateLayerTable, resident_rows, slot, recurrent_row_bytes,
                           conv_row_bytes, stream=None):
    """Zero row `slot` (or every row, slot -1) of both states of every layer."""
    lib = load_library()
    with torch.cuda.device(table.device):
        _check(lib.ssu_state_clear_layers(_ptr(table.table), table.num_layers, int(resident_rows),
                                          int(slot), int(recurrent_row_bytes),
                                          int(conv_row_bytes), _stream(table.device, stream)))


def _rows(t, name):
    """(rows, row_bytes, row stride in bytes) of a tensor whose leading dim is the row."""
    _dev(t, name)
    _need(t.dim() >= 1, f"{name} needs a leading row dimension")
    inner = t[0] if t.shape[0] > 0 else t.new_empty(t.shape[1:])
    _need(inner.is_contiguous(), f"{name} rows must be dense")
    row_bytes = inner.numel() * t.element_size()
    stride = t.stride(0) * t.element_size() if t.shape[0] > 1 else row_bytes
    return t.shape[0], row_bytes, stride


def ssu_state_gather(resident, active, state_indices, stream=None):
    """active[b] = resident[state_indices[b]]; a negative index gives a zero row."""
    lib = load_library()
    rr, rb, rs = _rows(resident, "resident")
    ar, ab, ast = _rows(active, "active")
    _need(rb == ab and resident.dtype == active.dtype, "resident and active rows must match")
    _dense(state_indices, "state_indices", (torch.int32,), (ar,))
    with torch.cuda.device(active.device):
        _check(lib.ssu_state_gather(_ptr(resident), rr, rs, _ptr(active), ast,
                                    _ptr(state_indices), ar, rb, _stream(active.device, stream)))


def ssu_state_scatter(active, resident, state_indices, stream=None):
    """resident[state_indices[b]] = active[b] for non-negative indices."""
    lib = load_library()
    rr, rb, rs = _rows(resident, "resident")
    ar, ab, ast = _rows(active, "active")
    _need(rb == ab and resident.dtype == active.dtype, "resident and active rows must match")
    _dense(state_indices, "state_indices", (torch.int32,), (ar,))
    with torch.cuda.device(active.device):
        _check(lib.ssu_state_scatter(_ptr(active), ast, _ptr(resident), rr, rs,
                                     _ptr(state_indices), ar, rb, _stream(active.device, stream)))


def pack_workspace_bytes(pool, batch, n_bystanders):
    """Bytes of the workspace ssu_state_pack / ssu_state_unpack need (pool: any
    tensor whose leading dimension is the row)."""
    row_bytes = int(torch.Size(pool.shape[1:]).numel()) * pool.element_size()
    return (batch + n_bystanders) * row_bytes


def _pack_call(fn, pool, homes, bystanders, workspace, stream):
    lib = load_library()
    rows, rb, rs = _rows(pool, "pool")
    _dense(homes, "homes", (torch.int32,))
    _need(homes.dim() == 1, "homes must be 1-D")
    nb = 0
    if bystanders is not None:
        _dense(bystanders, "bystanders", (torch.int32,))
        nb = bystanders.numel()
    _dev(workspace, "workspace")
    _need(workspace.numel() * workspace.element_size() >= (homes.numel() + nb) * rb,
          "workspace too small")
    with torch.cuda.device(pool.device):
        _check(getattr(lib, fn)(_ptr(pool), rows, rs, rb, _ptr(homes), homes.numel(),
                                _ptr(bystanders) if nb else None, nb, _ptr(workspace),
                                _stream(pool.device, stream)))


def ssu_state_pack(pool, homes, workspace, bystanders=None, stream=None):
    """Slots [0, len(homes)) of `pool` get the rows homes[b] held (all read first);
    bystander rows are saved in `workspace` for ssu_state_unpack."""
    _pack_call("ssu_state_pack", pool, homes, bystanders, workspace, stream)


def ssu_state_unpack(pool, homes, workspace, bystanders=None, stream=None):
    """Slots [0, len(homes)) go back to their homes; bystanders are restored."""
    _pack_call("ssu_state_unpack", pool, homes, bystanders, workspace, stream)


def ssu_gdn_decode(hidden_states, w_ba, mixed_qkv, conv_weight, conv_bias, conv_state, A_log,
                   dt_bias, scale, ssm_state, state_indices, *, num_q_heads, use_qk_l2norm=True,
                   out=None, workspace=None, stream=None):
    """Fused gated-delta-rule decode step (one token per batch entry) over paged
    conv / ssm pools, both updated in place. conv_state: a [P, qkv_dim, W-1]
    view of any strides (a dense pool, or the transposed view of a
    [P, W-1, qkv_dim] pool). workspace: a uint8 GPU tensor of at least
    gdn_workspace_bytes(...) bytes (allocated here when None). Returns
    out [B, 1, HV, D] (bf16)."""
    lib = load_library()
    bf = (torch.bfloat16,)
    _dense(hidden_states, "hidden_states", bf)
    B, hidden = hidden_states.shape
    _dense(w_ba, "w_ba", bf)
    _need(w_ba.dim() == 2 and w_ba.shape[0] == hidden and w_ba.shape[1] % 2 == 0,
          "w_ba must be [hidden, 2*HV]")
    hv = w_ba.shape[1] // 2
    hq = int(num_q_heads)
    _need(hq > 0 and hv % hq == 0, "num_v_heads must be a multiple of num_q_heads")
    _dense(conv_weight, "conv_weight", bf)
    qkv, width = conv_weight.shape
    _need(qkv % (2 * hq + hv) == 0, "qkv_dim must be (2*Hq + HV)*D")
    d = qkv // (2 * hq + hv)
    _dense(mixed_qkv, "mixed_qkv", bf, (B, qkv))
    _dense(conv_bias, "conv_bias", bf, (qkv,))
    _dev(conv_state, "conv_state", bf)
    _need(conv_state.dim() == 3 and tuple(conv_state.shape[1:]) == (qkv, width - 1),
          "conv_state must be a [P, qkv_dim, W-1] view")
    _dense(A_log, "A_log", (torch.float32,), (hv,))
    _dense(dt_bias, "dt_bias", bf, (hv,))
    _dev(ssm_state, "ssm_state", (torch.float32,))
    _need(ssm_state.dim() == 4 and tuple(ssm_state.shape[1:]) == (hv, d, d),
          "ssm_state must be [P, HV, D, D]")
    st = ssm_state.stride()
    _need(st[3] == 1 and st[2] == d and st[1] == d * d, "ssm_state rows must be dense")
    _need(ssm_state.shape[0] == conv_state.shape[0], "both pools have the same slots")
    _dense(state_indices, "state_indices", (torch.int32,), (B,))
    if out is None:
        out = _result((B, 1, hv, d), torch.bfloat16, hidden_states.device, stream)
    _dense(out, "out", bf, (B, 1, hv, d))
    cs = conv_state.stride()
    dims = ssu_gdn_dims(B, hidden, hq, hv, d, width, ssm_state.shape[0],
                        1 if use_qk_l2norm else 0,
                        st[0] if ssm_state.shape[0] > 1 else hv * d * d, cs[0], cs[1], cs[2])
    sc = 0.0 if scale is None else float(scale)
    need = int(lib.ssu_gdn_workspace_bytes(ctypes.byref(dims)))
    workspace, wp, wn = _scratch(workspace, max(need, 16), hidden_states.device, stream)
    with torch.cuda.device(hidden_states.device):
        _check(lib.ssu_gdn_decode(ctypes.byref(dims), _ptr(hidden_states), _ptr(w_ba),
                                  _ptr(mixed_qkv), _ptr(conv_weight), _ptr(conv_bias),
                                  _ptr(conv_state), _ptr(A_log), _ptr(dt_bias), sc,
                                  _ptr(ssm_state), _ptr(state_indices), _ptr(out),
                                  wp, wn, _stream(hidden_states.device, stream)))
    return out


def gdn_workspace_bytes(batch, hidden, num_q_heads, num_v_heads, head_dim):
    """Bytes of the workspace ssu_gdn_decode needs (no GPU needed)."""
    d = ssu_gdn_dims(batch, hidden, num_q_heads, num_v_heads, head_dim, 1, 1, 1, 0, 0, 0, 0)
    return int(load_library().ssu_gdn_workspace_bytes(ctypes.byref(d)))


# ---------------------------------------------------------------------------
# Per-channel scan, causal convolution, draft verification
# ---------------------------------------------------------------------------
def _fail(msg):
    raise ValueError(msg)


_DENSE = (0, 0)


def _outer(stride, shape, name, step):
    """(batch stride, token stride) of an activation [batch, (tokens,) *row] for the
    C call, 0 where the axis has one entry; rows must be dense and not broadcast, either
    outer axis may lie outside the other (the C call refuses strides that could overlap)."""
    n = len(shape)
    row = 1 if step else 2
    if stride[-1] != 1 and shape[-1] > 1:
        _fail(f"{name} must be dense in its last axes")
    if n > row + 1 and stride[-2] != shape[-1] and shape[-2] > 1:
        _fail(f"{name} must be dense in its last axes")
    bs, ts = stride[0], 0
    if shape[0] <= 1:
        bs = 0
    elif bs <= 0:
        _fail(f"{name} must not be broadcast over the batch")
    if not step and shape[1] > 1:
        ts = stride[1]
        if ts <= 0:
            _fail(f"{name} must not be broadcast over the tokens")
    return bs, ts


def _bad(t, name, kind, dtype, shape, dev):
    _fail(f"{name}: expected a {kind}{dtype} tensor {tuple(shape)} on cuda:{dev}, got {t.dtype} "
          f"{tuple(t.shape)} on {t.device}")


def _view(t, name, dtype, shape, dev, step):
    """_outer of an activation after its checks ((0, 0) where it is contiguous)."""
    if t.get_device() != dev or t.dtype is not dtype or t.shape != shape:
        _bad(t, name, "", dtype, shape, dev)
    return _DENSE if t.is_contiguous() else _outer(t.stride(), shape, name, step)


def _vector(t, name, dtype, shape, dev):
    """Address of a dense tensor after its checks (0 where there is none)."""
    if t is None:
        return 0
    if (t.get_device() != dev or t.dtype is not dtype or t.shape != shape
            or not t.is_contiguous()):
        _bad(t, name, "contiguous ", dtype, shape, dev)
    return t.data_ptr()


def _first(t, name, dims, what):
    """Device index of a call's first tensor after its checks."""
    if not t.is_cuda:
        _fail(f"{name} must be a GPU tensor")
    if t.dtype not in _FLOAT or t.dim() != dims:
        _fail(f"{name} must be {what}, fp32, fp16 or bf16")
    if max(t.shape) > 1 << 30:
        _fail(f"{name} has an axis above 2^30")
    return t.get_device()


def _launch(dev, stream, fn, *args):
    """fn(*args, stream) with device `dev` current; a failure raises."""
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(dev)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    if torch.cuda.current_device() == dev:
        rc = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, stream)
    if rc != SSU_OK:
        _check(rc)


def _conv_call(x, weight, bias, conv_state, out, silu, update_state, context_lengths,
               state_indices, stream, step):
    lib = _LIB or load_library()
    dev = _first(x, "x", 2 if step else 3, "[batch, channels]" if step else
                 "[batch, seq_len, channels]")
    shape, dtype = x.shape, x.dtype
    batch, channels = shape[0], shape[-1]
    xs = _DENSE if x.is_contiguous() else _outer(x.stride(), shape, "x", step)
    os_ = _DENSE if out is None else _view(out, "out", dtype, shape, dev, step)
    if weight.dim() != 2 or weight.shape[0] != channels or weight.dtype not in _FLOAT:
        _fail("weight must be [channels, width], fp32, fp16 or bf16")
    wdt = weight.dtype
    width = weight.shape[1]
    wp = _vector(weight, "weight", wdt, weight.shape, dev)
    bp = _vector(bias, "bias", wdt, (channels,), dev)
    if conv_state is not None:
        sdt, rows, ss, sp = (conv_state.dtype, conv_state.shape[0], conv_state.stride(),
                             conv_state.data_ptr())
        if (conv_state.get_device() != dev or conv_state.dim() != 3 or sdt not in _FLOAT
                or conv_state.shape[1] != channels or conv_state.shape[2] != width - 1):
            _fail(f"conv_state must be a [rows, {channels}, {width - 1}] view on cuda:{dev}")
        if rows > 1 << 30:
            _fail("conv_state has more than 2^30 rows")
        if width > 1 and ((ss[0] <= 0 and rows > 1) or (ss[1] <= 0 and channels > 1)
                          or (ss[2] <= 0 and width > 2)):
            _fail("conv_state must not be broadcast")
    else:
        if width != 1:
            _fail("conv_state is required")
        rows, sdt, ss, sp = max(batch, 1), dtype, (0, 0, 0), 0
    ip = _vector(state_indices, "state_indices", torch.int32, (batch,), dev)
    d = ssu_conv_dims(batch, channels, width, rows, _DT[dtype], _DT[wdt], _DT[sdt], 0, *xs, *os_,
                      *ss)
    op = 0 if out is None else out.data_ptr()
    if step:
        _launch(dev, stream, lib.ssu_conv_decode, d, x.data_ptr(), wp, bp, sp, op,
                1 if silu else 0, ip)
    else:
        cp = _vector(context_lengths, "context_lengths", torch.int32, (batch,), dev)
        _launch(dev, stream, lib.ssu_conv_prefill, d, shape[1], x.data_ptr(), wp, bp, sp, op,
                1 if silu else 0, 1 if update_state else 0, cp, ip)
    return out


def ssu_conv_prefill(x, weight, bias, conv_state, out, *, silu=True, context_lengths=None,
                     state_indices=None, update_state=True, stream=None):
    """Causal convolution of seq_len tokens, the last width-1 inputs kept in a pool.

    x, out [batch, seq_len, channels] (slices of wider tensors are fine: channels dense,
    the other two axes in either order); weight [channels, width]; bias [channels] or None; conv_state
    [rows, channels, width-1], its axes in any order, updated in place unless update_state is False;
    context_lengths, state_indices [batch] int32. out may be None when only the state is
    wanted (commit of a window: context_lengths = accepted lengths).
    """
    return _conv_call(x, weight, bias, conv_state, out, silu, update_state, context_lengths,
                      state_indices, stream, False)


def ssu_conv_decode(x, weight, bias, conv_state, out, *, silu=True, state_indices=None,
                    stream=None):
    """The causal convolution of one token: x, out [batch, channels]; the rest as
    ssu_conv_prefill. out may be x."""
    return _conv_call(x, weight, bias, conv_state, out, silu, True, None, state_indices, stream,
                      True)


def _scan_call(x, A, B, C, dt, state, out, dt_bias, D, z, dt_softplus, update_state,
               context_lengths, state_indices, workspace, stream, step):
    lib = _LIB or load_library()
    dev = _first(x, "x", 2 if step else 3, "[batch, dim]" if step else "[batch, seq_len, dim]")
    shape, dtype = x.shape, x.dtype
    batch, dim = shape[0], shape[-1]
    bshape, bdt, ddt, sdt = B.shape, B.dtype, dt.dtype, state.dtype
    if bdt not in _FLOAT or ddt not in _FLOAT or sdt not in _FLOAT:
        _fail("B, C, dt and state are fp32, fp16 or bf16")
    if len(bshape) != len(shape) + 1 or bshape[:-2] != shape[:-1]:
        _fail("B must be [batch, ngroups, dstate]" if step else
              "B must be [batch, seq_len, ngroups, dstate]")
    ngroups, dstate = bshape[-2], bshape[-1]
    xs = _DENSE if x.is_contiguous() else _outer(x.stride(), shape, "x", step)
    ds = _view(dt, "dt", ddt, shape, dev, step)
    bs = _view(B, "B", bdt, bshape, dev, step)
    cs = zs = os_ = _DENSE
    cp = zp = op = 0
    if C is not None:
        cs, cp = _view(C, "C", bdt, bshape, dev, step), C.data_ptr()
    if z is not None:
        zs, zp = _view(z, "z", dtype, shape, dev, step), z.data_ptr()
    if out is not None:
        if C is None:
            _fail("C is required")
        os_, op = _view(out, "out", dtype, shape, dev, step), out.data_ptr()
    f32 = torch.float32
    ap = _vector(A, "A", f32, (dim, dstate), dev)
    hp = _vector(dt_bias, "dt_bias", f32, (dim,), dev)
    kp = _vector(D, "D", f32, (dim,), dev)
    sshape, st = state.shape, state.stride()
    if (state.get_device() != dev or len(sshape) != 3 or sshape[1] != dim or sshape[2] != dstate):
        _fail(f"state must be [rows, {dim}, {dstate}] on cuda:{dev}, got {tuple(sshape)} on "
              f"{state.device}")
    rows = sshape[0]
    if (st[2] != 1 and dstate > 1) or (st[1] != dstate and dim > 1):
        _fail("state rows must be dense ([dim, dstate] contiguous)")
    if rows > 1 and st[0] < dim * dstate:
        _fail("state row stride too small")
    if rows > 1 << 30:
        _fail("state has more than 2^30 rows")
    ip = _vector(state_indices, "state_indices", torch.int32, (batch,), dev)
    d = ssu_scan_dims(batch, dim, dstate, ngroups, rows, _DT[sdt], _DT[dtype], _DT[ddt], _DT[bdt],
                      0, st[0] if rows > 1 else 0, *xs, *zs, *os_, *ds, *bs, *cs)
    soft = 1 if dt_softplus else 0
    if step:
        _launch(dev, stream, lib.ssu_scan_decode, d, x.data_ptr(), ap, B.data_ptr(), cp,
                dt.data_ptr(), hp, kp, zp, state.data_ptr(), op, soft, ip)
        return out
    lp = _vector(context_lengths, "context_lengths", torch.int32, (batch,), dev)
    workspace, wp, wn = _scratch(workspace, lib.ssu_scan_workspace_bytes(d, shape[1]), x.device, stream)
    _launch(dev, stream, lib.ssu_scan_prefill, d, shape[1], x.data_ptr(), ap, B.data_ptr(), cp,
            dt.data_ptr(), hp, kp, zp, state.data_ptr(), op, soft, 1 if update_state else 0, lp, ip,
            wp, wn)
    return out


def ssu_scan_prefill(x, A, B, C, dt, state, out, *, dt_bias=None, D=None, z=None,
                     dt_softplus=True, context_lengths=None, state_indices=None,
                     update_state=True, workspace=None, stream=None):
    """Per-channel selective scan of seq_len tokens.

    x, z, out, dt [batch, seq_len, dim]; B, C [batch, seq_len, ngroups, dstate] (slices of
    wider tensors are fine: a token's entries dense, the other two axes in either order); A [dim, dstate],
    dt_bias, D [dim] fp32; state [rows, dim, dstate], updated in place unless update_state is
    False; context_lengths, state_indices [batch] int32. out (and C) may be None when only
    the state is wanted (commit of a window: context_lengths = accepted lengths). workspace: a
    uint8 GPU tensor of at least scan_workspace_bytes(...) bytes for this call's sizes
    (allocated here when None).
    """
    return _scan_call(x, A, B, C, dt, state, out, dt_bias, D, z, dt_softplus, update_state,
                      context_lengths, state_indices, workspace, stream, False)


def scan_workspace_bytes(batch, seq_len, dim, dstate, ngroups=1):
    """Bytes of the workspace ssu_scan_prefill needs for exactly these sizes (no GPU needed;
    -1 for sizes that the call refuses). They do not grow with batch or seq_len: a workspace
    for several shapes needs the largest of their sizes, each of them asked for."""
    d = ssu_scan_dims(batch, dim, dstate, ngroups)
    return int(load_library().ssu_scan_workspace_bytes(d, seq_len))


def ssu_scan_decode(x, A, B, C, dt, state, out, *, dt_bias=None, D=None, z=None,
                    dt_softplus=True, state_indices=None, stream=None):
    """One token of the per-channel selective scan: x, z, out, dt [batch, dim]; B, C
    [batch, ngroups, dstate]; the rest as ssu_scan_prefill. out may be x or z."""
    return _scan_call(x, A, B, C, dt, state, out, dt_bias, D, z, dt_softplus, True, None,
                      state_indices, None, stream, True)


def verify_workspace_bytes(batch, vocab):
    """Bytes of the workspace ssu_draft_verify needs (no GPU needed)."""
    d = ssu_verify_dims(batch, 1, vocab, 0, 0, 0, 0, 0, 0, 0)
    return int(load_library().ssu_verify_workspace_bytes(ctypes.byref(d)))


def ssu_draft_verify(tokens, target_probs, uniforms, accepted_lengths, next_tokens, *,
                     draft_probs=None, parent_ids=None, context_lengths=None, state_indices=None,
                     accepted_node_ids=None, workspace=None, stream=None):
    """Which drafted tokens of a verify window stand, and the token drawn after them.

    tokens [batch, num_tokens] int32 (entry 0 certain, the others drafted); target_probs
    [batch, num_tokens, vocab]; uniforms [batch, num_tokens] fp32 in [0, 1) (entry 0 draws the
    next token); draft_probs [batch, num_tokens-1, vocab] (a chain drawn from them), or
    parent_ids [batch, num_tokens] int32 (a draft tree), or neither (a given chain).
    accepted_lengths, next_tokens [batch] int32 and accepted_node_ids [batch, max_accept_len]
    int32 are written: ssu_replay takes the lengths and node ids, the prefill calls take the
    lengths as context_lengths. workspace: a uint8 GPU tensor of at least
    verify_workspace_bytes(batch, vocab) bytes (allocated here when None).
    """
    lib = _LIB or load_library()
    if not tokens.is_cuda:
        _fail("tokens must be a GPU tensor")
    if tokens.dim() != 2:
        _fail("tokens must be [batch, num_tokens]")
    dev, i32, shape, dtype = tokens.get_device(), torch.int32, tokens.shape, target_probs.dtype
    batch, n = shape
    if dtype not in _FLOAT or target_probs.dim() != 3:
        _fail("target_probs must be [batch, num_tokens, vocab], fp32, fp16 or bf16")
    vocab = target_probs.shape[2]
    if vocab > 1 << 24 or batch > 65535:
        _fail(f"vocab {vocab} above 2^24, or batch {batch} above 65535")
    ts = _view(target_probs, "target_probs", dtype, (batch, n, vocab), dev, False)
    ds, qp = _DENSE, 0
    if draft_probs is not None:
        ds = _view(draft_probs, "draft_probs", dtype, (batch, n - 1, vocab), dev, False)
        qp = draft_probs.data_ptr()
        if n == 1:
            qp = 0  # no row
    tp = _vector(tokens, "tokens", i32, shape, dev)
    up = _vector(uniforms, "uniforms", torch.float32, shape, dev)
    pp = _vector(parent_ids, "parent_ids", i32, shape, dev)
    cp = _vector(context_lengths, "context_lengths", i32, (batch,), dev)
    ip = _vector(state_indices, "state_indices", i32, (batch,), dev)
    ap = _vector(accepted_lengths, "accepted_lengths", i32, (batch,), dev)
    np_ = _vector(next_tokens, "next_tokens", i32, (batch,), dev)
    most = kp = 0
    if accepted_node_ids is not None:
        most = accepted_node_ids.shape[-1]
        kp = _vector(accepted_node_ids, "accepted_node_ids", i32, (batch, most), dev)
    d = ssu_verify_dims(batch, n, vocab, most, _DT[dtype], 0, *ts, *ds)
    workspace, wp, wn = _scratch(workspace, max(lib.ssu_verify_workspace_bytes(d), 16), tokens.device,
                                 stream)
    _launch(dev, stream, lib.ssu_draft_verify, d, tp, target_probs.data_ptr(), qp, up, pp, cp, ip,
            ap, kp, np_, wp, wn)
    return accepted_lengths, next_tokens


# ---------------------------------------------------------------------------
# Gated delta rule, RMS norm, log probabilities
# ---------------------------------------------------------------------------
def _delta_call(q, k, v, a, b, state, out, A_log, dt_bias, scale, use_qk_l2norm, update_state,
                context_lengths, state_indices, workspace, stream, step):
    lib = _LIB or load_library()
    dev = _first(v, "v", 3 if step else 4, "[batch, HV, D]" if step else "[batch, seq_len, HV, D]")
    shape, dtype = v.shape, v.dtype
    batch, hv, d = shape[0], shape[-2], shape[-1]
    kshape, gdt, sdt = k.shape, a.dtype, state.dtype
    if len(kshape) != len(shape) or kshape[:-2] != shape[:-2] or kshape[-1] != d:
        _fail("k must be [batch, Hq, D]" if step else "k must be [batch, seq_len, Hq, D]")
    hq = kshape[-2]
    if gdt not in _FLOAT or sdt not in _FLOAT:
        _fail("a, b and state are fp32, fp16 or bf16")
    ks = _view(k, "k", dtype, kshape, dev, step)
    vs = _view(v, "v", dtype, shape, dev, step)
    as_ = _view(a, "a", gdt, shape[:-1], dev, step)
    bs = _view(b, "b", gdt, shape[:-1], dev, step)
    qs = os_ = _DENSE
    qp = op = 0
    if q is not None:
        qs, qp = _view(q, "q", dtype, kshape, dev, step), q.data_ptr()
    if out is not None:
        if q is None:
            _fail("q is required")
        os_, op = _view(out, "out", dtype, shape, dev, step), out.data_ptr()
    ap = _vector(A_log, "A_log", torch.float32, (hv,), dev)
    hdt = torch.float32
    if dt_bias is not None:
        hdt = dt_bias.dtype
        if hdt not in _FLOAT:
            _fail("dt_bias is fp32, fp16 or bf16")
    hp = _vector(dt_bias, "dt_bias", hdt, (hv,), dev)
    sshape, st = state.shape, state.stride()
    if state.device.index != dev or len(sshape) != 4 or tuple(sshape[1:]) != (hv, d, d):
        _fail(f"state must be [rows, {hv}, {d}, {d}] on cuda:{dev}, got {tuple(sshape)} on "
              f"{state.device}")
    rows = sshape[0]
    if st[3] != 1 or st[2] != d or (st[1] != d * d and hv > 1):
        _fail("state rows must be dense ([HV, D, D] contiguous)")
    if rows > 1 and st[0] < hv * d * d:
        _fail("state row stride too small")
    if rows > 1 << 30:
        _fail("state has more than 2^30 rows")
    ip = _vector(state_indices, "state_indices", torch.int32, (batch,), dev)
    dims = ssu_delta_dims(batch, hq, hv, d, rows, 1 if use_qk_l2norm else 0, _DT[sdt], _DT[dtype],
                          _DT[gdt], _DT[hdt], st[0] if rows > 1 else 0, *qs, *ks, *vs, *as_, *bs,
                          *os_)
    sc = 0.0 if scale is None else float(scale)
    if step:
        _launch(dev, stream, lib.ssu_delta_decode, dims, qp, k.data_ptr(), v.data_ptr(),
                a.data_ptr(), b.data_ptr(), ap, hp, sc, state.data_ptr(), op, ip)
        return out
    cp = _vector(context_lengths, "context_lengths", torch.int32, (batch,), dev)
    workspace, wp, wn = _scratch(workspace, lib.ssu_delta_workspace_bytes(dims, shape[1]), v.device,
                                 stream)
    _launch(dev, stream, lib.ssu_delta_prefill, dims, shape[1], qp, k.data_ptr(), v.data_ptr(),
            a.data_ptr(), b.data_ptr(), ap, hp, sc, state.data_ptr(), op, 1 if update_state else 0,
            cp, ip, wp, wn)
    return out


def ssu_delta_prefill(q, k, v, a, b, state, out, *, A_log=None, dt_bias=None, scale=None,
                      use_qk_l2norm=True, context_lengths=None, state_indices=None,
                      update_state=True, workspace=None, stream=None):
    """Gated delta rule of seq_len tokens.

    q, k [batch, seq_len, Hq, D]; v, out [batch, seq_len, HV, D], HV a multiple of Hq; a, b
    [batch, seq_len, HV] (slices of wider tensors are fine: a token's entries dense, the other
    two axes in either order); state [rows, HV, D, D], updated in place unless update_state is
    False; A_log [HV] fp32 and dt_bias [HV] make the decays and betas of a and b as
    ssu_gdn_decode does, without A_log they are the decays' logarithms and the betas;
    context_lengths, state_indices [batch] int32. out (and q) may be None when only the state
    is wanted (commit of a window: context_lengths = accepted lengths). workspace: a uint8 GPU
    tensor of at least delta_workspace_bytes(...) bytes for this call's sizes (allocated here
    when None).
    """
    return _delta_call(q, k, v, a, b, state, out, A_log, dt_bias, scale, use_qk_l2norm,
                       update_state, context_lengths, state_indices, workspace, stream, False)


def ssu_delta_decode(q, k, v, a, b, state, out, *, A_log=None, dt_bias=None, scale=None,
                     use_qk_l2norm=True, state_indices=None, stream=None):
    """One token of the gated delta rule: q, k [batch, Hq, D]; v, out [batch, HV, D]; a, b
    [batch, HV]; the rest as ssu_delta_prefill. out may be v."""
    return _delta_call(q, k, v, a, b, state, out, A_log, dt_bias, scale, use_qk_l2norm, True, None,
                       state_indices, None, stream, True)


def delta_workspace_bytes(batch, seq_len, num_q_heads, num_v_heads, head_dim,
                          dtype=torch.bfloat16):
    """Bytes of the workspace ssu_delta_prefill needs for exactly these sizes and type of q, k
    and v (no GPU needed; -1 for what the call refuses)."""
    d = ssu_delta_dims(batch, num_q_heads, num_v_heads, head_dim, 1, 1, 0, _DT[dtype])
    return int(load_library().ssu_delta_workspace_bytes(d, seq_len))


_E4M3 = torch.float8_e4m3fn


def ssu_rms_norm(x, weight, out, *, residual=None, z=None, scales=None, group_size=None, eps=1e-6,
                 unit_offset=False, gate_first=False, stream=None):
    """RMS norm of the rows of x, over groups of group_size columns (None: whole rows).

    x, z, residual, out [rows, n] or [batch, tokens, n] (slices of wider tensors are fine);
    weight [n] or [group_size]; unit_offset: the factor is 1 + weight. residual is added to x
    first and receives the sum; z gates by silu(z), behind the norm or, with gate_first, before
    it. out in float8_e4m3fn takes scales fp32 [.., m]: each of m blocks of a row is divided by
    its scale, its largest magnitude / 448. out may be x or z.
    """
    lib = _LIB or load_library()
    two = x.dim() == 2
    dev = _first(x, "x", 2 if two else 3, "[rows, n] or [batch, tokens, n]")
    shape, dtype = x.shape, x.dtype
    n = shape[-1]
    xs = _DENSE if x.is_contiguous() else _outer(x.stride(), shape, "x", two)
    zs = rs = _DENSE
    zp = rp = 0
    if z is not None:
        zs, zp = _view(z, "z", dtype, shape, dev, two), z.data_ptr()
    rdt = dtype
    if residual is not None:
        rdt = residual.dtype
        if rdt not in _FLOAT:
            _fail("residual is fp32, fp16 or bf16")
        rs, rp = _view(residual, "residual", rdt, shape, dev, two), residual.data_ptr()
    odt, wdt = out.dtype, weight.dtype
    if odt not in _FLOAT and odt is not _E4M3:
        _fail("out is fp32, fp16, bf16 or float8_e4m3fn")
    os_ = _view(out, "out", odt, shape, dev, two)
    group = n if group_size is None else int(group_size)
    if group <= 0 or n == 0 or n % group:
        _fail(f"group_size {group} does not divide {n} columns")
    if wdt not in _FLOAT or weight.dim() != 1 or weight.shape[0] not in (n, group):
        _fail(f"weight must be [{n}] or [{group}], fp32, fp16 or bf16")
    wp = _vector(weight, "weight", wdt, weight.shape, dev)
    block = sp = 0
    if odt is _E4M3:
        if scales is None:
            _fail("an output in float8_e4m3fn needs scales")
        m = scales.shape[-1] if scales.dim() else 0
        if m == 0 or n % m:
            _fail(f"scales must be [.., m] with m a divisor of {n}")
        sp = _vector(scales, "scales", torch.float32, shape[:-1] + (m,), dev)
        block = n // m
    elif scales is not None:
        _fail("scales are for an output in float8_e4m3fn")
    # the rows of a two-dimensional x are a batch of single tokens
    d = ssu_norm_dims(shape[0], 1 if two else shape[1], n, group, block, weight.shape[0],
                      _DT[dtype], _DT[wdt], _DT[rdt], SSU_E4M3 if block else _DT[odt],
                      1 if unit_offset else 0, 1 if gate_first else 0, *xs, *zs, *rs, *os_)
    _launch(dev, stream, lib.ssu_rms_norm, d, x.data_ptr(), wp, rp, zp, out.data_ptr(), sp,
            float(eps))
    return out


def logprobs_workspace_bytes(batch, num_tokens, vocab, top=0):
    """Bytes of the workspace ssu_token_logprobs needs for exactly these sizes (no GPU needed;
    -1 for what the call refuses)."""
    d = ssu_logprob_dims(batch, num_tokens, vocab, top)
    return int(load_library().ssu_logprobs_workspace_bytes(d))


def ssu_token_logprobs(logits, tokens, logprobs, *, entropy=None, top_ids=None, top_logprobs=None,
                       context_lengths=None, state_indices=None, workspace=None, stream=None):
    """Log probabilities of given tokens, the entropy and the most probable alternatives.

    logits [rows, vocab] or [batch, num_tokens, vocab] (slices of wider tensors are fine: the
    vocabulary dense); tokens int32, logprobs and entropy fp32 [rows] or [batch, num_tokens];
    top_ids int32 and top_logprobs fp32 [.., k], k up to 32, in descending order, equal logits
    by index. context_lengths, state_indices [batch] int32: rows past a length, and of negative
    indices, are not read. workspace: a uint8 GPU tensor of at least
    logprobs_workspace_bytes(...) bytes for this call's sizes (allocated here when None).
    """
    lib = _LIB or load_library()
    two = logits.dim() == 2
    dev = _first(logits, "logits", 2 if two else 3, "[rows, vocab] or [batch, num_tokens, vocab]")
    shape, dtype = logits.shape, logits.dtype
    vocab, lead = shape[-1], shape[:-1]
    if vocab < 1 or vocab > 1 << 24:
        _fail(f"vocab {vocab} outside [1, 2^24]")
    ls = _DENSE if logits.is_contiguous() else _outer(logits.stride(), shape, "logits", two)
    f32, i32 = torch.float32, torch.int32
    tp = _vector(tokens, "tokens", i32, lead, dev)
    pp = _vector(logprobs, "logprobs", f32, lead, dev)
    ep = _vector(entropy, "entropy", f32, lead, dev)
    top = tip = tlp = 0
    if (top_ids is None) != (top_logprobs is None):
        _fail("top_ids and top_logprobs go together")
    if top_ids is not None:
        top = top_ids.shape[-1] if top_ids.dim() else 0
        if not 1 <= top <= min(SSU_MAX_TOP, vocab):
            _fail(f"top_ids must be [.., k] with k in [1, {min(SSU_MAX_TOP, vocab)}]")
        tip = _vector(top_ids, "top_ids", i32, lead + (top,), dev)
        tlp = _vector(top_logprobs, "top_logprobs", f32, lead + (top,), dev)
    cp = _vector(context_lengths, "context_lengths", i32, shape[:1], dev)
    ip = _vector(state_indices, "state_indices", i32, shape[:1], dev)
    d = ssu_logprob_dims(shape[0], 1 if two else shape[1], vocab, top, _DT[dtype], 0, *ls)
    workspace, wp, wn = _scratch(workspace, lib.ssu_logprobs_workspace_bytes(d), logits.device, stream)
    _launch(dev, stream, lib.ssu_token_logprobs, d, logits.data_ptr(), tp, cp, ip, pp, ep, tip, tlp,
            wp, wn)
    return logprobs


# ---------------------------------------------------------------------------
# Recurrent-state pool
# ---------------------------------------------------------------------------
class DeviceArray:
    """Non-owning view of pool memory: enough of the tensor protocol for the SSU
    entry points (data_ptr, shape, stride, dtype, device) plus
    __cuda_array_interface__ for zero-copy interop."""

    _TYPESTR = {torch.float32: "<f4", torch.float16: "<f2", torch.bfloat16: "<V2",
                torch.uint8: "|u1"}

    def __init__(self, ptr, shape, dtype, device, owner):
        self._ptr, self.shape, self.dtype, self.device = ptr, tuple(shape), dtype, device
        self._owner = owner  # keeps the pool alive
        st, acc = [], 1
        for s in reversed(self.shape):
            st.append(acc)
            acc *= s
        self._stride = tuple(reversed(st))
        self.is_cuda = True

    def data_ptr(self):
        return self._ptr

    def stride(self):
        return self._stride

    def dim(self):
        return len(self.shape)

    @property
    def __cuda_array_interface__(self):
        return {"shape": self.shape, "typestr": self._TYPESTR[self.dtype],
                "data": (self._ptr, False), "version": 3, "strides": None}


class SsuPool:
    """Handle of an ssu_pool: one zeroed [slot_count] + shape slab per spec.

    specs: sequence of (kind, layer, shape, dtype) with dtype a torch dtype
    (float32, float16, bfloat16 or uint8). name: the pool's name in the
    library's diagnostics. base: None (the library allocates the slabs) or a
    uint8 GPU tensor of at least slab_bytes(specs, slot_count) bytes, 256-byte
    aligned, in which the states are laid out (the pool then owns no memory and
    keeps a reference to the tensor).
    """

    def __init__(self, specs: Sequence, slot_count: int, *, name=None, base=None, stream=None,
                 device=None):
        self._lib = load_library()
        if base is not None:
            _dense(base, "base", (torch.uint8,))
            device = base.device if device is None else device
        self.device = (torch.device("cuda", torch.cuda.current_device()) if device is None
                       else torch.device(device))
        arr = self._spec_array(specs)
        self.specs = [(kind, layer, tuple(int(v) for v in shape), dtype)
                      for (kind, layer, shape, dtype) in specs]
        self._base = base
        self._h = ctypes.c_void_p()
        with torch.cuda.device(self.device):
            _check(self._lib.ssu_pool_alloc(arr, len(specs), slot_count,
                                            None if name is None else name.encode(),
                                            _ptr(base) if base is not None else None,
                                            0 if base is None else base.numel(),
                                            _stream(self.device, stream), ctypes.byref(self._h)))
        self.slot_count = slot_count

    @staticmethod
    def _spec_array(specs):
        arr = (ssu_state_spec * max(len(specs), 1))()
        for i, (kind, layer, shape, dtype) in enumerate(specs):
            shape = tuple(int(v) for v in shape)
            _need(1 <= len(shape) <= 4, "spec shape must have 1..4 entries")
            arr[i].kind, arr[i].layer, arr[i].rank = kind, layer, len(shape)
            arr[i].dtype = _DT.get(dtype, 99)
            for k, v in enumerate(shape):
                arr[i].shape[k] = v
        return arr

    @staticmethod
    def bytes_per_slot(specs):
        lib = load_library()
        out = ctypes.c_size_t()
        _check(lib.ssu_pool_bytes_per_slot(SsuPool._spec_array(specs), len(specs),
                                           ctypes.byref(out)))
        return out.value

    @staticmethod
    def slab_bytes(specs, slot_count):
        """Bytes a caller slab (`base`) must hold for these specs and slots."""
        lib = load_library()
        out = ctypes.c_size_t()
        _check(lib.ssu_pool_slab_bytes(SsuPool._spec_array(specs), len(specs), slot_count,
                                       ctypes.byref(out)))
        return out.value

    @property
    def name(self):
        p = ctypes.c_char_p()
        _check(self._lib.ssu_pool_name(self._h, ctypes.byref(p)))
        return p.value.decode()

    @property
    def owns_memory(self):
        o = ctypes.c_int32()
        _check(self._lib.ssu_pool_owns_memory(self._h, ctypes.byref(o)))
        return bool(o.value)

    def spec(self, i):
        """(kind, layer, shape, dtype) of state i, as the library holds it."""
        sp = ssu_state_spec()
        _check(self._lib.ssu_pool_spec(self._h, i, ctypes.byref(sp)))
        return self._spec_tuple(sp)

    def specs_from_library(self):
        n = ctypes.c_int32()
        _check(self._lib.ssu_pool_specs(self._h, None, 0, ctypes.byref(n)))
        arr = (ssu_state_spec * max(n.value, 1))()
        _check(self._lib.ssu_pool_specs(self._h, arr, n.value, ctypes.byref(n)))
        return [self._spec_tuple(arr[i]) for i in range(n.value)]

    @staticmethod
    def _spec_tuple(sp):
        dt = {v: k for k, v in _DT.items()}[sp.dtype]
        return (sp.kind, sp.layer, tuple(int(sp.shape[k]) for k in range(sp.rank)), dt)

    def close(self):
        if getattr(self, "_h", None) and self._h.value:
            _check(self._lib.ssu_pool_free(self._h))
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def num_states(self):
        n, s = ctypes.c_int32(), ctypes.c_int32()
        _check(self._lib.ssu_pool_info(self._h, ctypes.byref(n), ctypes.byref(s)))
        return n.value

    def state_bytes_per_slot(self, i):
        out = ctypes.c_size_t()
        _check(self._lib.ssu_pool_state_bytes_per_slot(self._h, i, ctypes.byref(out)))
        return out.value

    def find_state(self, kind, layer):
        out = ctypes.c_int32()
        _check(self._lib.ssu_pool_find_state(self._h, kind, layer, ctypes.byref(out)))
        return out.value

    def state(self, i):
        """DeviceArray view of state i, shaped [slot_count] + spec shape."""
        p = ctypes.c_void_p()
        _check(self._lib.ssu_pool_state_ptr(self._h, i, ctypes.byref(p)))
        kind, layer, shape, dtype = self.specs[i]
        return DeviceArray(p.value or 0, (self.slot_count,) + shape, dtype, self.device, self)

    def clear(self, stream=None):
        _check(self._lib.ssu_pool_clear(self._h, _stream(self.device, stream)))

    def clear_slot(self, slot, stream=None):
        _check(self._lib.ssu_pool_clear_slot(self._h, slot, _stream(self.device, stream)))

    def capture(self, slot, dst=None, stream=None):
        """Copy one slot of every state into `dst` (list of GPU tensors, allocated
        here when None) and return it."""
        if dst is None:
            dst = [_result((1,) + shape, dtype, self.device, stream)
                   for (_, _, shape, dtype) in self.specs]
        n = len(dst)
        ptrs = (ctypes.c_void_p * max(n, 1))(*[t.data_ptr() for t in dst])
        sizes = (ctypes.c_size_t * max(n, 1))(*[t.numel() * t.element_size() for t in dst])
        _check(self._lib.ssu_pool_capture(self._h, slot, ptrs, sizes, n,
                                          _stream(self.device, stream)))
        return dst

    def restore(self, saved, slot, stream=None):
        n = len(saved)
        ptrs = (ctypes.c_void_p * max(n, 1))(*[t.data_ptr() for t in saved])
        sizes = (ctypes.c_size_t * max(n, 1))(*[t.numel() * t.element_size() for t in saved])
        _check(self._lib.ssu_pool_restore(self._h, slot, ptrs, sizes, n,
                                          _stream(self.device, stream)))

    def copy_slot_from(self, source: "SsuPool", dst_slot, src_slot, stream=None):
        _check(self._lib.ssu_pool_copy_slot_from(self._h, source._h, dst_slot, src_slot,
                                                 _stream(self.device, stream)))
