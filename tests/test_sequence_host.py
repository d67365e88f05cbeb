"""Host side of the convolution, scan and draft-verification calls (no GPU: every
path here returns before any HIP call): sizes of workspaces, calls without work,
the largest sizes, layouts, and where a call's scratch is allocated."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

from linear_rnn_recurrent_amd import ssu as S

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(S.LIB_PATH):
        from linear_rnn_recurrent_amd import build
        build.build()
    return S.load_library()


@pytest.mark.parametrize("batch,seq_len,dim,dstate", [(0, 64, 128, 16), (0, 1, 64, 16), (0, 4096, 5120, 16),
                                                      (0, 600, 70, 64), (4, 0, 128, 16), (0, 0, 8, 4)])
def test_an_empty_scan_needs_no_workspace(lib, batch, seq_len, dim, dstate):
    """In a process of its own: an integer division by zero ends the process."""
    code = ("from linear_rnn_recurrent_amd import ssu as S; import ctypes; "
            f"print(S.scan_workspace_bytes({batch}, {seq_len}, {dim}, {dstate}), "
            f"S.load_library().ssu_scan_workspace_bytes(ctypes.byref(S.ssu_scan_dims({batch}, {dim}, {dstate}, 1)), "
            f"{seq_len}))")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-500:]
    assert r.stdout.split() == ["0", "0"]


class _Allocations:
    """Records what is entered and allocated, in order."""

    def __init__(self, monkeypatch):
        self.log = log = []

        class Under:
            def __init__(self, stream):
                self.stream = stream

            def __enter__(self):
                log.append(("enter", self.stream))

            def __exit__(self, *_):
                log.append(("leave", self.stream))

        class Block:
            is_cuda, dtype = True, torch.uint8

            def data_ptr(self):
                return 4096

            def numel(self):
                return 100

            def record_stream(self, stream):
                log.append(("record", stream))

        def empty(*_, **__):
            log.append("empty")
            return Block()

        monkeypatch.setattr(torch.cuda, "stream", Under)
        monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device: ("external", handle, device))
        monkeypatch.setattr(torch, "empty", empty)


@pytest.mark.parametrize("stream,current", [(None, None), ("a stream", "a stream"),
                                            (7040, ("external", 7040, "gpu")), (0, ("external", 0, "gpu"))])
def test_scratch_belongs_to_the_stream_of_its_call(monkeypatch, stream, current):
    """The allocator orders a block by the stream that is current at its allocation:
    a block of another stream's may still be in use there by what was queued before
    it was freed, and nothing makes the call's stream wait for that."""
    seen = _Allocations(monkeypatch)
    block, address, size = S._scratch(None, 100, "gpu", stream)
    assert block is not None and (address, size) == (4096, 100)
    if current is None:
        assert seen.log == ["empty"]
    else:
        assert seen.log[:3] == [("enter", current), "empty", ("leave", current)]


def test_no_scratch_where_none_is_needed(monkeypatch):
    seen = _Allocations(monkeypatch)
    assert S._scratch(None, 0, "gpu", "a stream") == (None, 0, 0) and seen.log == []


def test_results_belong_to_the_stream_of_their_call_and_wait_for_their_reader(monkeypatch):
    seen = _Allocations(monkeypatch)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device: ("current", device))
    S._result((3, 4), torch.float32, "gpu", None)
    assert seen.log == ["empty"]
    S._result((3, 4), torch.float32, "gpu", "a stream")
    assert seen.log[1:] == [("enter", "a stream"), "empty", ("leave", "a stream"),
                            ("record", ("current", "gpu"))]


class OnGpu(torch.Tensor):
    """A CPU tensor that the binding takes for one of cuda:0."""
    is_cuda = True

    def get_device(self):
        return 0


def on_gpu(t):
    return t.as_subclass(OnGpu)


@pytest.fixture
def launched(monkeypatch):
    """(entry point, arguments) of every call that the binding would make."""
    calls = []
    monkeypatch.setattr(S, "_launch", lambda dev, stream, fn, *args: calls.append((fn, args)))
    return calls


def conv_prefill(state, batch=2, seq_len=5, channels=8, width=4, x=None, out=None):
    x = torch.zeros(batch, seq_len, channels) if x is None else x
    out = torch.zeros(batch, seq_len, channels) if out is None else out
    S.ssu_conv_prefill(on_gpu(x), on_gpu(torch.zeros(channels, width)), None,
                       None if state is None else on_gpu(state), on_gpu(out))


@pytest.mark.parametrize("make", [
    lambda: torch.zeros(()).expand(6, 8, 3), lambda: torch.zeros(8, 3).expand(6, 8, 3),
    lambda: torch.zeros(6, 1, 3).expand(6, 8, 3), lambda: torch.zeros(6, 8, 1).expand(6, 8, 3),
    lambda: torch.zeros(1, 1, 3).expand(6, 8, 3)])
def test_a_broadcast_conv_state_is_refused(lib, launched, make):
    """Three strides of 0 are the library's word for a dense pool: passed on, the call
    would read and write past the one entry that is there."""
    with pytest.raises(ValueError, match="conv_state must not be broadcast"):
        conv_prefill(make())
    assert not launched


@pytest.mark.parametrize("shape,channels,width", [((1, 1, 1), 1, 2), ((1, 8, 3), 8, 4), ((1, 1, 3), 1, 4),
                                                  ((2, 8, 0), 8, 1)])
def test_axes_of_one_entry_may_have_any_stride(lib, launched, shape, channels, width):
    state = torch.zeros(shape)
    state = state.as_strided(shape, [0 if n == 1 else s for n, s in zip(shape, state.stride())])
    conv_prefill(state, batch=1, channels=channels, width=width)
    dims = launched[0][1][0]
    assert (dims.pool_rows, dims.channels, dims.width) == (shape[0], channels, width)


def conv_dims(**kw):
    d = dict(batch=0, channels=16, width=4, pool_rows=4, io_dtype=2, weight_dtype=2, state_dtype=2,
             reserved=0, x_batch_stride=0, x_token_stride=0, out_batch_stride=0, out_token_stride=0,
             state_row_stride=0, state_chan_stride=0, state_tap_stride=0)
    d.update(kw)
    return S.ssu_conv_dims(*d.values())


def conv_status(lib, seq_len=8, **kw):
    """With batch 0 a call returns after its checks of sizes and strides."""
    return lib.ssu_conv_prefill(conv_dims(**kw), seq_len, *([None] * 5), 1, 1, None, None, None)


@pytest.mark.parametrize("row,chan,tap", [
    (48, 3, 1), (48, 1, 16), (3, 12, 1), (1, 12, 4), (1, 4, 64), (16, 1, 64), (50, 3, 1), (5, 23, 1)])
def test_every_order_of_the_pools_axes_is_taken(lib, row, chan, tap):
    assert conv_status(lib, state_row_stride=row, state_chan_stride=chan, state_tap_stride=tap) == 0


@pytest.mark.parametrize("row,chan,tap", [(47, 3, 1), (2, 12, 1), (3, 11, 1), (1, 3, 48), (1, 4, 63), (15, 1, 64),
                                          (16, 1, 63), (0, 3, 1), (3, 3, 1), (48, 3, 0), (1, 1, 1)])
def test_overlapping_pools_are_refused(lib, row, chan, tap):
    assert conv_status(lib, state_row_stride=row, state_chan_stride=chan, state_tap_stride=tap) == 1
    assert "conv_state" in lib.ssu_last_error().decode()


def test_huge_strides_do_not_wrap(lib):
    assert conv_status(lib, state_row_stride=1 << 62, state_chan_stride=1 << 61, state_tap_stride=1) == 1


def scan_dims(**kw):
    d = dict(batch=0, dim=16, dstate=16, ngroups=1, pool_rows=4, state_dtype=0, io_dtype=2,
             dt_dtype=0, bc_dtype=2, reserved=0, state_row_stride=0)
    for k in ("x", "z", "out", "dt", "b", "c"):
        d[k + "_batch_stride"] = d[k + "_token_stride"] = 0
    d.update(kw)
    return S.ssu_scan_dims(*d.values())


# A null pointer is the first thing refused after the strides: status 1 with its name.
@pytest.mark.parametrize("bs,ts,taken", [
    (16, 48, True), (20, 60, True), (16, 1000, True), (128, 16, True), (16, 47, False), (15, 48, False),
    (17, 49, False), (20, 55, False), (127, 16, False), (16, 16, False), (1 << 61, 1 << 62, False)])
def test_sequence_major_activations_are_taken(lib, bs, ts, taken):
    """3 batch entries of 8 tokens of 16 channels: rows that do not overlap are taken
    in either order of the axes, others refused."""
    def told(rc, needle):
        assert rc == 1 and needle in lib.ssu_last_error().decode(), lib.ssu_last_error()

    for name in ("x", "out"):
        kw = {name + "_batch_stride": bs, name + "_token_stride": ts}
        told(conv_status(lib, batch=3, **kw), "'x'" if taken else f"{name} batch stride")
    for name, arg in (("x", "x"), ("z", "z"), ("out", "out"), ("dt", "dt"), ("b", "B"), ("c", "C")):
        kw = {name + "_batch_stride": bs, name + "_token_stride": ts}
        rc = lib.ssu_scan_prefill(scan_dims(batch=3, **kw), 8, *([None] * 10), 1, 1, None, None, None, 0, None)
        told(rc, "'x'" if taken else f"{arg} batch stride")
    for name, tokens in (("target", 8), ("draft", 9)):
        kw = dict(batch=3, num_tokens=tokens, vocab=16, max_accept_len=1, prob_dtype=0, reserved=0,
                  target_batch_stride=0, target_row_stride=0, draft_batch_stride=0, draft_row_stride=0)
        kw[name + "_batch_stride"], kw[name + "_row_stride"] = bs, ts
        rc = lib.ssu_draft_verify(S.ssu_verify_dims(*kw.values()), *([None] * 11), 0, None)
        told(rc, "'tokens'" if taken else f"{name}_probs batch stride")


@pytest.mark.skipif(torch.cuda.device_count() > 0, reason="its pointers may not reach a launch on a GPU")
@pytest.mark.parametrize("batch,seq_len,channels,V", [
    (1, 8380000, (1 << 20) + 1, 1),   # sixteens of tokens fit a launch, eights do not
    (1, 1 << 20, 65537, 1),           # workgroups fit in 31 bits, threads do not in 32
    (1 << 20, 1 << 20, 1 << 20, 8), ((1 << 31) - 1, 1 << 30, (1 << 31) - 1, 1)])
def test_convolutions_past_one_launch_are_refused(lib, batch, seq_len, channels, V):
    p = 0x100000
    d = conv_dims(batch=batch, channels=channels)
    assert lib.ssu_conv_prefill(d, seq_len, p, p, None, p, p + (16 if V == 8 else 2), 1, 1, None, p, None) == 2
    assert "too large" in lib.ssu_last_error().decode()


@pytest.mark.skipif(torch.cuda.device_count() > 0, reason="its pointers may not reach a launch on a GPU")
@pytest.mark.parametrize("seq_len", [1, 2])
@pytest.mark.parametrize("batch,dim,dstate", [(1 << 14, 1 << 14, 256), (1 << 16, 1 << 13, 64)])
def test_scans_past_one_launch_are_refused(lib, seq_len, batch, dim, dstate):
    p = 0x100000
    d = scan_dims(batch=batch, dim=dim, dstate=dstate)
    args = [p] * 5 + [None] * 3 + [p, p + 16, 1]
    if seq_len == 1:
        rc = lib.ssu_scan_decode(d, *args, p, None)
    else:
        rc = lib.ssu_scan_prefill(d, seq_len, *args, 1, None, p, p, 1 << 60, None)
    assert rc == 2 and "too large" in lib.ssu_last_error().decode()


@pytest.mark.parametrize("stream", [None, 7040])
def test_a_workspace_on_another_device_is_refused(stream):
    class Block:
        is_cuda, dtype, shape = True, torch.uint8, (100,)

        def __init__(self, device):
            self.device = torch.device(device)

        def is_contiguous(self):
            return True

        def data_ptr(self):
            return 4096

        def numel(self):
            return 100

    dev = torch.device("cuda:0")
    with pytest.raises(ValueError, match="workspace.*cuda:1.*cuda:0"):
        S._scratch(Block("cuda:1"), 100, dev, stream)
    here = Block("cuda:0")
    assert S._scratch(here, 100, dev, stream) == (here, 4096, 100)


def test_an_empty_convolution_of_width_one_is_a_call_without_work(lib, launched):
    conv_prefill(None, batch=0, width=1)
    assert launched[0][1][0].pool_rows > 0  # the library refuses a pool without rows


@pytest.mark.parametrize("batch,seq_len,dim,dstate,ngroups", [
    (1, 64, 5120, 18, 1), (1, 64, 5120, 260, 1), (1, 64, 5120, 0, 1), (1, (1 << 30) + 1, 64, 16, 1),
    (1, -1, 64, 16, 1), (-1, 64, 64, 16, 1), (1, 64, 64, 16, 3), (1, 64, (1 << 25) + 1, 16, 1),
    (1 << 20, 64, 1 << 11, 16, 1)])
def test_workspace_of_sizes_that_the_scan_refuses(lib, batch, seq_len, dim, dstate, ngroups):
    assert S.scan_workspace_bytes(batch, seq_len, dim, dstate, ngroups) == -1
    d = scan_dims(batch=batch, dim=dim, dstate=dstate, ngroups=ngroups, pool_rows=(1 << 31) - 1)
    assert lib.ssu_scan_prefill(d, seq_len, *([None] * 10), 1, 1, None, None, None, 0, None) in (1, 2)
    assert "'x'" not in lib.ssu_last_error().decode()


def test_workspace_of_a_scan_is_that_of_its_sizes_alone(lib):
    """What the header says of it: neither batch nor seq_len bounds it, and nothing but
    the five sizes counts."""
    need = [S.scan_workspace_bytes(b, 4096, 5120, 16) for b in (1, 2, 4, 8, 16)]
    assert need[0] > need[2] > 0 and need[3] == 0 < need[4]
    assert S.scan_workspace_bytes(4, 2048, 5120, 16) == 0 < S.scan_workspace_bytes(1, 2048, 5120, 16)
    for types in range(3):
        d = scan_dims(batch=1, dim=5120, pool_rows=9 + types, state_dtype=types, io_dtype=types, dt_dtype=types,
                      bc_dtype=2 - types, x_token_stride=6000, b_token_stride=33, state_row_stride=5120 * 20)
        assert lib.ssu_scan_workspace_bytes(d, 4096) == need[0]
    d = scan_dims(batch=4, dim=5120, pool_rows=4)
    for given in (need[2] - 1, need[3]):
        rc = lib.ssu_scan_prefill(d, 4096, *([0x100000] * 5), None, None, None, 0x100000, 0x200000, 1, 1, None,
                                  None, 0x100000, given, None)
        assert rc == 1 and f"{need[2]} required" in lib.ssu_last_error().decode()


@pytest.mark.skipif(torch.cuda.device_count() > 0, reason="its pointers may not reach a launch on a GPU")
def test_single_tokens_in_an_inputs_place(lib):
    """out may be x or z of the same strides; rows of other strides would overlap other
    rows' inputs, and B and C are read by every channel."""
    p, q = 0x100000, 0x200000
    told = lambda: lib.ssu_last_error().decode()  # noqa: E731

    def scan(x=p, z=None, B=p, C=p, dt=p, **kw):
        d = scan_dims(batch=2, **kw)
        return lib.ssu_scan_decode(d, x, p, B, C, dt, None, None, z, p, q, 1, None, None)

    def conv(x, **kw):
        return lib.ssu_conv_decode(conv_dims(batch=2, **kw), x, p, None, p, q, 1, None, None)

    for kw in (dict(B=q), dict(C=q)):
        assert scan(**kw) == 1 and "overlap" in told(), kw
    for kw in (dict(x=q, x_batch_stride=32), dict(z=q, out_batch_stride=24), dict(x=q, z=q, z_batch_stride=48)):
        assert scan(**kw) == 1 and "strides" in told(), kw
    assert conv(q, x_batch_stride=32) == 1 and "strides" in told()
    # taken (the launch fails without a GPU)
    for rc in (scan(x=q), scan(z=q), scan(x=q, x_batch_stride=24, out_batch_stride=24), conv(q),
               conv(q, x_batch_stride=17, out_batch_stride=17), scan(x=p, x_batch_stride=32)):
        assert rc == 3, told()
