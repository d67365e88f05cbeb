"""Host side of the convolution, scan and draft-verification calls (no GPU: every
path here returns before any HIP call): sizes of workspaces, calls without work,
the largest sizes, layouts, and where a call's scratch is allocated."""
import ctypes
import os
import subprocess
import sys

import pytest

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
