"""Which evaluation of the per-channel scan a call takes, decided on the host by its
sizes and checked on the CPU: the choice is compiled by the host's compiler alone."""
import os
import subprocess

import pytest

from linear_rnn_recurrent_amd import ssu as S
from scan_evaluations import SIZES, TYPED

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ALL = {**SIZES, **TYPED}

PROGRAM = r"""
#include <cstdio>
#include "ssu_scan_plan.h"
int main()
{
    long b, t, d, n, g, lengths;
    while (std::scanf("%ld %ld %ld %ld %ld %ld", &b, &t, &d, &n, &g, &lengths) == 6) {
        const ssu::ScanPlan q = ssu::scan_plan(b, d, n, g, t, lengths != 0);
        if (q.rows)
            std::printf("rows %d\n", n <= 16 ? 4 : n <= 32 ? 8 : n <= 64 ? 16 : n <= 128 ? 32 : 64);
        else if (q.sweep)
            std::printf("sweep %d %d\n", q.sweep, q.s.tiles);
        else
            std::printf("chunks %d %d %d %d\n", q.s.tiles, q.s.chunk, q.s.chunks, q.s.team);
    }
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    src, exe = d / "plan.cpp", d / "plan"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-O1", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(ROOT, "linear_rnn_recurrent_amd", "csrc"), "-I", "/opt/rocm/include",
                    str(src), "-o", str(exe)], check=True, capture_output=True)

    def ask(sizes):
        lines = "\n".join(" ".join(str(int(v)) for v in s) for s in sizes)
        out = subprocess.run([str(exe)], input=lines, check=True, capture_output=True, text=True).stdout
        rows = [ln.split() for ln in out.splitlines()]
        return [(r[0], *map(int, r[1:])) for r in rows]

    return ask


def test_the_listed_sizes_take_the_listed_evaluations(plan):
    got = dict(zip(ALL, plan(ALL)))
    assert got == ALL


def test_the_list_reaches_every_kind_of_kernel():
    kinds = set(SIZES.values())
    assert {k[1] for k in kinds if k[0] == "rows"} == {4, 8, 16, 32, 64}
    for waves in (4, 8, 16):
        assert {1, 2, 3} < {k[2] for k in kinds if k[:2] == ("sweep", waves)}
    chunks = [k[1:] for k in kinds if k[0] == "chunks"]
    assert {c[3] for c in chunks if c[0] == 1} == {1, 2, 4}  # workgroups of one, two and four chunks
    assert {1, 2, 3, 4} <= {c[0] for c in chunks if c[3] == 4 and c[0] <= 4}
    assert {c[0] for c in chunks if c[2] > 1 and c[3] == 2 and c[0] > 4} >= {5, 7, 8}
    assert {c[0] for c in chunks if c[2] > 1 and c[3] == 1} >= {13, 16}
    assert {c[0] for c in chunks if c[1] > 32 and c[2] > 1} >= {1, 2, 3, 4, 7, 8, 16}  # longer than 32 tokens
    assert {c[0] for c in chunks if c[2] == 1} >= {1, 2, 3, 13}  # one chunk to a row


def test_workspace_covers_both_choices(plan):
    """The size query does not know whether a call has context_lengths: it covers the
    chunks of either."""
    sizes = [s[:5] for s in ALL]
    for flag in (False, True):
        for s, kind in zip(sizes, plan([(*s, flag) for s in sizes])):
            b, t, d, n, g = s
            need = S.scan_workspace_bytes(b, t, d, n, g)
            if kind[0] == "chunks":
                tiles, _, chunks, _ = kind[1:]
                blocks = g * ((d // g + 63) // 64)
                assert need >= 4 * (b * t * g * tiles * 32 + 32 + b * (chunks + 1) * blocks * (tiles * 1024 + 64))


def test_sizes_past_one_launch_take_no_chunks(plan):
    """Packed B and C of 2^32 values a half or more, and other sizes at the limits."""
    for size in [(64, 65536, 1024, 128, 8, False), (1, 1 << 30, 64, 16, 4, True), (1, 1 << 28, 64, 16, 1, False)]:
        assert plan([size])[0][0] != "chunks", size
    assert plan([(1, (1 << 28) - 1, 64, 16, 1, False)])[0][0] == "chunks"


@pytest.mark.parametrize("size,kind", [
    # a block of each channel, 2^22 blocks and more: chunks as long as their own launches fit
    ((4096, 40, 1024, 16, 1024, False), "chunks"), ((8192, 20, 1024, 16, 1024, False), "chunks"),
    # rows of 64 lanes past 2^32 threads, sweeps within
    ((8192, 2, 8192, 256, 1, False), "sweep"), ((8192, 3, 8192, 256, 1, True), "sweep"),
    # the rows' launch just fits
    ((4095, 2, 16384, 256, 1, False), "rows"), ((1 << 16, 1, 1 << 15, 16, 1, False), "rows")])
def test_the_choice_keeps_to_what_one_launch_holds(plan, size, kind):
    assert plan([size])[0][0] == kind
