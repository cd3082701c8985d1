"""The launch shape that segquant_adapter_add chooses, read from the library's
own planning by a small program linked against it (no GPU)."""
import os
import shutil
import subprocess

import pytest

import segmented_dual_scale_amd as S
from segmented_dual_scale_amd import build as B

HERE = os.path.dirname(os.path.abspath(__file__))
CUS = 256

pytestmark = pytest.mark.skipif(not (os.path.exists(B._hipcc()) or shutil.which(B._hipcc())),
                                reason="needs hipcc")


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("plan") / "adapter_plan")
    lib = S.library_path()
    src = os.path.join(HERE, "numerics", "adapter_plan.hip")
    for cmd in ([*B.CFLAGS, "-I", B.CSRC, "-c", src, "-o", exe + ".o"],
                [exe + ".o", lib, f"-Wl,-rpath,{os.path.dirname(lib)}", "-o", exe]):
        r = subprocess.run([B._hipcc(), *cmd], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
    return exe


def plans(program, *cases):
    r = subprocess.run([program] + [",".join(map(str, c)) for c in cases], check=True,
                       capture_output=True, text=True)
    keys = ("one", "tile_rows", "by_row", "run_blocks", "splits")
    return [dict(zip(keys, map(int, line.split()))) for line in r.stdout.splitlines()]


def workgroups(plan, lens, N, n_nseg):
    tiles = sum(-(-n // plan["tile_rows"]) for n in lens)
    return tiles * n_nseg * -(-(N // n_nseg) // (64 * plan["run_blocks"]))


@pytest.mark.parametrize("requests,rows,K,N,rank,segs", [
    (64, 8, 1536, 1536, 16, 1), (64, 2, 1536, 1536, 16, 1), (48, 16, 1536, 1536, 32, 1),
    (16, 16, 1536, 9216, 32, 6), (32, 4, 1024, 4608, 16, 3)])
def test_a_few_rows_per_request_fill_the_chip(program, requests, rows, K, N, rank, segs):
    """Up to 16 rows of a request make one tile of rows, so the columns have to
    be cut into enough runs for the CUs."""
    plan, = plans(program, (requests * rows, N, K, requests, rank, segs))
    assert plan["one"]
    assert workgroups(plan, [rows] * requests, N, segs) >= CUS, plan


def test_single_rows_keep_their_runs(program):
    for plan, n in zip(plans(program, (2, 9216, 1536, 2, 16, 6), (64, 9216, 1536, 64, 32, 6)),
                       (2, 64)):
        assert plan["one"] and plan["by_row"]
        assert plan["run_blocks"] == (4 if n == 2 else 12)


def test_few_rows_per_request_with_an_x_beyond_the_caches(program):
    """Every segment after the first reads x again in one launch: two launches
    where that is more than the last-level cache holds."""
    case = (65536, 4608, 4096, 4096, 16)
    one, large, small = plans(program, (*case, 1), (*case, 3), (4096, 4608, 4096, 512, 16, 3))
    assert one["one"] and small["one"] and not large["one"]
