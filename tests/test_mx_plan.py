"""The forms of the MXFP4 product that the GPU tests' sizes reach, read from the
library's own choice by a small program linked against it (no GPU)."""
import os
import shutil
import subprocess

import pytest

import segmented_dual_scale_amd as S
import test_gpu_mx_placement as placement
from segmented_dual_scale_amd import build as B
from test_gpu_mxfp4 import FORMS, SHAPES

HERE = os.path.dirname(os.path.abspath(__file__))
SPLIT_K, SHAPE_COUNT = -1, 6  # 256x256, 224x256, 192x256, 128x256, 128x128, 64x128

pytestmark = pytest.mark.skipif(not (os.path.exists(B._hipcc()) or shutil.which(B._hipcc())),
                                reason="needs hipcc")


@pytest.fixture(scope="module")
def choices(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("plan") / "mx_plan")
    lib = S.library_path()
    src = os.path.join(HERE, "numerics", "mx_plan.hip")
    for cmd in ([*B.CFLAGS, "-I", B.CSRC, "-c", src, "-o", exe + ".o"],
                [exe + ".o", lib, f"-Wl,-rpath,{os.path.dirname(lib)}", "-o", exe]):
        r = subprocess.run([B._hipcc(), *cmd], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr

    def of(sizes):
        r = subprocess.run([exe] + [",".join(map(str, s)) for s in sizes], check=True,
                           capture_output=True, text=True)
        return [tuple(map(int, line.split())) for line in r.stdout.splitlines()]
    return of


def test_every_form_and_every_end_of_k(choices):
    """Six tile shapes and the product that splits K; K ends in each of the four steps
    of a block of scales, and only the last of them may be half full."""
    reached = {(form, -(-K // 128) % 4)
               for (M, N, K), (form, _) in zip(FORMS, choices(FORMS))}
    assert reached == {(form, end) for form in range(SPLIT_K, SHAPE_COUNT) for end in range(4)}


def test_every_form_at_scales_of_every_four_bytes(choices):
    sizes = [args for mark in placement.test_product_of_scales_at_every_four_bytes.pytestmark
             if mark.args[0] == "M,N,K" for args in mark.args[1]]
    assert {form for form, _ in choices([s for s in sizes if s[0] > 16])} == \
        set(range(SPLIT_K, SHAPE_COUNT))


def test_more_than_16_rows_quantised_inside_and_ahead(choices):
    sizes = [s for s in SHAPES + FORMS if s[0] > 16]
    inside = [i for _, i in choices(sizes)]
    assert 10 < sum(inside) < len(sizes) - 10
    for (M, N, K), i in zip(sizes, inside):
        assert not i or (K <= 1536 and -(-M // 32) * -(-N // 64) <= 256)
