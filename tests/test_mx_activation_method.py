"""The GELU in front of MXFP4 quantisation, checked on the CPU by a C mirror of its
fp32 operations (tests/numerics/mx_activation_sweep.c) over every bf16 value,
with the hardware reciprocal and exp2 each off by up to one ulp: within 2^-17
relative of the fp64 definition."""
import os
import shutil
import subprocess

import pytest

SRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "numerics", "mx_activation_sweep.c")


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs a C compiler")
def test_gelu_within_bound(tmp_path):
    exe = str(tmp_path / "mx_activation_sweep")
    subprocess.run(["gcc", "-O2", "-ffp-contract=off", "-o", exe, SRC, "-lm"], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
    assert r.stdout.count("max relative error") == 9
