"""The group norm kernel's evaluation of its activations, checked on the CPU by
a C mirror of its fp32 operations (tests/numerics/norm_activation_sweep.c),
with the hardware reciprocal and exp2 each off by up to one ulp and flushing
below the normal range: within 2^-17 relative of the fp64 definitions.
test_gpu_norm_activations.py applies the bound to the device's results."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
SRC = os.path.join(HERE, "numerics", "norm_activation_sweep.c")
FUNCTIONS = 2


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs a C compiler")
def test_norm_activations_within_bound(tmp_path):
    exe = str(tmp_path / "norm_activation_sweep")
    subprocess.run(["gcc", "-O2", "-ffp-contract=off", "-o", exe, SRC, "-lm"], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
    assert r.stdout.count("max relative error") == 9 * FUNCTIONS
