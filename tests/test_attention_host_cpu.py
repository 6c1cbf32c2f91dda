"""The attention-layer kernels' own arithmetic, compiled for the host (no GPU)."""
import os
import subprocess

import pytest

from allreduce_residual_rmsnorm_gb300 import build as BUILD

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def check(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("host") / "attention_check")
    subprocess.check_call([BUILD.nvcc(), "-O2", "-std=c++17", "-I", BUILD.INCLUDE, "-I", BUILD.CSRC,
                           os.path.join(HERE, "host_attention_check.cu"), "-o", exe])

    def run(name):
        r = subprocess.run([exe, name], capture_output=True, text=True)
        assert r.returncode == 0, r.stdout + r.stderr
    return run


def test_units_past_2_to_31(check):
    check("places")
