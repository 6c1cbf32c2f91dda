"""The attention-layer kernels' own arithmetic, compiled for the host (no GPU)."""
import os
import struct
import subprocess
from fractions import Fraction

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
        return r.stdout
    return run


def test_units_past_2_to_31(check):
    check("places")


def test_blocks_that_share_a_prompts_items_have_equal_work(check):
    check("shares")


# to 2^-180
PI = Fraction(314159265358979323846264338327950288419716939937510582097494, 10 ** 59)


def test_angles_at_any_position(check):
    """half_turns against exact arithmetic.  A turn's fixed-point part lacks 2 units of 2^-64 turns
    from the inverse of 2 pi and one of each of two roundings down, times f where that is above 1;
    the position takes them times itself, and they are rounded to a float once (2^-24 relative)."""
    lines = check("turns").split("\n")[:-1]
    assert len(lines) > 20000
    for line in lines:
        p, f, t = (int(x) for x in line.split())
        f, t = (Fraction(struct.unpack("<f", struct.pack("<I", x))[0]) for x in (f, t))
        off = (t - p * f / PI) % 2
        off = min(off, 2 - off)
        lacking = 2 * 4 * abs(p) * max(abs(f), 1) * Fraction(2) ** -64
        assert off <= lacking + abs(t) * Fraction(2) ** -24, line
