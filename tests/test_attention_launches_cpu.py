"""The order of the attention-layer calls' launches when several threads call at once, over a
runtime that only notes them (no GPU)."""
import os
import subprocess

from allreduce_residual_rmsnorm_gb300 import build as BUILD

HERE = os.path.dirname(os.path.abspath(__file__))
PARTS = ["attention_api.cu", "rope_append.cu", "decode_attention.cu", "prompt_attention.cu"]


def test_a_split_calls_two_launches_stay_together(tmp_path):
    objects = [os.path.join(BUILD.BUILD, f + ".o") for f in PARTS]
    BUILD.build(force=not all(map(os.path.exists, objects)))
    exe = str(tmp_path / "launch_order")
    include = os.path.join(os.path.dirname(BUILD.cuda_lib_dir()), "include")
    subprocess.check_call(["g++", "-O1", "-std=c++17", "-w", "-I", BUILD.INCLUDE, "-I", BUILD.CSRC,
                           "-I", include, os.path.join(HERE, "launch_order.cpp"), *objects, "-o", exe,
                           "-lpthread"])
    said = ""
    for _ in range(5):          # until the threads have met often enough
        r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
        said += r.stdout + r.stderr
        if r.returncode != 4:
            break
    assert r.returncode in (0, 4), said
