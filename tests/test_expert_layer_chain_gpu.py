"""The expert-layer calls and the fused call queued one behind the other, with no
synchronisation between them: each kernel is resident while the one before it
still writes.  The results are those of the same calls waited for one by one."""
import os
import subprocess
import sys

import pytest
import torch

from allreduce_residual_rmsnorm_gb300 import binding as B
from test_expert_layer_gpu import Layer

pytestmark = pytest.mark.gpu


class Chain:
    """Two ranks' layers, the fused call on their outputs, and the next layer's
    quantisation of its normed rows."""

    def __init__(self, T, H):
        self.ranks = [Layer(T, H, 256, 64, 6, first, 32, seed=60 + first) for first in (0, 32)]
        self.ws = B.ar_fusion_workspace_create(2, max(T, 16), H, B.AR_DT_BF16)
        self.T = T
        self.gamma = torch.ones(H, dtype=torch.bfloat16, device="cuda")
        self.res, self.norm = (torch.empty_like(self.ranks[0].x) for _ in range(2))
        self.q = torch.empty(T, H, dtype=torch.uint8, device="cuda")
        self.scale = torch.empty(T, -(-H // 128), device="cuda")

    def run(self, wait):
        sync = torch.cuda.synchronize if wait else (lambda: None)
        for r in self.ranks:
            r.run()
            sync()
        B.ar_fusion_run(self.ws, [r.out for r in self.ranks], self.ranks[0].x, self.gamma, 1e-6,
                        B.PATTERNS["res_norm"], residual_out=self.res, norm_out=self.norm)
        sync()
        B.ar_fusion_quant_blocks(self.norm, self.q, self.scale)
        sync()
        for r in self.ranks:                # the next pass runs on other rows
            r.x.copy_(self.norm)
        return self.res.clone(), self.norm.clone(), self.q.clone(), self.scale.clone()


@pytest.mark.parametrize("T", [1, 40, 300])
def test_layers_and_fused_calls_without_a_wait_between_them(cuda_lib, T):
    a, b = Chain(T, 512), Chain(T, 512)
    for r, s in zip(a.ranks, b.ranks):
        assert torch.equal(r.x, s.x) and torch.equal(r.logits, s.logits)
    want = [a.run(True) for _ in range(12)]
    torch.cuda.synchronize()
    got = [b.run(False) for _ in range(12)]
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(w, g))
    assert B.ar_fusion_workspace_status(b.ws)[0] == B.AR_OK
    assert B.ar_fusion_matmul_status() == (B.AR_OK, -1)
    for c in (a, b):
        B.ar_fusion_workspace_destroy(c.ws)


FIRST_CALLS = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import torch
import test_expert_layer_gpu as E
from allreduce_residual_rmsnorm_gb300 import binding as B
layer = E.Layer(20, 512, 256, 64, 6, 0, 64, seed=9)
g = E.gen(1)
a, b = E.codes(g, 20000, 128).cuda(), E.codes(g, 272, 128).cuda()
sa, sb = E.scales(g, 20000, 1).cuda(), E.scales(g, 3, 1).cuda()
out = torch.empty(20000, 272, dtype=torch.bfloat16, device="cuda")
s = torch.cuda.Stream()
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph, stream=s):
    layer.run()
    B.ar_fusion_matmul_fp8(a, sa, b, sb, out)
graph.replay()
torch.cuda.synchronize()
layer.check()
many = out.clone()
B.ar_fusion_matmul_fp8(a, sa, b, sb, out)
assert torch.equal(many, out) and B.ar_fusion_matmul_status() == (B.AR_OK, -1)
"""


def test_first_calls_of_a_process_under_capture(cuda_lib):
    tests = os.path.dirname(os.path.abspath(__file__))
    code = FIRST_CALLS.format(root=os.path.dirname(tests), tests=tests)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-2000:]
