"""The block quantiser's activation where a block's gates are all far from zero,
so that its scale shows the error of the activation there.

Bound, u = 2^-24: ex2.approx is off by 2.45 u at most, the sum 1 + e^-g, the
quotient and the product with the other half by one u each: y by 5.5 u.  The scale
is y's largest magnitude divided by 448 and rounded: 6.5 u.  A decoded value is
y times a rounded reciprocal of the scale, times the scale: three more u beside
half an E4M3 step of y (2^-4 of it, or 2^-10 scales below the normal range).
"""
import numpy as np
import pytest
import torch

import expert_ref as R
from allreduce_residual_rmsnorm_gb300 import binding as B

U = 2.0 ** -24
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("gate", [-87.0, -80.0, -60.0, -40.0, -30.0, -20.0, -12.0, -6.0, -1.5, 1.5,
                                  12.0, 60.0, 87.0])
def test_scale_of_blocks_of_far_gates(cuda_lib, gate, dt):
    g = torch.Generator()
    g.manual_seed(int(2 * gate) + 500)
    rows, hidden = 600, 272                     # two whole blocks and one of 16
    x = torch.empty(rows, 2 * hidden)
    x[:, :hidden] = gate + 0.9 * torch.rand(rows, hidden, generator=g) - 0.45
    # one element of each block far above its others, its y above the floor
    x[:, hidden:] = torch.randn(rows, hidden, generator=g)
    x[:, [hidden + 3, hidden + 200, hidden + 265]] += 4096.0
    if gate < 0:
        x[:, hidden:] *= 2.0 ** min(100.0, -1.4427 * gate)
    x = x.to(dt)
    assert bool((x[:, :hidden].abs() < 88.0).all()) and bool(x.isfinite().all())
    q = torch.empty(rows, hidden, dtype=torch.uint8, device="cuda")
    s = torch.empty(rows, 3, device="cuda")
    B.ar_fusion_quant_blocks(x.cuda(), q, s, activation=B.AR_ACT_SILU_MUL)
    y = R.activate(x, True)
    amax = R.block_amax(y)
    assert (amax > R.FLOOR).all()
    scale = s.cpu().double().numpy()
    off = np.abs(scale * 448.0 - amax) / amax / U
    assert (off <= 6.5).all(), off.max()
    wide = R.spread(scale, hidden)
    err = np.abs(R.e4m3(q.cpu().numpy()) * wide - y)
    assert (err <= np.maximum(np.abs(y) * 2.0 ** -4, wide * 2.0 ** -10) + 9 * U * np.abs(y)).all()
