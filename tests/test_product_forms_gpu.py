"""Every form of the product for few rows, and the one for many, on the same sizes:
rows that end inside a tile, loads of an expert above what one pass of its
blocks takes (so that a cluster sums several tiles one after the other), a depth
whose blocks the split does not divide and whose last one is short."""
import pytest
import torch

import expert_ref as R
import product_forms
from allreduce_residual_rmsnorm_gb300 import binding as B
from test_product_waits_gpu import Product

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def forms(cuda_lib, tmp_path_factory):
    return product_forms.load(tmp_path_factory.mktemp("forms"), 1_000_000)


SIZES = [((150, 300, 1296), None), ((229, 264, 1296), [0, 1, 200, 0, 17, 3]), ((65, 129, 2064), None)]


@pytest.fixture(scope="module", params=[(s, d) for s in SIZES for d in DT],
                ids=lambda p: "-".join(map(str, p[0][0])) + ("-experts-" if p[0][1] else "-") + p[1])
def product(cuda_lib, request):
    (dims, loads), dt = request.param
    return Product(*dims, DT[dt], loads, seed=dims[0])


@pytest.mark.parametrize("tokens,split", [(t, s) for t in (16, 32, 64) for s in (1, 2, 4, 8)] + [(0, 0)])
def test_form(forms, product, tokens, split):
    assert product.run(forms, tokens, split) == (B.AR_OK, -1)
    product.check()


# sizes whose call takes a form that the tests of the calls do not reach otherwise
@pytest.mark.parametrize("rows,cols,depth,loads,form", [
    (800, 136, 4112, [500, 0, 291], (32, 2)), (300, 136, 4112, [7, 250, 40], (32, 4)),
    (200, 136, 8208, [1, 0, 190], (32, 8)), (3000, 136, 128, [2000, 1, 990], (64, 1)),
    (1000, 136, 16400, [30, 900, 65], (64, 4))])
def test_call_that_takes_the_form(forms, rows, cols, depth, loads, form):
    assert product_forms.choice(forms, rows, cols, depth, len(loads)) == form
    p = Product(rows, cols, depth, torch.bfloat16, loads, seed=rows)
    p.guard.fill_(77.0)
    out = p.guard[:rows * cols].view(rows, cols)
    a, sa, b, sb = p.dev
    B.ar_fusion_expert_matmul_fp8(a, sa, b, sb, p.off, out)
    torch.cuda.synchronize()
    p.check()
    assert bool((p.guard[p.rows_used * cols:] == 77.0).all())
    assert R.blocks(depth) == p.nb and B.ar_fusion_matmul_status() == (B.AR_OK, -1)


@pytest.mark.parametrize("rows,cols,depth,dt", [(5000, 136, 128, "fp16"), (5003, 133, 112, "bf16"),
                                               (5003, 133, 112, "fp32")])
def test_dense_call_of_64_rows_at_a_time(forms, rows, cols, depth, dt):
    assert product_forms.choice(forms, rows, cols, depth) == (64, 1)
    p = Product(rows, cols, depth, DT[dt], seed=rows)
    p.guard.fill_(77.0)
    a, sa, b, sb = p.dev
    B.ar_fusion_matmul_fp8(a, sa, b[0], sb[0], p.guard[:rows * cols].view(rows, cols))
    torch.cuda.synchronize()
    p.check()
    assert bool((p.guard[rows * cols:] == 77.0).all())
