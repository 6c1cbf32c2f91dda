"""The products' bounded waits: one that runs out, what the status call says of it,
and kernels whose waits give up almost at once with copies and products in
flight.  Those answer right or report the wait; either way they end, write nothing
outside the output and leave the device usable."""
import numpy as np
import pytest
import torch

import expert_ref as R
import product_forms
from allreduce_residual_rmsnorm_gb300 import binding as B

U = 2.0 ** -24
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def forms(cuda_lib, tmp_path_factory):
    return product_forms.load(tmp_path_factory.mktemp("forms"), 1_000_000)


@pytest.fixture(scope="module", params=[1, 500, 3_000])
def hasty(cuda_lib, tmp_path_factory, request):
    """The kernels with waits that give up after that many nanoseconds."""
    return product_forms.load(tmp_path_factory.mktemp("hasty"), request.param, alone=True)


def test_a_wait_that_runs_out_is_reported_once(forms):
    out = torch.full((3,), -1, dtype=torch.int32, device="cuda")
    assert B.ar_fusion_matmul_status() == (B.AR_OK, -1)
    assert forms.lone_wait(3, out.data_ptr()) == 0
    torch.cuda.synchronize()
    assert out.tolist() == [0, 0, 1]        # gave up; gave up at once; has arrived
    assert forms.lone_wait(40, out.data_ptr()) == 0     # the first one is kept
    assert B.ar_fusion_matmul_status() == (B.AR_ERR_TIMEOUT, 3)
    assert B.ar_fusion_matmul_status() == (B.AR_OK, -1)


class Product:
    def __init__(self, rows, cols, depth, dtype, loads=None, seed=1):
        g = torch.Generator()
        g.manual_seed(seed)
        self.dims, self.dtype, self.nb = (rows, cols, depth), dtype, R.blocks(depth)
        E = 1 if loads is None else len(loads)
        codes = lambda *s: (150.0 * torch.randn(s, generator=g)).clamp(-448, 448).to(  # noqa: E731
            torch.float8_e4m3fn).view(torch.uint8)
        scales = lambda *s: 0.01 * torch.exp(0.5 * torch.randn(s, generator=g))  # noqa: E731
        a, b = codes(rows, depth), codes(E, cols, depth)
        sa, sb = scales(rows, self.nb), scales(E, R.blocks(cols), self.nb)
        ends = [0, rows] if loads is None else np.concatenate([[0], np.cumsum(loads)]).tolist()
        self.want, self.mags = np.zeros((rows, cols)), np.zeros((rows, cols))
        for e in range(E):
            lo, hi = ends[e], ends[e + 1]
            self.want[lo:hi], self.mags[lo:hi] = R.matmul(a.numpy()[lo:hi], sa.numpy()[lo:hi],
                                                          b.numpy()[e], sb.numpy()[e])
        self.rows_used, self.experts = ends[-1], E
        self.dev = [t.cuda() for t in (a, sa, b, sb)]
        self.off = None if loads is None else torch.tensor(ends, dtype=torch.int32, device="cuda")
        self.guard = torch.empty(rows * cols + 4096, dtype=dtype, device="cuda")

    def run(self, forms, tokens, split):
        rows, cols, depth = self.dims
        self.guard.fill_(77.0)
        rc = forms.product_form(
            *(t.data_ptr() for t in self.dev), None if self.off is None else self.off.data_ptr(),
            self.experts, rows, cols, depth, B._ELEM[self.dtype], self.guard.data_ptr(), tokens,
            split, B._stream(None))
        assert rc == 0
        status = product_forms.status(forms)
        assert bool((self.guard[self.rows_used * cols:] == 77.0).all())
        return status

    def check(self):
        rows, cols, _ = self.dims
        n = self.rows_used
        got = self.guard[:n * cols].view(n, cols).double().cpu().numpy()
        want = self.want[:n]
        # 128 additions a block, off by a whole step of the sum of magnitudes each at
        # most; a scale product, an addition a block, a split's sums, one rounding
        tol = ((256 + self.nb + 12) * U * self.mags[:n] + R.half_step(self.dtype) * np.abs(want) +
               2.0 ** -140 + 2.0 ** -25 * (self.dtype == torch.float16))
        bad = ~(np.abs(got - want) <= tol)
        assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5])


@pytest.mark.parametrize("tokens,split,dims,loads", [
    (16, 1, (40, 300, 2064), None), (16, 8, (40, 300, 2064), None), (64, 4, (150, 520, 4112), None),
    (32, 2, (300, 260, 656), [0, 1, 130, 40, 120]), (0, 0, (700, 1032, 2064), None),
    (0, 0, (900, 1028, 400), [300, 0, 2, 129, 460])])
def test_products_whose_waits_give_up_at_once(hasty, forms, tokens, split, dims, loads):
    p = Product(*dims, torch.bfloat16, loads)
    gave_up = 0
    for _ in range(20):
        code, detail = p.run(hasty, tokens, split)
        if code == B.AR_OK:
            p.check()
        else:
            assert code == B.AR_ERR_TIMEOUT and detail in range(1, 7)
            gave_up += 1
        assert p.run(forms, tokens, split) == (B.AR_OK, -1)
        p.check()
    print("gave up", gave_up, "of 20")
