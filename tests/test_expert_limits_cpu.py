"""Sizes at the ends of the expert-layer calls' ranges, answered by the C entry
points before any CUDA call."""
import ctypes

import pytest

from allreduce_residual_rmsnorm_gb300 import binding as B
from allreduce_residual_rmsnorm_gb300 import build as BUILD

P = ctypes.c_void_p(4096)
# the multiples of 16 whose number of blocks, (n + 127) / 128, does not fit 32 bits
TOO_LONG = [2 ** 31 - 16 * i for i in range(1, 8)]


@pytest.fixture(scope="module")
def L():
    BUILD.build()
    return B.load()


def unsupported(rc, part):
    assert rc == B.AR_ERR_UNSUPPORTED, (rc, B.ar_fusion_last_error())
    assert part in B.ar_fusion_last_error(), B.ar_fusion_last_error()


@pytest.mark.parametrize("n", TOO_LONG)
def test_depth_and_hidden_near_2_to_31_are_refused(L, n):
    unsupported(L.ar_fusion_matmul_fp8(P, P, P, P, 1, 1, n, 0, P, None), "depth")
    unsupported(L.ar_fusion_expert_matmul_fp8(P, P, P, P, P, 1, 1, 1, n, 0, P, None), "depth")
    for act in (B.AR_ACT_NONE, B.AR_ACT_SILU_MUL):
        unsupported(L.ar_fusion_quant_blocks(P, 1, n, 0, act, None, 1, None, 1, P, P, None),
                    "hidden")


def test_rows_for_no_place_are_taken(L):
    """out_rows 0: every position lies outside, and an empty tensor has no address."""
    assert L.ar_fusion_quant_blocks(P, 4, 128, 0, 0, P, 2, None, 0, None, None, None) == B.AR_OK
    rc = L.ar_fusion_quant_blocks(P, 4, 128, 0, 0, P, 2, None, 1, None, None, None)
    assert rc == B.AR_ERR_INVALID and "quant_out" in B.ar_fusion_last_error()


def test_no_rows_of_such_a_depth_either(L):
    unsupported(L.ar_fusion_matmul_fp8(P, P, P, P, 0, 1, 2 ** 31 - 16, 0, P, None), "depth")
    assert L.ar_fusion_matmul_fp8(P, P, P, P, 0, 1, 2 ** 31 - 128, 0, P, None) == B.AR_OK
    assert L.ar_fusion_quant_blocks(P, 0, 2 ** 31 - 128, 0, 0, None, 1, None, 1, P, P,
                                    None) == B.AR_OK
