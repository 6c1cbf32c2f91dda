"""Argument checks of the expert-layer calls that need no GPU: the C entry
points answer with a status before any CUDA call, the binding refuses operands
of the wrong type, shape, layout or place."""
import ctypes

import numpy as np
import pytest
import torch

import expert_ref as R
from allreduce_residual_rmsnorm_gb300 import binding as B
from allreduce_residual_rmsnorm_gb300 import build as BUILD

P, ODD, ODD4 = ctypes.c_void_p(4096), ctypes.c_void_p(4096 + 8), ctypes.c_void_p(4096 + 2)


@pytest.fixture(scope="module")
def L():
    BUILD.build()
    return B.load()


def refused(rc, code, part):
    assert rc == code, (rc, B.ar_fusion_last_error())
    assert part in B.ar_fusion_last_error(), B.ar_fusion_last_error()


def route(L, **kw):
    a = dict(logits=P, tokens=4, experts=64, dtype=0, bias=None, score=1, groups=4, kept=2, gs=1,
             topk=6, renorm=1, scale=1.0, ids=P, w=P)
    a.update(kw)
    return L.ar_fusion_route(a["logits"], a["tokens"], a["experts"], a["dtype"], a["bias"],
                             a["score"], a["groups"], a["kept"], a["gs"], a["topk"], a["renorm"],
                             a["scale"], a["ids"], a["w"], None)


@pytest.mark.parametrize("kw,code,part", [
    (dict(dtype=5), B.AR_ERR_UNSUPPORTED, "dtype"), (dict(tokens=-1), B.AR_ERR_INVALID, "tokens"),
    (dict(experts=0), B.AR_ERR_INVALID, "experts"), (dict(topk=0), B.AR_ERR_INVALID, "topk"),
    (dict(experts=1025, groups=1, kept=1), B.AR_ERR_UNSUPPORTED, "experts"),
    (dict(experts=64, groups=1, kept=1, topk=33), B.AR_ERR_UNSUPPORTED, "topk"),
    (dict(experts=99, groups=33, kept=33), B.AR_ERR_UNSUPPORTED, "groups"),
    (dict(groups=0), B.AR_ERR_INVALID, "groups"), (dict(groups=5), B.AR_ERR_INVALID, "divide"),
    (dict(kept=0), B.AR_ERR_INVALID, "groups_kept"), (dict(kept=5), B.AR_ERR_INVALID, "groups_kept"),
    (dict(experts=8, topk=5), B.AR_ERR_INVALID, "topk"), (dict(score=2), B.AR_ERR_INVALID, "score"),
    (dict(gs=2), B.AR_ERR_INVALID, "group_score"), (dict(renorm=2), B.AR_ERR_INVALID, "renormalize"),
    (dict(logits=None), B.AR_ERR_INVALID, "logits"), (dict(logits=ODD), B.AR_ERR_INVALID, "logits"),
    (dict(ids=None), B.AR_ERR_INVALID, "ids"), (dict(w=ODD4), B.AR_ERR_INVALID, "weights"),
    (dict(bias=ODD4), B.AR_ERR_INVALID, "bias")])
def test_route_refusals(L, kw, code, part):
    refused(route(L, **kw), code, part)


def test_plan_refusals(L):
    f = L.ar_fusion_expert_plan
    refused(f(P, -1, 8, 0, 8, P, P, None), B.AR_ERR_INVALID, "tokens")
    refused(f(P, 4, 0, 0, 8, P, P, None), B.AR_ERR_INVALID, "topk")
    refused(f(P, 4, 8, -1, 8, P, P, None), B.AR_ERR_INVALID, "first_expert")
    refused(f(P, 4, 8, 0, 0, P, P, None), B.AR_ERR_INVALID, "experts")
    refused(f(P, 4, 8, 0, 1025, P, P, None), B.AR_ERR_UNSUPPORTED, "experts")
    refused(f(P, 1 << 30, 8, 0, 8, P, P, None), B.AR_ERR_UNSUPPORTED, "topk")
    refused(f(P, 4, 8, 2 ** 31 - 4, 8, P, P, None), B.AR_ERR_UNSUPPORTED, "first_expert")
    refused(f(P, 4, 8, 0, 8, None, P, None), B.AR_ERR_INVALID, "offsets")
    refused(f(None, 4, 8, 0, 8, P, P, None), B.AR_ERR_INVALID, "ids")
    refused(f(P, 4, 8, 0, 8, P, ODD4, None), B.AR_ERR_INVALID, "position")


def test_quant_blocks_refusals(L):
    def f(i=P, rows=4, hidden=128, dt=0, act=0, pos=None, copies=1, count=None, out=4, q=P, s=P):
        return L.ar_fusion_quant_blocks(i, rows, hidden, dt, act, pos, copies, count, out, q, s, None)
    refused(f(dt=3), B.AR_ERR_UNSUPPORTED, "dtype")
    refused(f(rows=-1), B.AR_ERR_INVALID, "rows")
    refused(f(out=-1, pos=P), B.AR_ERR_INVALID, "out_rows")
    refused(f(hidden=0), B.AR_ERR_INVALID, "hidden")
    refused(f(hidden=136), B.AR_ERR_INVALID, "hidden")
    refused(f(act=2), B.AR_ERR_INVALID, "activation")
    refused(f(copies=2), B.AR_ERR_INVALID, "copies")
    refused(f(copies=0, pos=P), B.AR_ERR_INVALID, "copies")
    refused(f(out=3), B.AR_ERR_INVALID, "out_rows")
    refused(f(i=ODD), B.AR_ERR_INVALID, "in")
    refused(f(q=None), B.AR_ERR_INVALID, "quant_out")
    refused(f(s=None), B.AR_ERR_INVALID, "scale_out")
    refused(f(pos=ODD4), B.AR_ERR_INVALID, "position")
    refused(f(count=ODD4), B.AR_ERR_INVALID, "row_count")
    assert f(rows=0) == B.AR_OK


def test_matmul_refusals(L):
    def f(a=P, sa=P, b=P, sb=P, rows=4, cols=8, depth=32, dt=0, out=P):
        return L.ar_fusion_matmul_fp8(a, sa, b, sb, rows, cols, depth, dt, out, None)

    def x(off=P, experts=3, rows=4, **kw):
        return L.ar_fusion_expert_matmul_fp8(kw.get("a", P), P, P, P, off, experts, rows, 8,
                                             kw.get("depth", 32), kw.get("dt", 0), P, None)
    refused(f(dt=9), B.AR_ERR_UNSUPPORTED, "dtype")
    refused(f(rows=-2), B.AR_ERR_INVALID, "rows")
    refused(f(cols=0), B.AR_ERR_INVALID, "cols")
    refused(f(depth=0), B.AR_ERR_INVALID, "depth")
    refused(f(depth=24), B.AR_ERR_INVALID, "depth")
    refused(f(a=ODD), B.AR_ERR_INVALID, "aligned")
    refused(f(b=None), B.AR_ERR_INVALID, "NULL")
    refused(f(out=ODD), B.AR_ERR_INVALID, "aligned")
    refused(f(sa=ODD4), B.AR_ERR_INVALID, "a_scale")
    refused(f(sb=None), B.AR_ERR_INVALID, "b_scale")
    assert f(rows=0, a=None, out=None) == B.AR_OK
    refused(x(off=None), B.AR_ERR_INVALID, "offsets")
    refused(x(experts=0), B.AR_ERR_INVALID, "experts")
    refused(x(experts=2000), B.AR_ERR_UNSUPPORTED, "experts")
    refused(x(depth=8), B.AR_ERR_INVALID, "depth")
    assert x(rows=0, off=None) == B.AR_OK


def test_combine_refusals(L):
    def f(r=P, n=9, pos=P, w=P, T=4, k=2, H=64, dt=0, add=None, out=P):
        return L.ar_fusion_combine(r, n, pos, w, T, k, H, dt, add, out, None)
    refused(f(dt=4), B.AR_ERR_UNSUPPORTED, "dtype")
    refused(f(n=-1), B.AR_ERR_INVALID, "in_rows")
    refused(f(T=-1), B.AR_ERR_INVALID, "tokens")
    refused(f(k=0), B.AR_ERR_INVALID, "topk")
    refused(f(H=12), B.AR_ERR_INVALID, "hidden")
    refused(f(r=ODD), B.AR_ERR_INVALID, "rows_in")
    refused(f(add=ODD), B.AR_ERR_INVALID, "add")
    refused(f(out=None), B.AR_ERR_INVALID, "out")
    refused(f(pos=None), B.AR_ERR_INVALID, "position")
    refused(f(w=ODD4), B.AR_ERR_INVALID, "weights")
    assert f(T=0) == B.AR_OK


def test_binding_refuses_types_shapes_and_host_tensors():
    i32 = torch.int32
    z = torch.zeros
    with pytest.raises(TypeError, match="logits"):
        B.ar_fusion_route(z(2, 8, dtype=torch.float64), None, z(2, 2, dtype=i32), z(2, 2))
    with pytest.raises(ValueError, match="weights_out"):
        B.ar_fusion_route(z(2, 8), None, z(2, 2, dtype=i32), z(2, 3))
    with pytest.raises(ValueError, match="bias"):
        B.ar_fusion_route(z(2, 8), z(7), z(2, 2, dtype=i32), z(2, 2))
    with pytest.raises(ValueError, match="CUDA"):
        B.ar_fusion_route(z(2, 8), None, z(2, 2, dtype=i32), z(2, 2))
    with pytest.raises(ValueError, match="offsets_out"):
        B.ar_fusion_expert_plan(z(2, 2, dtype=i32), 8, z(8, dtype=i32), z(2, 2, dtype=i32))
    with pytest.raises(TypeError, match="ids"):
        B.ar_fusion_expert_plan(z(2, 2, dtype=torch.int64), 8, z(9, dtype=i32), z(2, 2, dtype=i32))
    u8 = torch.uint8
    with pytest.raises(ValueError, match="x: shape"):
        B.ar_fusion_quant_blocks(z(2, 32), z(2, 32, dtype=u8), z(2, 1),
                                 activation=B.AR_ACT_SILU_MUL)
    with pytest.raises(ValueError, match="scale_out"):
        B.ar_fusion_quant_blocks(z(2, 144), z(2, 144, dtype=u8), z(2, 1))
    with pytest.raises(ValueError, match="position"):
        B.ar_fusion_quant_blocks(z(2, 32), z(2, 32, dtype=u8), z(2, 1), position=z(3, 1, dtype=i32))
    with pytest.raises(ValueError, match="row_count"):
        B.ar_fusion_quant_blocks(z(2, 32), z(2, 32, dtype=u8), z(2, 1), row_count=z(2, dtype=i32))
    with pytest.raises(ValueError, match="b: shape"):
        B.ar_fusion_matmul_fp8(z(2, 32, dtype=u8), z(2, 1), z(3, 48, dtype=u8), z(1, 1), z(2, 3))
    with pytest.raises(ValueError, match="b_scale"):
        B.ar_fusion_matmul_fp8(z(2, 32, dtype=u8), z(2, 1), z(130, 32, dtype=u8), z(1, 1), z(2, 130))
    with pytest.raises(TypeError, match="out"):
        B.ar_fusion_matmul_fp8(z(2, 32, dtype=u8), z(2, 1), z(3, 32, dtype=u8), z(1, 1),
                               z(2, 3, dtype=torch.float64))
    with pytest.raises(ValueError, match="offsets"):
        B.ar_fusion_expert_matmul_fp8(z(2, 32, dtype=u8), z(2, 1), z(4, 3, 32, dtype=u8), z(4, 1, 1),
                                      z(4, dtype=i32), z(2, 3))
    with pytest.raises(TypeError, match="out"):
        B.ar_fusion_combine(z(4, 16), z(2, 2, dtype=i32), z(2, 2), z(2, 16, dtype=torch.float16))
    with pytest.raises(ValueError, match="add"):
        B.ar_fusion_combine(z(4, 16), z(2, 2, dtype=i32), z(2, 2), z(2, 16), add=z(1, 16))


def test_binding_refuses_numbers_past_32_bits(L):
    """ctypes alone would pass the lower 32 bits."""
    for first in (1 << 32, 1 << 31, -(1 << 31) - 1):
        with pytest.raises(ValueError, match="32-bit"):
            B._call("ar_fusion_expert_plan", (4096, 1, 1, first, 8, 4096, 4096, None))


# ------------------------------------------- the 64-bit reference itself

def test_reference_decodes_e4m3_as_torch_does():
    all_codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(all_codes).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(R.e4m3(all_codes), want.astype(np.float64), equal_nan=True)


def test_reference_route_by_hand():
    x = torch.tensor([[1.0, 3.0, 2.0, 3.0, -1.0, 0.0]])
    ids, w = R.route(x, None, 3, "softmax", 1, 1, "max", True, 1.0)
    assert ids.tolist() == [[1, 3, 2]]               # the tie goes to the lower index
    e = np.exp(np.array([3.0, 3.0, 2.0]))
    assert np.allclose(w[0], e / e.sum(), rtol=1e-14)
    # groups {1, 3}, {2, 3}, {-1, 0}: sums of two of the sigmoids
    ids, _ = R.route(x, None, 2, "sigmoid", 3, 1, "top2", False, 1.0)
    assert ids.tolist() == [[3, 2]]
    bias = torch.tensor([0.0, -float("inf"), 0.0, 0.0, 5.0, 0.0])
    ids, w = R.route(x, bias, 6, "sigmoid", 1, 1, "max", False, 1.0)
    assert ids.tolist() == [[4, 3, 2, 0, 5, -1]] and w[0, 5] == 0.0


def test_reference_plan_by_hand():
    off, pos = R.plan(np.array([[2, 0], [5, 2], [0, -1]]), 0, 3)
    assert off.tolist() == [0, 2, 2, 4] and pos.tolist() == [[2, 0], [-1, 3], [1, -1]]
