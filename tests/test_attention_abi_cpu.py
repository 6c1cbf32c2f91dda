"""Argument checks of the attention-layer calls that need no GPU."""
import ctypes

import pytest
import torch

import attention_ref as R
from allreduce_residual_rmsnorm_gb300 import binding as B
from allreduce_residual_rmsnorm_gb300 import build as BUILD


@pytest.fixture(scope="module")
def L():
    BUILD.build()
    return B.load()


def refused(rc, code, part):
    assert rc == code, (rc, B.ar_fusion_last_error())
    assert part in B.ar_fusion_last_error(), B.ar_fusion_last_error()


P, ODD, ODD4 = 4096, 4096 + 8, 4096 + 2


def cache(**kw):
    a = dict(k=P, v=P, k_page=2048, k_row=128, k_head=64, v_page=2048, v_row=128, v_head=64, dtype=0,
             pages=10, page_size=16, heads=2, head_dim=64, sequences=3, max_pages=5, scale=None,
             page_table=P, lengths=P)
    a.update(kw)
    return B._KvCache(**a)


def rows(data=P, row=512, head=64):
    return B._HeadRows(data, row, head)


def decode(L, c=None, q=None, out=None, lse=None, heads=8, dtype=0, scale=0.1, window=0, sinks=0,
           work=P, size=1 << 20):
    return L.ar_fusion_decode_attention(c or cache(), q or rows(), out or rows(), lse, heads, dtype,
                                        scale, window, sinks, work, size, None)


def prompt(L, c=None, q=None, out=None, lse=None, starts=P, tokens=9, heads=8, dtype=0, scale=0.1,
           window=0, sinks=0, work=P, size=1 << 20):
    return L.ar_fusion_prompt_attention(c or cache(), q or rows(), out or rows(), lse, starts, tokens,
                                        heads, dtype, scale, window, sinks, work, size, None)


def append(L, c=None, q=0, q_out=0, k=None, v=None, tokens=3, heads=8, dtype=0, starts=P,
           positions=None, f=P, rot=64, sections=None, axes=1, inter=0):
    q = rows() if q == 0 else q
    q_out = rows() if q_out == 0 else q_out
    table = None if sections is None else (ctypes.c_int * len(sections))(*sections)
    return L.ar_fusion_rope_append(c or cache(), q, q_out, k or rows(), v or rows(), tokens, heads,
                                   dtype, starts, positions, f, rot, table, axes, inter, None)


I, N = B.AR_ERR_INVALID, B.AR_ERR_UNSUPPORTED
CACHES = [
    (dict(dtype=2), N, "cache dtype"), (dict(dtype=4), N, "cache dtype"), (dict(dtype=1), I, "cache dtype"),
    (dict(pages=0), I, "pages"), (dict(heads=0), I, "heads"), (dict(max_pages=0), I, "max_pages"),
    (dict(sequences=-1), I, "sequences"), (dict(sequences=2049), N, "sequences"),
    (dict(page_size=24), I, "page_size"), (dict(page_size=0), I, "page_size"),
    (dict(page_size=4), N, "page_size"), (dict(page_size=1 << 17), N, "page_size"),
    (dict(max_pages=1 << 28), N, "max_pages"), (dict(head_dim=0), I, "head_dim"),
    (dict(head_dim=68), I, "head_dim"), (dict(head_dim=136), N, "head_dim"),
    (dict(dtype=3, head_dim=72), I, "head_dim"), (dict(scale=P), I, "scale"),
    (dict(k_page=0), I, "k: stride"), (dict(k_row=-128), I, "k: stride"), (dict(v_head=12), I, "v: stride"),
    (dict(v_page=1 << 40), I, "v: stride"), (dict(dtype=3, k_row=136), I, "k: stride"),
    (dict(k=None), I, "k or v"), (dict(v=ODD), I, "k or v"), (dict(page_table=None), I, "page_table"),
    (dict(lengths=ODD4), I, "lengths"), (dict(dtype=3, scale=ODD4), I, "scale")]


@pytest.mark.parametrize("kw,code,part", CACHES, ids=str)
def test_caches_refused_by_every_call(L, kw, code, part):
    refused(decode(L, cache(**kw)), code, part)
    refused(prompt(L, cache(**kw)), code, part)
    refused(append(L, cache(**kw)), code, part)


@pytest.mark.parametrize("call", [decode, prompt])
def test_attention_refusals(L, call):
    refused(call(L, dtype=2), N, "dtype")
    refused(call(L, heads=0), I, "q_heads")
    refused(call(L, heads=7), I, "q_heads")
    refused(call(L, heads=258), N, "share")
    for scale in (0.0, -1.0, float("inf"), float("nan"), 3.4e38):
        refused(call(L, scale=scale), I, "scale")
    refused(call(L, window=-1), I, "window")
    refused(call(L, sinks=-1), I, "sinks")
    refused(call(L, sinks=4), I, "without a window")
    refused(call(L, work=ODD), I, "workspace")
    refused(call(L, work=None), I, "workspace")
    refused(call(L, q=rows(ODD)), I, "q NULL")
    refused(call(L, out=rows(None)), I, "out NULL")
    refused(call(L, q=rows(row=12)), I, "q: strides")
    refused(call(L, out=rows(head=1 << 41)), I, "out: strides")
    refused(call(L, lse=ODD4), I, "lse")
    assert call(L, cache(sequences=0)) == B.AR_OK


def test_prompt_refusals(L):
    refused(prompt(L, tokens=-1), I, "tokens")
    refused(prompt(L, tokens=1 << 30), N, "rows")
    refused(prompt(L, starts=None), I, "starts")
    assert prompt(L, tokens=0) == B.AR_OK


def test_append_refusals(L):
    refused(append(L, dtype=2), N, "dtype")
    refused(append(L, tokens=-1), I, "tokens")
    refused(append(L, starts=None, tokens=4), I, "starts")
    refused(append(L, heads=3), I, "q_heads")
    refused(append(L, rot=-16), I, "rot")
    refused(append(L, rot=24), I, "rot")
    refused(append(L, rot=80), I, "rot")
    refused(append(L, axes=0), I, "axes")
    refused(append(L, axes=5, sections=[8, 8, 8, 8, 0]), I, "axes")
    refused(append(L, axes=2), I, "sections NULL")
    refused(append(L, axes=2, sections=[16, 15]), I, "sections add up")
    refused(append(L, axes=2, sections=[33, -1]), I, "sections[1]")
    refused(append(L, axes=2, sections=[2 ** 31 - 1, 2 ** 31 - 1]), I, "sections add up")
    refused(append(L, inter=2), I, "interleaved")
    refused(append(L, f=None), I, "inv_freq")
    refused(append(L, starts=ODD4), I, "starts")
    refused(append(L, positions=ODD4), I, "positions")
    refused(append(L, q=rows(ODD)), I, "q NULL")
    refused(append(L, q_out=None), I, "q_out NULL")
    refused(append(L, k=rows(None)), I, "k NULL")
    refused(append(L, v=rows(row=4)), I, "v: strides")
    assert append(L, tokens=0) == B.AR_OK
    assert append(L, cache(sequences=0), tokens=0, starts=None) == B.AR_OK


def test_status_without_a_call(L):
    assert L.ar_fusion_decode_attention(None, None, None, None, 1, 0, 1.0, 0, 0, None, 0, None) == I


def test_binding_refuses_types_shapes_and_host_tensors():
    z, i32, bf = torch.zeros, torch.int32, torch.bfloat16
    kc, table, n = z(4, 16, 2, 64, dtype=bf), z(3, 2, dtype=i32), z(3, dtype=i32)
    q, out = z(3, 8, 64, dtype=bf), z(3, 8, 64, dtype=bf)
    f = B.ar_fusion_decode_attention
    for bad, kind, part in [
            (dict(q=z(3, 8, dtype=bf)), ValueError, "q"), (dict(q=z(3, 8, 64)), TypeError, "q"),
            (dict(k_cache=z(4, 16, 2, 64)), TypeError, "k_cache"),
            (dict(v_cache=z(4, 16, 2, 32, dtype=bf)), ValueError, "v_cache"),
            (dict(v_cache=z(4, 16, 2, 64, dtype=torch.float16)), TypeError, "v_cache"),
            (dict(page_table=z(3, dtype=i32)), ValueError, "page_table"), ({}, ValueError, "CUDA")]:
        a = dict(q=q, k_cache=kc, v_cache=kc, page_table=table, lengths=n, out=out)
        a.update(bad)
        with pytest.raises(kind, match=part):
            f(**a)
    with pytest.raises(ValueError, match="k: 2 dim"):
        B.ar_fusion_rope_append(q, z(3, 2), z(3, 2), kc, kc, table, n, None)
    with pytest.raises(TypeError, match="k: unsupported"):
        B.ar_fusion_rope_append(q, z(3, 2, 64), z(3, 2, 64), kc, kc, table, n, None)


# ------------------------------------------- the 64-bit reference itself

def test_reference_attention_by_hand():
    # two keys of one head, scores 0 and log 3: weights 1/4, 3/4
    k = torch.zeros(1, 8, 1, 8)
    v = torch.zeros(1, 8, 1, 8)
    k[0, 1, 0, 0] = 1.0
    v[0, 0, 0, 1], v[0, 1, 0, 1] = 4.0, 8.0
    q = torch.zeros(2, 1, 8)
    q[1, 0, 0] = float(torch.log(torch.tensor(3.0)))
    out, lse, mags, reach, count, big = R.attention(
        q, k, v, torch.tensor([[0]]), torch.tensor([2]), [0, 2], 1.0, 0, 0)
    assert torch.allclose(out[:, 0, 1], torch.tensor([4.0, 7.0], dtype=torch.float64), atol=1e-6)
    assert torch.allclose(lse[:, 0], torch.tensor([0.0, 4.0]).double().clamp_min(1).log(), atol=1e-6)
    assert count[:, 0].tolist() == [1, 2] and big[1, 0] == 8.0
    # a window of one sees the own key alone, with a first token visible both
    one = R.attention(q, k, v, torch.tensor([[0]]), torch.tensor([2]), [0, 2], 1.0, 1, 0)[0]
    assert one[1, 0, 1] == 8.0
    both = R.attention(q, k, v, torch.tensor([[0]]), torch.tensor([2]), [0, 2], 1.0, 1, 1)[0]
    assert abs(float(both[1, 0, 1]) - 7.0) < 1e-6


def test_reference_turn_by_hand():
    x = torch.zeros(1, 1, 4, dtype=torch.float64)
    x[0, 0] = torch.tensor([1.0, 2.0, 3.0, 4.0])
    quarter = torch.tensor([torch.pi / 2, 0.0], dtype=torch.float64)
    half = R.turn(x, torch.tensor([[1]]), quarter, [0, 0], False)[0, 0]
    assert torch.allclose(half, torch.tensor([-3.0, 2.0, 1.0, 4.0]).double())
    near = R.turn(x, torch.tensor([[1]]), quarter, [0, 0], True)[0, 0]
    assert torch.allclose(near, torch.tensor([-2.0, 1.0, 3.0, 4.0]).double())
