"""Expert-layer operators on the GPU against plain 64-bit implementations
(expert_ref): routing and row layout are equal, floating outputs lie within
bounds that follow from the roundings the operators make.

Bounds, u = 2^-24 (half a step of fp32):
  weights   sigmoid: expf 2u, 1 + e and the division u each, renormalisation
            twice that, a butterfly of 5 additions, a division and the scale:
            below 16u, and where all chosen logits are negative the exponent is
            a rounded difference, which moves it by u * (maximum - minimum of
            the row): (16 + 2 * span) u.  softmax: the same of every exponent;
            its sum has at most 32 + 5 additions: below (64 + 2 * span) u.
  codes     the block's scale and codes follow from fp32 operations that round
            once each: equal.  With the activation y is off by 5u (expf 2u,
            1 + e, division, product u each): the scale is off by 6u, a decoded
            value by half an E4M3 step (2^-4 of the value, 2^-10 scales below
            the normal range) and 16u.
  product   factors are exact in fp32; 128 additions per block, each off by at
            most a whole step 2u of the sum of magnitudes (an accumulator that
            truncates), a scale product, one addition per block: (256 + nb + 4) u
            of the sum of magnitudes, and half a step of the output type.
  combine   one fused multiply-add per term: (k + 1) u of the sum of
            magnitudes, and half a step of the output type.
"""
import numpy as np
import pytest
import torch

import expert_ref as R
import oracle
from allreduce_residual_rmsnorm_gb300 import binding as B
from allreduce_residual_rmsnorm_gb300 import workloads as W

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _library(cuda_lib):
    yield
    torch.cuda.synchronize()


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


# ------------------------------------------------------------------ routing

def run_route(x, bias, topk, score, groups=1, kept=1, gscore="top2", renorm=True, scale=1.0,
              stream=None):
    T = x.shape[0]
    ids = torch.full((T, topk), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, topk), float("nan"), device="cuda")
    B.ar_fusion_route(x.cuda(), None if bias is None else bias.cuda(), ids, w,
                      score={"softmax": 0, "sigmoid": 1}[score], groups=groups, groups_kept=kept,
                      group_score={"max": 0, "top2": 1}[gscore], renormalize=renorm, scale=scale,
                      stream=stream)
    torch.cuda.synchronize()
    return ids.cpu().numpy(), w.cpu().double().numpy()


def check_route(x, bias, topk, score, **kw):
    args = dict(groups=1, kept=1, gscore="top2", renorm=True, scale=1.0)
    args.update(kw)
    ids, w = run_route(x, bias, topk, score, **args)
    r_ids, r_w = R.route(x, bias, topk, score, args["groups"], args["kept"], args["gscore"],
                         args["renorm"], args["scale"])
    assert np.array_equal(ids, r_ids), np.argwhere(ids != r_ids)[:5]
    f = x.double()
    f = torch.where(torch.isfinite(f), f, torch.zeros_like(f))
    span = (f.amax(1) - f.amin(1)).numpy()[:, None]
    tol = ((16 if score == "sigmoid" else 64) + 2 * span) * U
    nan = np.isnan(r_w)
    assert np.array_equal(np.isnan(w), nan)
    # 2^-140: exponentials below the normal range
    assert (np.abs(w - r_w) <= tol * np.abs(r_w) + 2.0 ** -140)[~nan].all()


def make_bias(kind, E, g):
    if kind == "none":
        return None
    if kind == "zero":
        return torch.zeros(E)
    b = 0.1 * torch.randn(E, generator=g)
    if kind == "masked":
        b[torch.rand(E, generator=g) < 0.4] = -float("inf")
    if kind == "lowest":
        b[torch.rand(E, generator=g) < 0.4] = torch.finfo(torch.float32).min
    return b


ROUTES = [  # T, E, topk, groups, kept, score, group score, renorm, dtype, bias
    (1, 256, 8, 8, 4, "sigmoid", "top2", True, "fp32", "random"),
    (130, 256, 8, 8, 4, "sigmoid", "top2", True, "bf16", "random"),
    (33, 256, 8, 8, 4, "sigmoid", "top2", True, "bf16", "zero"),
    (17, 64, 6, 1, 1, "softmax", "max", False, "fp32", "none"),
    (65, 60, 4, 1, 1, "softmax", "max", True, "bf16", "none"),
    (9, 160, 6, 8, 3, "softmax", "max", False, "fp16", "none"),
    (31, 160, 6, 8, 3, "softmax", "top2", True, "fp32", "none"),
    (12, 96, 5, 4, 2, "softmax", "top2", True, "fp32", "random"),
    (12, 96, 5, 4, 2, "sigmoid", "max", False, "fp16", "random"),
    (5, 1, 1, 1, 1, "softmax", "max", True, "fp32", "none"),
    (5, 7, 7, 7, 7, "sigmoid", "top2", True, "fp32", "random"),
    (6, 1024, 32, 32, 5, "sigmoid", "top2", True, "fp32", "random"),
    (3, 1000, 10, 1, 1, "softmax", "max", True, "fp32", "random"),
    (40, 66, 3, 3, 2, "sigmoid", "top2", True, "bf16", "masked"),
    (40, 128, 8, 4, 2, "softmax", "top2", True, "fp32", "masked"),
    (40, 128, 8, 4, 2, "sigmoid", "top2", True, "fp32", "lowest"),
    (7, 31, 31, 1, 1, "sigmoid", "max", True, "fp32", "masked"),
    (11, 512, 16, 16, 7, "sigmoid", "max", True, "bf16", "random"),
]


@pytest.mark.parametrize("case", ROUTES, ids=lambda c: "-".join(map(str, c)))
def test_route(case):
    T, E, k, G, kept, score, gs, renorm, dt, bias = case
    g = gen(T * 1000 + E)
    x = (1.5 * torch.randn(T, E, generator=g)).to(DT[dt])
    check_route(x, make_bias(bias, E, g), k, score, groups=G, kept=kept, gscore=gs, renorm=renorm,
                scale=2.5 if E % 3 == 0 else 1.0)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("bias", ["none", "zero", "random"])
@pytest.mark.parametrize("groups", [1, 4])
def test_route_ties_go_to_the_lower_index(score, bias, groups):
    g = gen(3)
    x = torch.randint(-2, 3, (50, 64), generator=g).float()
    b = make_bias(bias, 64, g)
    if b is not None:
        b = (b * 8).round() / 8
    check_route(x, b, 8, score, groups=groups, kept=max(1, groups // 2))


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("groups", [1, 4])
def test_route_order_below_fp32_rounding(score, groups):
    """Choice values that agree to fp32 and differ in fp64: the bias is the rounded
    distance of each score to one number, so c is that number and the rounding."""
    g = gen(4)
    T, E = 24, 128
    x = torch.randn(1, E, generator=g).repeat(T, 1)
    x += 2.0 ** -12 * torch.randn(T, E, generator=g) * (torch.arange(T) % 3 == 0).float()[:, None]
    d = x[1].double()
    s = torch.sigmoid(d) if score == "sigmoid" else torch.softmax(d, 0)
    check_route(x, (0.75 - s).float(), 8, score, groups=groups, kept=max(1, groups // 2))


def test_route_masked_and_special_logits():
    g = gen(5)
    inf, low = float("inf"), torch.finfo(torch.float32).min
    for score in ("sigmoid", "softmax"):
        for groups, kept in ((1, 1), (4, 2)):
            for bias in ("none", "random"):
                x = torch.randn(12, 32, generator=g)
                x[0] = -inf                                  # nothing left
                x[1, :] = -inf
                x[1, 9] = 0.3                                # one left
                x[2, 4:] = -inf                              # fewer than topk
                x[3] = low                                   # the lowest number everywhere
                x[4, ::2] = low
                x[5, 7] = float("nan")
                x[6] = float("nan")
                x[7] = 200.0                                 # saturated scores
                x[8] = -200.0
                x[9, 3] = -inf
                x[10] *= 40.0
                check_route(x, make_bias(bias, 32, g), 6, score, groups=groups, kept=kept)
    # +inf: under softmax the row's weights are NaN, under sigmoid its score is 1
    x = torch.randn(2, 32, generator=g)
    x[0, 5] = inf
    check_route(x, None, 4, "sigmoid")


def test_route_nan_in_masked_places():
    g = gen(6)
    for score in ("sigmoid", "softmax"):
        x = torch.randn(8, 64, generator=g)
        bias = torch.zeros(64)
        bias[::3] = -float("inf")
        x[:, ::3] = float("nan")
        x[2, ::3] = float("inf")
        check_route(x, bias, 8, score)
        check_route(x, bias, 8, score, groups=4, kept=2)
        bias += torch.randn(64, generator=g) * 0.1
        check_route(x, bias, 8, score, groups=4, kept=2)


@pytest.mark.parametrize("seed", range(24))
def test_route_random(seed):
    g = gen(100 + seed)
    pick = lambda *v: v[int(torch.randint(len(v), (1,), generator=g))]  # noqa: E731
    G = pick(1, 1, 2, 5, 8)
    E = G * pick(4, 9, 16, 33)
    kept = pick(*range(1, G + 1))
    k = pick(*range(1, min(12, kept * (E // G)) + 1))
    x = (torch.randn(pick(1, 4, 37), E, generator=g) * pick(0.3, 1.0, 6.0)).to(
        DT[pick("bf16", "fp16", "fp32")])
    check_route(x, make_bias(pick("none", "zero", "random", "masked", "lowest"), E, g), k,
                pick("sigmoid", "softmax"), groups=G, kept=kept, gscore=pick("max", "top2"),
                renorm=pick(True, False), scale=pick(1.0, 0.5))


# ------------------------------------------------------------------- layout

@pytest.mark.parametrize("T,k,E,first,lo,hi", [
    (1, 1, 1, 0, 0, 1), (1, 8, 256, 0, 0, 256), (16, 8, 256, 0, 0, 256), (127, 3, 60, 0, 0, 60),
    (512, 8, 64, 0, 0, 64), (513, 8, 64, 0, 0, 64),      # one block of threads, a cluster
    (3001, 7, 256, 0, 0, 256), (700, 8, 32, 64, 0, 256),  # local experts 64..95
    (700, 8, 32, 0, -1, 3), (900, 6, 1024, 0, 0, 1024), (5000, 4, 5, 2, 2, 3),
    (8192, 8, 17, 0, 20, 40),                             # no local expert at all
])
def test_plan(T, k, E, first, lo, hi):
    ids = torch.randint(lo, hi, (T, k), generator=gen(T), dtype=torch.int32)
    off = torch.full((E + 1,), -5, dtype=torch.int32, device="cuda")
    pos = torch.full((T, k), -5, dtype=torch.int32, device="cuda")
    B.ar_fusion_expert_plan(ids.cuda(), E, off, pos, first_expert=first)
    r_off, r_pos = R.plan(ids.numpy(), first, E)
    assert np.array_equal(off.cpu().numpy(), r_off)
    assert np.array_equal(pos.cpu().numpy(), r_pos)


@pytest.mark.parametrize("T,k,E", [(6144, 8, 256), (6145, 8, 256), (8193, 8, 256), (6700, 10, 1024),
                                   (16384, 8, 33), (16385, 8, 256), (100003, 5, 1000)])
def test_plan_of_many_slots(T, k, E):
    """Around the sizes where the cluster grows and where slots are loaded twice."""
    test_plan(T, k, E, 0, -1, E + 3)


def test_plan_of_no_tokens_writes_zero_offsets():
    off = torch.full((9,), -5, dtype=torch.int32, device="cuda")
    none = torch.empty(0, 4, dtype=torch.int32, device="cuda")
    B.ar_fusion_expert_plan(none, 8, off, none.clone())
    assert (off == 0).all()


# --------------------------------------------------------- block quantiser

def nearest_e4m3(v):
    """float32 values to E4M3 bytes: nearest even, saturating (numpy, by search)."""
    table = R.e4m3(np.arange(127))                     # 0 .. 448, ascending
    a = np.minimum(np.abs(v.astype(np.float64)), R.FP8_MAX)
    nan = np.isnan(a)
    a = np.where(nan, 0.0, a)
    hi = np.clip(np.searchsorted(table, a), 1, 126)
    lo = hi - 1
    up, down = table[hi] - a, a - table[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return np.where(nan, 0x7F, code | np.where(np.signbit(v), 0x80, 0)).astype(np.uint8)


def run_quant(x, hidden, act, position=None, out_rows=None, row_count=None, stream=None):
    out_rows = x.shape[0] if out_rows is None else out_rows
    q = torch.full((out_rows, hidden), 0xAA, dtype=torch.uint8, device="cuda")
    s = torch.full((out_rows, R.blocks(hidden)), -3.0, device="cuda")
    B.ar_fusion_quant_blocks(x.cuda(), q, s, position=position, row_count=row_count,
                             activation=B.AR_ACT_SILU_MUL if act else B.AR_ACT_NONE, stream=stream)
    torch.cuda.synchronize()
    return q.cpu().numpy(), s.cpu().numpy()


def check_quant_rows(q, s, x, hidden, act):
    y = R.activate(x, act)
    amax = R.block_amax(y)
    if not act:
        assert np.array_equal(s, amax.astype(np.float32) / np.float32(448))
        inv = np.float32(448) / amax.astype(np.float32)
        want = nearest_e4m3(y.astype(np.float32) * R.spread(inv, hidden))
        nan = (want & 0x7F) == 0x7F
        assert np.array_equal(q[~nan], want[~nan])
        assert ((q[nan] & 0x7F) == 0x7F).all()
        return
    assert (np.abs(s - amax / 448) <= 6 * U * amax / 448).all()
    wide = R.spread(s.astype(np.float64), hidden)
    err = np.abs(R.e4m3(q) * wide - y)
    assert (err <= np.maximum(np.abs(y) * 2.0 ** -4, wide * 2.0 ** -10) + 16 * U * np.abs(y)).all()


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("act", [False, True])
@pytest.mark.parametrize("rows,hidden", [(1, 16), (3, 128), (5, 144), (130, 512), (33, 7168),
                                         (2, 1936), (257, 112)])
def test_quant_blocks(dt, act, rows, hidden):
    g = gen(rows + hidden)
    x = torch.randn(rows, hidden * (2 if act else 1), generator=g)
    x[:, ::97] *= 40.0
    x[rows // 2] = 0.0
    x = x.to(DT[dt])
    q, s = run_quant(x, hidden, act)
    check_quant_rows(q, s, x, hidden, act)


def test_quant_blocks_special_values():
    g = gen(11)
    x = torch.randn(6, 256, generator=g)
    x[0, 3] = float("nan")
    x[0, 130:140] = float("nan")
    x[1] = 0.0
    x[2] *= 2.0 ** -110                     # below the floor of the amax
    x[3] = torch.finfo(torch.float32).max
    x[4, 128:] = 2.0 ** -149
    x[5, 7] = torch.finfo(torch.float32).min
    q, s = run_quant(x, 256, False)
    check_quant_rows(q, s, x, 256, False)
    y = torch.randn(1, 256, generator=g)
    y[0, 9] = float("inf")
    q, s = run_quant(y, 256, False)
    assert np.isinf(s[0, 0]) and (q[0, 9] & 0x7F) == 0x7F and np.isfinite(s[0, 1])
    assert ((np.delete(q[0, :128], 9) & 0x7F) == 0).all()
    # gates up to and beyond where e^-g leaves the fp32 range, in both directions
    far = torch.tensor([87.9, 88.0, 88.1, 88.72, 88.73, 89.0, 103.0, 104.0, 1e4, 3e38])
    w = torch.randn(4, 256, generator=g)
    w[0, :10], w[1, :10], w[2, 50:60] = -far, far, -far
    w[3, :128] = -88.5                       # a whole block of gates all but closed
    q, s = run_quant(w, 128, True)
    check_quant_rows(q, s, w, 128, True)
    w[1, 3], w[2, 4] = float("nan"), -float("inf")
    w[0, 5] = float("inf")
    q, s = run_quant(w, 128, True)
    assert (q[1, 3] & 0x7F) == 0x7F and (q[2, 4] & 0x7F) == 0x7F and np.isinf(s[0, 0])
    check_quant_rows(q[3:], s[3:], w[3:], 128, True)
    # a gate far below zero closes, without NaN
    z = torch.randn(2, 256, generator=g)
    z[:, :64] = -1000.0
    q, s = run_quant(z, 128, True)
    check_quant_rows(q, s, z, 128, True)


def test_quant_blocks_spread_copies_and_leaves_other_rows():
    g = gen(12)
    T, k, hidden, out_rows = 19, 4, 400, 90
    x = torch.randn(T, hidden, generator=g).to(torch.bfloat16)
    pos = torch.randperm(out_rows, generator=g)[:T * k].view(T, k).to(torch.int32)
    pos[3] = -1
    pos[4, 2] = out_rows                     # outside: skipped
    pos[5, 0] = 2 ** 31 - 1
    q, s = run_quant(x, hidden, False, position=pos.cuda(), out_rows=out_rows)
    one_q, one_s = run_quant(x, hidden, False)
    written = np.zeros(out_rows, bool)
    for t in range(T):
        for j in range(k):
            p = int(pos[t, j])
            if 0 <= p < out_rows:
                written[p] = True
                assert np.array_equal(q[p], one_q[t]) and np.array_equal(s[p], one_s[t])
    assert (q[~written] == 0xAA).all() and (s[~written] == -3.0).all()


@pytest.mark.parametrize("count", [-4, 0, 1, 20, 33, 1000])
def test_quant_blocks_row_count(count):
    x = torch.randn(33, 160, generator=gen(13)).to(torch.float16)
    q, s = run_quant(x, 160, False,
                     row_count=torch.tensor([count], dtype=torch.int32, device="cuda"))
    n = min(max(count, 0), 33)
    if n:
        check_quant_rows(q[:n], s[:n], x[:n], 160, False)
    assert (q[n:] == 0xAA).all() and (s[n:] == -3.0).all()


# ----------------------------------------------------------------- products

def codes(g, *shape):
    return (150.0 * torch.randn(shape, generator=g)).clamp(-448, 448).to(torch.float8_e4m3fn)


def scales(g, *shape):
    return 0.01 * torch.exp(0.5 * torch.randn(shape, generator=g))


def check_product(out, want, mags, blocks, dtype):
    got = out.double().cpu().numpy()
    tol = (256 + blocks + 4) * U * mags + R.half_step(dtype) * np.abs(want) + 2.0 ** -140
    if dtype == torch.float16:
        tol += 2.0 ** -25
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5])


PRODUCTS = [(1, 1, 16), (1, 128, 128), (2, 130, 272), (7, 64, 144), (16, 512, 2048), (17, 520, 400),
            (33, 257, 128), (64, 384, 640), (65, 1000, 1936), (100, 96, 48), (128, 256, 512),
            (129, 264, 1040), (200, 129, 256), (255, 640, 896), (300, 1288, 2064), (513, 392, 160),
            (1003, 520, 272)]


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,cols,depth", PRODUCTS)
def test_matmul(dt, rows, cols, depth):
    g = gen(rows * 7 + cols + depth)
    nb = R.blocks(depth)
    a, b = codes(g, rows, depth), codes(g, cols, depth)
    sa, sb = scales(g, rows, nb), scales(g, R.blocks(cols), nb)
    guard = torch.full((rows * cols + 64,), 77.0, dtype=DT[dt], device="cuda")
    out = guard[:rows * cols].view(rows, cols)
    B.ar_fusion_matmul_fp8(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), out)
    want, mags = R.matmul(a.view(torch.uint8).numpy(), sa.numpy(), b.view(torch.uint8).numpy(),
                          sb.numpy())
    check_product(out, want, mags, nb, DT[dt])
    assert (guard[rows * cols:] == 77.0).all()


# rows, columns and depths where 256 x 256 tiles of a pair of blocks are the faster
# kernel: several tiles per pair, rows and columns that end inside a tile, rows whose
# bytes are no multiple of 16, one block of the depth and a part of one
@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,cols,depth", [
    (1100, 1288, 656), (2000, 1027, 784), (700, 4104, 1040), (5200, 2312, 400),
    (2561, 3976, 128), (4095, 2049, 144), (1, 70000, 2064), (1024, 2048, 1152),
    (20000, 272, 128), (12000, 608, 64)])
def test_matmul_many_rows(dt, rows, cols, depth):
    test_matmul(dt, rows, cols, depth)


def test_matmul_status_is_clear():
    assert B.ar_fusion_matmul_status() == (B.AR_OK, -1)


def test_operands_that_are_not_contiguous_or_aligned_are_refused():
    z = lambda d, *s: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
    u8, f32 = torch.uint8, torch.float32
    a, sa, b, sb, out = z(u8, 64, 64), z(f32, 64, 1), z(u8, 64, 64), z(f32, 1, 1), z(f32, 64, 64)
    with pytest.raises(ValueError, match="contiguous"):
        B.ar_fusion_matmul_fp8(a.t(), sa, b, sb, out)
    with pytest.raises(ValueError, match="out: expected a contiguous"):
        B.ar_fusion_matmul_fp8(a, sa, b, sb, out.t())
    with pytest.raises(B.ArFusionError, match="aligned"):
        B.ar_fusion_matmul_fp8(z(u8, 64 * 64 + 8)[8:].view(64, 64), sa, b, sb, out)
    with pytest.raises(B.ArFusionError, match="multiple of 16"):
        B.ar_fusion_matmul_fp8(z(u8, 8, 40), z(f32, 8, 1), z(u8, 8, 40), sb, z(f32, 8, 8))
    with pytest.raises(ValueError, match="scale_out: shape"):
        B.ar_fusion_quant_blocks(z(f32, 4, 256), z(u8, 4, 256), z(f32, 4, 1))
    with pytest.raises(ValueError, match="CUDA"):
        B.ar_fusion_combine(z(f32, 4, 16), torch.zeros(2, 2, dtype=torch.int32), z(f32, 2, 2),
                            z(f32, 2, 16))


def test_matmul_nan_and_infinite_scales_stay_in_their_row():
    g = gen(21)
    for rows in (5, 200):
        a, b = codes(g, rows, 256), codes(g, 300, 256)
        sa, sb = scales(g, rows, 2), scales(g, 3, 2)
        byte = a.view(torch.uint8)
        byte[2, 7] = 0x7F
        sa[3, 1] = float("inf")
        out = torch.empty(rows, 300, dtype=torch.bfloat16, device="cuda")
        B.ar_fusion_matmul_fp8(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), out)
        clean = [r for r in range(rows) if r not in (2, 3)]
        want, mags = R.matmul(byte.numpy()[clean], sa.numpy()[clean], b.view(torch.uint8).numpy(),
                              sb.numpy())
        check_product(out[clean], want, mags, 2, torch.bfloat16)
        assert out[2].isnan().all() and not out[3].isfinite().any()


def check_experts(rows, cols, depth, bounds, dt, seed):
    """bounds: the offsets array as given to the call."""
    g = gen(seed)
    E, nb = len(bounds) - 1, R.blocks(depth)
    a, b = codes(g, rows, depth), codes(g, E, cols, depth)
    sa, sb = scales(g, rows, nb), scales(g, E, R.blocks(cols), nb)
    out = torch.full((rows, cols), 77.0, dtype=dt, device="cuda")
    B.ar_fusion_expert_matmul_fp8(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(),
                                  torch.tensor(bounds, dtype=torch.int32, device="cuda"), out)
    touched = np.zeros(rows, bool)
    ab, bb = a.view(torch.uint8).numpy(), b.view(torch.uint8).numpy()
    for e in range(E):
        lo = min(max(bounds[e], 0), rows)
        hi = min(max(bounds[e + 1], lo), rows)
        if hi > lo:
            touched[lo:hi] = True
            want, mags = R.matmul(ab[lo:hi], sa.numpy()[lo:hi], bb[e], sb.numpy()[e])
            check_product(out[lo:hi], want, mags, nb, dt)
    assert (out[torch.from_numpy(~touched).cuda()] == 77.0).all()


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("cols,depth,loads", [
    (128, 128, [1]), (136, 160, [0, 3, 0]), (256, 512, [5, 0, 17, 1, 0, 0, 40]),
    (520, 400, [1, 1, 1, 1, 1, 1, 1, 1]), (384, 256, [300, 0, 2, 129]), (200, 144, [0, 0, 0]),
    (264, 640, [64, 65, 63, 1, 200, 128, 127]), (1000, 272, [700, 1, 30]),
    (128, 256, [2] * 100), (256, 128, [0] * 40 + [500] + [3] * 9),
    # pairs of blocks: tiles that end at, before and behind an expert's last row
    (1288, 656, [300, 0, 2, 129, 500]), (1027, 784, [256, 255, 257, 1, 0, 512]),
    (2312, 1040, [900, 130, 31, 33, 700])])
def test_expert_matmul(dt, cols, depth, loads):
    bounds = np.concatenate([[0], np.cumsum(loads)]).tolist()
    rows = bounds[-1] + 9                    # rows behind the last expert stay as they were
    check_experts(rows, cols, depth, bounds, DT[dt], sum(loads) + cols)


def test_expert_matmul_first_offset_above_zero_and_clamped_offsets():
    check_experts(70, 136, 144, [10, 20, 20, 55], torch.bfloat16, 1)
    check_experts(70, 136, 144, [-30, 20, 65, 9000], torch.bfloat16, 2)
    check_experts(300, 136, 144, [-30, 200, 250, 2 ** 31 - 1], torch.float32, 3)


def test_expert_matmul_of_many_experts_and_columns():
    """Weights past half of L2 in more blocks than six per SM; experts of none,
    one and several tiles of rows."""
    loads = [0, 1, 3, 16, 17, 40] + [1, 0, 2] * 9
    bounds = np.concatenate([[0], np.cumsum(loads)]).tolist()
    check_experts(bounds[-1] + 2, 4104, 528, bounds, torch.float32, 77)
    check_experts(5, 32776, 2064, [0, 5], torch.bfloat16, 78)


# ------------------------------------------------------------------ combine

@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("T,k,hidden", [(1, 1, 8), (5, 8, 1000), (33, 3, 7168), (7, 13, 264),
                                        (129, 6, 512)])
def test_combine(dt, add, T, k, hidden):
    g = gen(T + k)
    n = T * k + 3
    rows = torch.randn(n, hidden, generator=g).to(DT[dt])
    pos = torch.randperm(n, generator=g)[:T * k].view(T, k).to(torch.int32)
    pos[T // 2] = -1                          # a token that has no row
    if T > 3:
        pos[0, k - 1] = n                     # outside
        pos[1, 0] = -2 ** 31
        pos[2, 0] = pos[3, 0]                 # one row of two tokens
    w = torch.rand(T, k, generator=g) - 0.3
    base = torch.randn(T, hidden, generator=g).to(DT[dt]) if add else None
    out = torch.full((T, hidden), float("nan"), dtype=DT[dt], device="cuda")
    B.ar_fusion_combine(rows.cuda(), pos.cuda(), w.cuda(), out,
                        add=None if base is None else base.cuda())
    want, mags = R.combine(rows, pos, w, base)
    tol = (k + 1) * U * mags + R.half_step(DT[dt]) * np.abs(want) + 2.0 ** -25 * (dt == "fp16")
    assert (np.abs(out.double().cpu().numpy() - want) <= tol).all()


def test_combine_skips_rows_that_no_slot_names():
    rows = torch.full((4, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    rows[2] = 3.0
    pos = torch.tensor([[2, -1], [-1, -1]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[0.5, float("nan")], [float("inf"), 1.0]], device="cuda")
    out = torch.empty(2, 64, dtype=torch.bfloat16, device="cuda")
    B.ar_fusion_combine(rows, pos, w, out)
    assert (out[0] == 1.5).all() and (out[1] == 0.0).all()


def test_empty_calls_launch_nothing():
    e = lambda *s, d=torch.float32: torch.empty(*s, dtype=d, device="cuda")  # noqa: E731
    i32 = torch.int32
    B.ar_fusion_route(e(0, 8), None, e(0, 2, d=i32), e(0, 2))
    B.ar_fusion_quant_blocks(e(0, 32), e(0, 32, d=torch.uint8), e(0, 1))
    B.ar_fusion_matmul_fp8(e(0, 32, d=torch.uint8), e(0, 1), e(5, 32, d=torch.uint8), e(1, 1),
                           e(0, 5))
    B.ar_fusion_combine(e(0, 16), e(0, 2, d=i32), e(0, 2), e(0, 16))
    torch.cuda.synchronize()


# ------------------------------------------------------- used as one layer

class Layer:
    """One expert layer on random weights: routing, layout, quantisation, both
    products with the activation between them, and the combination into a
    rank's partial of the fused epilogue."""

    def __init__(self, T, H, I, E, k, first, local, seed):
        g = gen(seed)
        self.dims = T, H, I, E, k, first, local
        c = lambda t: t.cuda()  # noqa: E731
        self.x = c(torch.randn(T, H, generator=g).to(torch.bfloat16))
        self.logits = c(torch.randn(T, E, generator=g))
        self.bias = c(0.1 * torch.randn(E, generator=g))
        self.w1, self.s1 = c(codes(g, local, 2 * I, H)), c(
            3e-4 * torch.exp(0.3 * torch.randn(local, R.blocks(2 * I), R.blocks(H), generator=g)))
        self.w2, self.s2 = c(codes(g, local, H, I)), c(
            3e-4 * torch.exp(0.3 * torch.randn(local, R.blocks(H), R.blocks(I), generator=g)))
        rows = T * k
        f32, i32, u8, bf = torch.float32, torch.int32, torch.uint8, torch.bfloat16
        z = lambda d, *s: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
        self.ids, self.w = z(i32, T, k), z(f32, T, k)
        self.off, self.pos = z(i32, local + 1), z(i32, T, k)
        self.q, self.qs = z(u8, rows, H), z(f32, rows, R.blocks(H))
        self.h = z(bf, rows, 2 * I)
        self.hq, self.hs = z(u8, rows, I), z(f32, rows, R.blocks(I))
        self.y = z(bf, rows, H)
        self.out = z(bf, T, H)

    def run(self, stream=None):
        first, local = self.dims[5:]
        B.ar_fusion_route(self.logits, self.bias, self.ids, self.w, groups=4, groups_kept=2,
                          scale=2.5, stream=stream)
        B.ar_fusion_expert_plan(self.ids, local, self.off, self.pos, first_expert=first,
                                stream=stream)
        B.ar_fusion_quant_blocks(self.x, self.q, self.qs, position=self.pos, stream=stream)
        B.ar_fusion_expert_matmul_fp8(self.q, self.qs, self.w1, self.s1, self.off, self.h,
                                      stream=stream)
        B.ar_fusion_quant_blocks(self.h, self.hq, self.hs, activation=B.AR_ACT_SILU_MUL,
                                 row_count=self.off[-1:], stream=stream)
        B.ar_fusion_expert_matmul_fp8(self.hq, self.hs, self.w2, self.s2, self.off, self.y,
                                      stream=stream)
        B.ar_fusion_combine(self.y, self.pos, self.w, self.out, stream=stream)

    def check(self):
        T, H, I, E, k, first, local = self.dims
        ids, w = R.route(self.logits, self.bias, k, "sigmoid", 4, 2, "top2", True, 2.5)
        assert np.array_equal(self.ids.cpu().numpy(), ids)
        assert (np.abs(self.w.cpu().double().numpy() - w) <= 40 * U * np.abs(w)).all()
        off, pos = R.plan(ids, first, local)
        assert np.array_equal(self.off.cpu().numpy(), off)
        assert np.array_equal(self.pos.cpu().numpy(), pos)
        n = int(off[-1])
        row_token = np.zeros(n, dtype=np.int64)
        for t in range(T):
            for j in range(k):
                if pos[t, j] >= 0:
                    row_token[pos[t, j]] = t
        q, qs = self.q.cpu().numpy(), self.qs.cpu().numpy()
        check_quant_rows(q[:n], qs[:n], self.x.cpu()[row_token], H, False)
        hq, hs = self.hq.cpu().numpy(), self.hs.cpu().numpy()
        check_quant_rows(hq[:n], hs[:n], self.h.cpu()[:n], I, True)
        for e in range(local):
            lo, hi = int(off[e]), int(off[e + 1])
            if hi == lo:
                continue
            for src, ss, wt, ws, dst in ((q, qs, self.w1, self.s1, self.h),
                                         (hq, hs, self.w2, self.s2, self.y)):
                want, mags = R.matmul(src[lo:hi], ss[lo:hi], wt[e].view(torch.uint8).cpu().numpy(),
                                      ws[e].cpu().numpy())
                check_product(dst[lo:hi], want, mags, ss.shape[1], torch.bfloat16)
        want, mags = R.combine(self.y, self.pos, self.w, None)
        tol = (k + 1) * U * mags + R.half_step(torch.bfloat16) * np.abs(want)
        assert (np.abs(self.out.double().cpu().numpy() - want) <= tol).all()


@pytest.mark.parametrize("T", [1, 5, 150])
def test_layer_into_the_fused_epilogue(T):
    """Two ranks' halves of the experts, each run as a layer; their outputs are
    the partials of the fused call, whose result matches the oracle's."""
    H, E = 512, 64
    ranks = [Layer(T, H, 256, E, 6, first, 32, seed=7) for first in (0, 32)]
    ranks[1].w1, ranks[1].w2 = (w.view(torch.uint8).roll(1, 0) for w in (ranks[1].w1, ranks[1].w2))
    for r in ranks:
        r.run()
    torch.cuda.synchronize()
    for r in ranks:
        r.check()
    gamma = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    res, nrm = torch.empty_like(ranks[0].x), torch.empty_like(ranks[0].x)
    ws = B.ar_fusion_workspace_create(2, max(T, 16), H, B.AR_DT_BF16)
    B.ar_fusion_run(ws, [r.out for r in ranks], ranks[0].x, gamma, 1e-6, B.PATTERNS["res_norm"],
                    residual_out=res, norm_out=nrm)
    torch.cuda.synchronize()
    o_res, _, _ = oracle.fused(oracle.BF16, W.bits(torch.stack([r.out.cpu() for r in ranks])),
                               W.bits(ranks[0].x.cpu()), W.bits(gamma.cpu()), 1e-6)
    assert np.array_equal(W.bits(res.cpu()), o_res)
    B.ar_fusion_workspace_destroy(ws)


def test_dense_product_writes_a_partial_of_the_workspace():
    g = gen(31)
    T, H, K = 200, 640, 256
    ws = B.ar_fusion_workspace_create(2, T, H, B.AR_DT_BF16)
    parts = []
    for r in range(2):
        a, b = codes(g, T, K), codes(g, H, K)
        sa, sb = scales(g, T, 2), 1e-3 * scales(g, R.blocks(H), 2)
        out = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
        dev = [t.cuda() for t in (a, sa, b, sb)]
        B.ar_fusion_matmul_fp8(*dev, out)
        to = B.ar_fusion_workspace_partial_ptr(ws, r, T, B.AR_MODE_BUFFER)
        L = B.lib()
        assert L.ar_fusion_matmul_fp8(dev[0].data_ptr(), dev[1].data_ptr(), dev[2].data_ptr(),
                                      dev[3].data_ptr(), T, H, K, B.AR_DT_BF16, to, None) == B.AR_OK
        torch.cuda.synchronize()
        parts.append(out)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
    gamma = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    got, want = torch.empty_like(x), torch.empty_like(x)
    B.ar_fusion_workspace_set_mode(ws, B.AR_MODE_BUFFER)
    B.ar_fusion_run(ws, None, x, gamma, 1e-6, B.AR_NORM_OUT, norm_out=got)
    B.ar_fusion_run(ws, parts, x, gamma, 1e-6, B.AR_NORM_OUT, norm_out=want)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    B.ar_fusion_workspace_destroy(ws)


def test_layer_captured_and_replayed_on_new_inputs():
    layer = Layer(20, 512, 256, 64, 6, 0, 64, seed=9)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer.run()                          # once uncaptured
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            layer.run()
    g = gen(10)
    for _ in range(3):
        layer.logits.copy_(torch.randn(layer.logits.shape, generator=g))
        layer.x.copy_(torch.randn(layer.x.shape, generator=g).to(torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        layer.check()


def test_layers_on_two_streams_at_once():
    layers = [Layer(40 + 60 * i, 512, 256, 32, 6, 0, 32, seed=20 + i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in layers]
    torch.cuda.synchronize()
    for _ in range(5):
        for layer, s in zip(layers, streams):
            layer.run(stream=s)
    torch.cuda.synchronize()
    for layer in layers:
        layer.check()


@pytest.mark.parametrize("native", [True, False])
def test_marshalling_in_c_and_through_ctypes(native, monkeypatch):
    """The same calls with the C++ marshalling and without it; optional operands,
    another stream, and refusals that both answer alike."""
    if native and B._native is None:
        pytest.skip("marshal.cpp was not built")
    if not native:
        monkeypatch.setattr(B, "_native", None)
    layer = Layer(33, 512, 256, 32, 6, 8, 16, seed=50)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    layer.run(stream=s)
    s.synchronize()
    layer.check()
    layer.run()
    torch.cuda.synchronize()
    layer.check()
    add = layer.x.clone()
    B.ar_fusion_combine(layer.y, layer.pos, layer.w, layer.out, add=add)
    want, mags = R.combine(layer.y, layer.pos, layer.w, add)
    tol = 8 * U * mags + R.half_step(torch.bfloat16) * np.abs(want)
    assert (np.abs(layer.out.double().cpu().numpy() - want) <= tol).all()
    a, sa = layer.q.view(torch.float8_e4m3fn), layer.qs
    out = torch.empty(a.shape[0], 512, dtype=torch.float16, device="cuda")
    B.ar_fusion_matmul_fp8(a, sa, layer.w1[0], layer.s1[0], out, stream=s.cuda_stream)
    s.synchronize()
    with pytest.raises(ValueError, match="b: shape"):
        B.ar_fusion_matmul_fp8(a, sa, layer.w1[0][:, :64], layer.s1[0], out)
    with pytest.raises(TypeError, match="out"):
        B.ar_fusion_matmul_fp8(a, sa, layer.w1[0], layer.s1[0], out.double())
    with pytest.raises(TypeError, match="offsets"):
        B.ar_fusion_expert_matmul_fp8(a, sa, layer.w1, layer.s1, layer.off.long(), layer.h)
    with pytest.raises(ValueError, match="ids: 1 dimensions"):
        B.ar_fusion_expert_plan(layer.ids.view(-1), 16, layer.off, layer.pos)
    with pytest.raises(B.ArFusionError, match="groups"):
        B.ar_fusion_route(layer.logits, layer.bias, layer.ids, layer.w, groups=5)
    with pytest.raises(B.ArFusionError, match="score"):
        B.ar_fusion_route(layer.logits, layer.bias, layer.ids, layer.w, score=7, scale=1)
    with pytest.raises(ValueError, match="row_count"):
        B.ar_fusion_quant_blocks(layer.x, layer.q[:33], layer.qs[:33], row_count=layer.off)


@pytest.mark.parametrize("native", [True, False])
def test_numbers_past_32_bits_are_refused(native, monkeypatch):
    B.load()
    if not native:
        monkeypatch.setattr(B, "_native", None)
    layer = Layer(3, 128, 128, 32, 6, 8, 16, seed=51)
    with pytest.raises(ValueError, match="32-bit"):
        B.ar_fusion_expert_plan(layer.ids, 16, layer.off, layer.pos, first_expert=1 << 32)
    with pytest.raises(ValueError, match="32-bit"):
        B.ar_fusion_route(layer.logits, layer.bias, layer.ids, layer.w, groups=(1 << 32) + 1)


def test_same_inputs_give_the_same_bits():
    a, b = (Layer(150, 512, 256, 32, 6, 0, 32, seed=40) for _ in range(2))
    a.run()
    b.run()
    torch.cuda.synchronize()
    assert torch.equal(a.out, b.out) and torch.equal(a.hq, b.hq) and torch.equal(a.w, b.w)
