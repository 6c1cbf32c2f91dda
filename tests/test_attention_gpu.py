"""The attention-layer calls against 64-bit arithmetic: rotation and append, attention of
one new token per sequence, attention of prompts."""
import math

import pytest
import torch

import attention_ref as R
from allreduce_residual_rmsnorm_gb300 import binding as B

pytestmark = pytest.mark.gpu
BF16, FP16, E4M3 = torch.bfloat16, torch.float16, torch.float8_e4m3fn
U = R.U
# of a fp16 weight, next to a largest one taken as 1, by the calls' contract
LOST_ONE, LOST_PROMPT = 2.0 ** -39, 2.0 ** -30


@pytest.fixture(scope="module")
def workspace(cuda_lib):
    return torch.empty(B.AR_ATTENTION_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


# --------------------------------------------------------- rotation, append

def check_append(new, lengths, P, H, K, D, rot, dtype, cache_dtype, interleaved=False, sections=None,
                 positions=None, hnd=False, in_place=False, first=0, behind=0, no_starts=False,
                 seed=1):
    """first: rows before the first sequence, behind: rows behind the last one."""
    pages = R.Pages(lengths, P, K, D, cache_dtype, seed=seed, hnd=hnd, junk=False)
    T = first + sum(new) + behind
    starts = torch.tensor([first + sum(new[:b]) for b in range(len(new) + 1)], dtype=torch.int32)
    g = gen(seed + 1)
    qkv = torch.randn(T, H + 2 * K, D, generator=g).to(dtype)
    q, k, v = qkv[:, :H], qkv[:, H:H + K], qkv[:, H + K:]
    f = 1e4 ** (-torch.arange(0, rot, 2) / max(rot, 1))
    axes = 1 if sections is None else len(sections)
    kc, vc, table, dev_lengths, scale = pages.cuda()
    want_k, want_v = (pages.view(t).float().double() for t in (pages.k, pages.v))
    d = qkv.cuda()
    dq = d[:, :H]
    q_out = dq if in_place else torch.full((T, H, D), 7.0, dtype=dtype, device="cuda")
    B.ar_fusion_rope_append(
        dq, d[:, H:H + K], d[:, H + K:], kc, vc, table, dev_lengths, f.cuda() if rot else None,
        None if in_place else q_out, starts=None if no_starts else starts.cuda(),
        positions=None if positions is None else positions.cuda(), sections=sections,
        interleaved=interleaved, kv_scale=scale)
    torch.cuda.synchronize()
    index = torch.full((T,), -(1 << 30))
    seq = torch.full((T,), -1)
    for row, b, i in R.rows_of(starts, lengths, T, table.shape[1] * P):
        index[row], seq[row] = i, b
    where = index[None].expand(axes, T) if positions is None else positions.reshape(axes, T)
    axis_of = [x for x, n in enumerate(sections or (rot // 2,)) for _ in range(n)]
    live = seq >= 0
    want_q = torch.full((T, H, D), 7.0, dtype=torch.float64) if not in_place else q.double().clone()
    want_q[live] = R.turn(q.double(), where, f, axis_of, interleaved)[live]
    turned = R.turn(k.double(), where, f, axis_of, interleaved)
    # cos and sin: half-turns off by 4 U at most, times pi, and 2 U of their own; two products
    # and a sum.  Of the larger of the pair's two elements.
    span = (x.double().abs().amax(-1, keepdim=True) for x in (q, k))
    sq, sk = (24 * U * s if rot else 0 * s for s in span)
    tol_q = sq + R.half_step(dtype) * want_q.abs() + (2.0 ** -25 if dtype == FP16 else 0.0)
    got_q = q_out.double().cpu()
    assert bool(((got_q - want_q).abs() <= tol_q).all()), (got_q - want_q).abs().amax()
    assert torch.equal(got_q[~live], want_q[~live])
    tol_k, tol_v = torch.zeros_like(want_k), torch.zeros_like(want_v)
    half = R.half_step(cache_dtype) if cache_dtype != E4M3 else 2.0 ** -4
    # below the normal range half a step is a fixed number
    least = {BF16: 2.0 ** -134, FP16: 2.0 ** -25, E4M3: 2.0 ** -10}[cache_dtype]
    for row in range(T):
        if not live[row] or index[row] < 0:
            continue
        p = int(pages.table[seq[row], index[row] // P])
        if not 0 <= p < kc.shape[0]:
            continue
        at = int(index[row]) % P
        for want, tol, x, near, s in ((want_k, tol_k, turned[row], sk[row], pages.scales[0]),
                                      (want_v, tol_v, v[row].double(), 0.0, pages.scales[1])):
            y = x / s
            want[p, at] = y.clamp(-448, 448) if cache_dtype == E4M3 else y
            tol[p, at] = (near + 3 * U * x.abs()) / s + half * want[p, at].abs() + least
    for got, want, tol in ((kc, want_k, tol_k), (vc, want_v, tol_v)):
        off = (got.float().cpu().double() - want).abs()
        assert bool((off <= tol).all()), (off - tol).amax()
    return q_out, kc, vc


@pytest.mark.parametrize("dtype,cache", [(BF16, BF16), (FP16, FP16), (BF16, E4M3), (FP16, E4M3)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot,H,K", [(128, 128, 8, 1), (128, 64, 32, 8), (80, 64, 15, 5), (64, 64, 3, 3),
                                       (16, 16, 2, 1), (112, 0, 5, 5), (96, 16, 70, 2)])
def test_append(cuda_lib, D, rot, H, K, interleaved, dtype, cache):
    check_append([1, 3, 0, 130, 1], [1, 5, 9, 200, 64], 16, H, K, D, rot, dtype, cache, interleaved)


def test_append_heads_of_8_elements_and_24(cuda_lib):
    check_append([2, 3], [2, 30], 8, 4, 2, 8, 0, BF16, BF16)
    check_append([2, 3], [2, 30], 8, 4, 2, 24, 16, FP16, FP16, True)


@pytest.mark.parametrize("kw", [
    dict(hnd=True), dict(in_place=True), dict(first=3, behind=5), dict(in_place=True, behind=2),
    dict(no_starts=True)], ids=str)
def test_append_forms(cuda_lib, kw):
    new = [1] * 5 if kw.get("no_starts") else [4, 0, 1, 7, 33]
    check_append(new, [40, 12, 1, 300, 33], 32, 8, 2, 128, 128, BF16, BF16, **kw)


def test_append_rows_without_a_place(cuda_lib):
    # more rows than the sequence holds, lengths of nothing and below, an entry of no page
    check_append([5, 2, 3], [3, 0, -4], 8, 4, 2, 64, 64, BF16, BF16)
    pages = R.Pages([20], 8, 2, 64, BF16, junk=False)
    kc, vc, table, lengths, _ = pages.cuda()
    before = kc.clone()
    table[0, 1] = 1 << 20
    d = torch.randn(20, 2, 64, device="cuda").to(BF16)
    B.ar_fusion_rope_append(None, d, d, kc, vc, table, lengths, None,
                            starts=torch.tensor([0, 20], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    at = pages.table[0].tolist()
    assert torch.equal(kc[at[0]], d[:8]) and torch.equal(vc[at[2], :4], d[16:])
    untouched = [p for p in range(kc.shape[0]) if p not in (at[0], at[2])]
    assert torch.equal(kc[untouched], before[untouched])


@pytest.mark.parametrize("axes", [(8, 12, 12), (0, 32), (32, 0, 0, 0), (5, 9, 11, 7)])
def test_append_axes(cuda_lib, axes):
    g = gen(4)
    T = 37
    where = torch.randint(0, 1 << 20, (len(axes), T), generator=g, dtype=torch.int32)
    for interleaved in (False, True):
        check_append([30, 7], [50, 7], 16, 6, 2, 96, 64, FP16, FP16, interleaved, sections=axes,
                     positions=where)


@pytest.mark.parametrize("far", [4095, 4096, 1 << 20, (1 << 24) + 1, (1 << 31) - 1, -1, -70000])
def test_append_far_positions(cuda_lib, far):
    where = torch.tensor([far, far // 2, far // 3 * 2], dtype=torch.int32)
    check_append([3], [3], 16, 2, 1, 128, 128, FP16, FP16, positions=where)


def test_append_many_sequences(cuda_lib):
    g = gen(9)
    new = torch.randint(0, 3, (700,), generator=g).tolist()
    check_append(new, [n + 3 for n in new], 8, 2, 1, 64, 64, BF16, BF16)
    check_append([1] * 2048, [1 + b % 9 for b in range(2048)], 16, 1, 1, 16, 16, BF16, BF16)


# --------------------------------------------------- one token per sequence

def check_decode(lengths, P, H, K, D, dtype, cache_dtype, workspace, window=0, sinks=0, scale=None,
                 hnd=False, seed=3, lse=True, factor=1.0, table=None, q=None, touch=None):
    pages = R.Pages(lengths, P, K, D, cache_dtype, seed=seed, hnd=hnd, extra=1)
    S = len(lengths)
    if table is not None:
        table(pages.table)
    if touch is not None:
        touch(pages)
    if q is None:
        q = (factor * torch.randn(S, H + 3, D, generator=gen(seed + 1))).to(dtype)[:, 1:H + 1]
    kc, vc, dev_table, dev_lengths, kv_scale = pages.cuda()
    out = torch.full((S + 1, H, D + 8), 5.0, dtype=dtype, device="cuda")
    L = torch.full((S, H), 5.0, device="cuda") if lse else None
    dq = q.cuda() if q.is_contiguous() else torch.zeros(S, H + 3, D, dtype=dtype, device="cuda")[:, 1:H + 1]
    dq.copy_(q)
    if workspace is not None:
        workspace.fill_(255)                        # NaN: nothing of an earlier call is read
    B.ar_fusion_decode_attention(dq, kc, vc, dev_table, dev_lengths, out[:S, :, :D], workspace,
                                 scale=scale, window=window, sinks=sinks, lse=L, kv_scale=kv_scale)
    torch.cuda.synchronize()
    want = R.attention(q, pages.view(pages.k), pages.view(pages.v), pages.table, pages.lengths,
                       list(range(S + 1)), D ** -0.5 if scale is None else scale, window, sinks,
                       pages.scales)
    R.check_attention(out[:S, :, :D], L, want, dtype, FP16 if cache_dtype == E4M3 else dtype,
                      LOST_ONE, splits=40)
    assert bool((out[S] == 5.0).all()) and bool((out[:, :, D:] == 5.0).all())
    return out[:S, :, :D], L


KINDS = [(BF16, BF16), (FP16, FP16), (BF16, E4M3), (FP16, E4M3)]
LENGTHS = [1, 0, 7, 16, 17, 64, 65, 300, 1000, 2, 129, -5]


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("H,K,D", [(8, 1, 128), (8, 8, 128), (14, 2, 64), (15, 3, 80), (40, 2, 96),
                                   (16, 1, 16), (33, 1, 128)])
def test_decode(workspace, H, K, D, dtype, cache):
    check_decode(LENGTHS, 16, H, K, D, dtype, cache, workspace)


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (16, 0), (33, 16), (100, 17), (64, 500), (5000, 4)])
def test_decode_window(workspace, window, sinks, dtype, cache):
    check_decode(LENGTHS + [2000, 513], 32, 8, 2, 128, dtype, cache, workspace, window, sinks)


@pytest.mark.parametrize("P", [8, 64, 1024])
@pytest.mark.parametrize("hnd", [False, True])
def test_decode_layouts(workspace, P, hnd):
    for dtype, cache in KINDS:
        check_decode(LENGTHS, P, 12, 3, 64, dtype, cache, workspace, hnd=hnd)
        check_decode(LENGTHS, P, 12, 3, 112, dtype, cache, workspace, window=90, sinks=3, hnd=hnd)


def test_decode_small_heads(workspace):
    for D in (8, 24, 40, 72, 104, 120):
        check_decode([5, 100, 33], 16, 4, 2, D, BF16, BF16, workspace)


@pytest.mark.parametrize("dtype,cache", KINDS)
def test_decode_long_and_split(workspace, dtype, cache):
    check_decode([30011], 64, 8, 1, 128, dtype, cache, workspace)
    check_decode([9000, 3, 20000], 64, 4, 2, 64, dtype, cache, workspace)


def test_decode_many_sequences(workspace):
    g = gen(8)
    for S in (129, 600):
        lengths = torch.randint(0, 90, (S,), generator=g).tolist()
        check_decode(lengths, 16, 4, 2, 64, BF16, BF16, workspace)
    check_decode([1 + b % 3 for b in range(2048)], 8, 1, 1, 16, BF16, BF16, workspace)
    check_decode([0] * 50, 8, 2, 1, 64, BF16, BF16, workspace)


@pytest.mark.parametrize("nbytes", [0, 16, 100_000, 3_000_000])
def test_decode_with_less_workspace(cuda_lib, nbytes):
    work = torch.empty(nbytes, dtype=torch.uint8, device="cuda") if nbytes else None
    check_decode([5000, 0, 1, 700, 64], 16, 8, 2, 128, BF16, BF16, work)
    g = gen(2)
    check_decode(torch.randint(0, 400, (300,), generator=g).tolist(), 16, 6, 3, 64, FP16, FP16, work)


def test_decode_scores_far_apart(workspace):
    """Weights from 1 down to nothing, large negative scores first, and a scale of the user's."""
    check_decode([700, 33], 16, 8, 2, 128, BF16, BF16, workspace, factor=20.0)
    check_decode([700, 33], 16, 8, 2, 128, FP16, E4M3, workspace, factor=20.0)
    check_decode([700, 33], 16, 8, 2, 128, BF16, E4M3, workspace, factor=2.0 ** -70, scale=2.0 ** 60)
    check_decode([700, 33], 16, 8, 2, 128, BF16, E4M3, workspace, factor=2.0 ** 60, scale=2.0 ** -62)
    check_decode([700, 33], 16, 8, 2, 64, BF16, BF16, workspace, scale=1.0)
    check_decode([700, 33], 16, 8, 2, 64, BF16, BF16, workspace, factor=0.0)


def test_decode_entries_of_no_page_read_as_zeros(workspace):
    def some(table):
        table[0, 1], table[0, 3], table[1, 0] = -1, 1 << 29, -(1 << 31)
    for dtype, cache in KINDS:
        check_decode([100, 20, 50], 16, 8, 2, 128, dtype, cache, workspace, table=some)


def test_decode_lengths_past_the_table(workspace):
    pages = R.Pages([64], 16, 2, 64, BF16)
    kc, vc, table, lengths, _ = pages.cuda()
    q = torch.randn(1, 4, 64).to(BF16)
    out = [torch.empty(1, 4, 64, dtype=BF16, device="cuda") for _ in range(2)]
    for o, n in zip(out, (64, 1 << 30)):
        B.ar_fusion_decode_attention(q.cuda(), kc, vc, table,
                                     torch.tensor([n], dtype=torch.int32, device="cuda"), o, workspace)
    assert torch.equal(*out)


def test_decode_same_bits_again(workspace):
    a = check_decode([5000, 300, 9000], 16, 8, 2, 128, BF16, BF16, workspace)
    for _ in range(3):
        b = check_decode([5000, 300, 9000], 16, 8, 2, 128, BF16, BF16, workspace)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ------------------------------------------------------------------ prompts

def check_prompt(new, lengths, P, H, K, D, dtype, workspace, window=0, sinks=0, scale=None, hnd=False,
                 seed=5, lse=True, factor=1.0, table=None, first=0, behind=0, cache=None, touch=None):
    pages = R.Pages(lengths, P, K, D, cache or dtype, seed=seed, hnd=hnd, extra=1)
    if table is not None:
        table(pages.table)
    if touch is not None:
        touch(pages)
    T = first + sum(new) + behind
    starts = torch.tensor([first + sum(new[:b]) for b in range(len(new) + 1)], dtype=torch.int32)
    q = (factor * torch.randn(T, H + 2 * K, D, generator=gen(seed + 1))).to(dtype)
    dq = q.cuda()[:, :H]
    q = q[:, :H]
    kc, vc, dev_table, dev_lengths, kv_scale = pages.cuda()
    out = torch.full((T, H, D + 8), 5.0, dtype=dtype, device="cuda")
    L = torch.full((T, H), 5.0, device="cuda") if lse else None
    if workspace is not None:
        workspace.fill_(255)
    B.ar_fusion_prompt_attention(dq, kc, vc, dev_table, dev_lengths, starts.cuda(), out[:, :, :D],
                                 workspace, scale=scale, window=window, sinks=sinks, lse=L, kv_scale=kv_scale)
    torch.cuda.synchronize()
    assert B.ar_fusion_attention_status() == (B.AR_OK, -1)
    want = R.attention(q, pages.view(pages.k), pages.view(pages.v), pages.table, pages.lengths,
                       starts, D ** -0.5 if scale is None else scale, window, sinks, pages.scales)
    R.check_attention(out[:, :, :D], L, want, dtype, dtype, LOST_PROMPT, splits=40)
    dead = torch.isnan(want[4][:, 0])
    assert bool((out[:, :, D:] == 5.0).all()) and bool((out.cpu()[dead] == 5.0).all())
    if lse:
        assert bool((L.cpu()[dead] == 5.0).all())
    return out[:, :, :D], L


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("H,K,D", [(8, 1, 128), (8, 8, 128), (14, 2, 64), (15, 3, 80), (40, 2, 96),
                                   (16, 1, 16), (33, 1, 128), (128, 1, 64)])
def test_prompt(workspace, H, K, D, dtype):
    check_prompt([1, 0, 5, 64, 130, 33], [1, 4, 300, 64, 130, 200], 16, H, K, D, dtype, workspace)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("H,K,D", [(8, 1, 128), (8, 8, 128), (14, 2, 64), (15, 3, 80), (40, 2, 96),
                                   (16, 1, 16), (33, 1, 128), (128, 1, 64)])
def test_prompt_e4m3(workspace, H, K, D, dtype):
    check_prompt([1, 0, 5, 64, 130, 33], [1, 4, 300, 64, 130, 200], 16, H, K, D, dtype, workspace,
                 cache=E4M3)
    check_prompt([70, 40], [300, 900], 8, H, K, D, dtype, workspace, 100, 9, hnd=True, cache=E4M3)
    check_prompt([3, 100, 9], [5, 90, 3000], 128, H, K, D, dtype, None, cache=E4M3, behind=2)


def test_prompt_e4m3_long_and_bad_pages(workspace):
    def some(table):
        table[0, 1], table[0, 3], table[1, 0] = -1, 1 << 29, -(1 << 31)
    for dtype in (BF16, FP16):
        check_prompt([100, 20, 2], [100, 20, 50], 16, 8, 2, 128, dtype, workspace, table=some, cache=E4M3)
        check_prompt([3], [9011], 64, 8, 1, 128, dtype, workspace, cache=E4M3)
        check_prompt([700], [1500], 64, 2, 1, 64, dtype, workspace, factor=20.0, cache=E4M3)
        check_prompt([600], [600], 64, 6, 3, 64, dtype, workspace, 1024, 0, cache=E4M3)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (16, 0), (33, 16), (100, 17), (64, 500),
                                          (128, 0), (129, 128), (5000, 4)])
def test_prompt_window(workspace, window, sinks):
    for dtype in (BF16, FP16):
        check_prompt([300, 1, 77, 40], [300, 500, 400, 1000], 32, 8, 2, 128, dtype, workspace, window,
                     sinks)


@pytest.mark.parametrize("P", [8, 64, 128, 1024])
@pytest.mark.parametrize("hnd", [False, True])
def test_prompt_layouts(workspace, P, hnd):
    check_prompt([100, 20], [260, 20], P, 6, 3, 64, BF16, workspace, hnd=hnd)
    check_prompt([100, 20], [260, 20], P, 6, 3, 112, FP16, workspace, 90, 3, hnd=hnd)


def test_prompt_small_heads(workspace):
    for D in (8, 24, 40, 72, 104, 120):
        check_prompt([20, 3], [33, 140], 16, 4, 2, D, BF16, workspace)


def test_prompt_rows_outside_and_without_keys(workspace):
    check_prompt([10, 3, 20], [4, 0, -3], 16, 4, 2, 64, BF16, workspace, first=3, behind=9)
    check_prompt([200, 0, 20], [150, 9, 20], 16, 4, 1, 128, FP16, workspace, behind=1)
    check_prompt([200, 0, 20], [150, 9, 20], 16, 4, 1, 128, FP16, workspace, 20, 2, behind=1)


def test_prompt_long_and_split(workspace):
    check_prompt([3], [9011], 64, 8, 1, 128, BF16, workspace)
    check_prompt([4, 1, 9], [2000, 5000, 9], 64, 4, 2, 64, FP16, workspace)
    check_prompt([4, 1, 9], [2000, 5000, 9], 64, 4, 2, 64, FP16, workspace, 700, 130)


@pytest.mark.parametrize("nbytes", [0, 16, 200_000, 3_000_000])
def test_prompt_with_less_workspace(cuda_lib, nbytes):
    work = torch.empty(nbytes, dtype=torch.uint8, device="cuda") if nbytes else None
    check_prompt([4, 1, 9], [2000, 3000, 9], 64, 4, 2, 64, FP16, work)
    check_prompt([100, 200], [600, 200], 16, 8, 2, 128, BF16, work)


def test_prompt_many_sequences(workspace):
    g = gen(8)
    new = torch.randint(0, 4, (700,), generator=g).tolist()
    check_prompt(new, [n + b % 40 for b, n in enumerate(new)], 16, 2, 1, 64, BF16, workspace)
    check_prompt([b % 2 for b in range(2048)], [1 + b % 3 for b in range(2048)], 8, 1, 1, 16, BF16,
                 workspace)


def test_prompt_scores_far_apart(workspace):
    for dtype in (BF16, FP16):
        check_prompt([100, 33], [400, 33], 16, 8, 2, 128, dtype, workspace, factor=20.0)
        check_prompt([100, 33], [400, 33], 16, 8, 2, 64, dtype, workspace, scale=1.0)
        check_prompt([100, 33], [400, 33], 16, 8, 2, 64, dtype, workspace, factor=0.0)


def test_prompt_entries_of_no_page_read_as_zeros(workspace):
    def some(table):
        table[0, 1], table[0, 3], table[1, 0] = -1, 1 << 29, -(1 << 31)
    check_prompt([100, 20, 2], [100, 20, 50], 16, 8, 2, 128, BF16, workspace, table=some)


def test_prompt_same_bits_again(workspace):
    a = check_prompt([300, 7], [300, 2000], 16, 8, 2, 128, BF16, workspace)
    for _ in range(3):
        b = check_prompt([300, 7], [300, 2000], 16, 8, 2, 128, BF16, workspace)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_prompt_and_decode_agree(workspace):
    """The last rows of prompts are what one-token calls answer."""
    lengths = [1, 40, 333]
    out, lse = check_prompt([1, 40, 100], lengths, 16, 8, 2, 128, BF16, workspace)
    pages = R.Pages(lengths, 16, 2, 128, BF16, seed=5, extra=1)
    q = torch.randn(141, 12, 128, generator=gen(6)).to(BF16)[:, :8]
    kc, vc, table, dev_lengths, _ = pages.cuda()
    one = torch.empty(3, 8, 128, dtype=BF16, device="cuda")
    last = [0, 40, 140]
    B.ar_fusion_decode_attention(q[last].cuda(), kc, vc, table, dev_lengths, one, workspace)
    assert bool(((one.float() - out[last].float()).abs() <= 2.0 ** -6).all())


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("prompt", [False, True])
def test_many_light_keys(workspace, prompt, dtype, cache):
    """One key of weight 1 and value 0, and 65535 of 2^-25 whose values are all there is to the
    output: they are half of what fp16 has next to a largest weight of 1."""
    n, D, P = 65536, 64, 1024
    k = torch.zeros(n // P, P, 1, D)
    v = torch.ones(n // P, P, 1, D)
    k[0, 5, 0, 0] = 25.0 if cache != E4M3 else 24.0
    v[0, 5] = 0.0
    k, v = k.to(cache), v.to(cache)
    q = torch.zeros(2, 2, D)
    q[:, :, 0] = 1.0
    q = q.to(dtype)
    table = torch.arange(n // P, dtype=torch.int32)[None]
    lengths = torch.tensor([n], dtype=torch.int32)
    starts = torch.tensor([0, 2 if prompt else 1], dtype=torch.int32)
    T = int(starts[1])
    scale = math.log(2.0) * (1.0 if cache != E4M3 else 25.0 / 24.0)
    out = torch.empty(T, 2, D, dtype=dtype, device="cuda")
    lse = torch.empty(T, 2, device="cuda")
    args = [t.cuda() for t in (q[:T], k, v, table, lengths)]
    if prompt:
        B.ar_fusion_prompt_attention(*args, starts.cuda(), out, workspace, scale=scale, lse=lse)
    else:
        B.ar_fusion_decode_attention(*args, out, workspace, scale=scale, lse=lse)
    want = R.attention(q[:T], k, v, table, lengths, starts, scale, 0, 0)
    assert 2.0 ** -10 < float(want[0].min()) < 2.0 ** -8
    R.check_attention(out, lse, want, dtype, FP16 if cache == E4M3 and not prompt else dtype,
                      LOST_PROMPT if prompt else LOST_ONE, splits=200)


def places(pages, b, index):
    """Page and row of the tokens of sequence b with these indexes."""
    P = pages.view(pages.k).shape[1]
    return pages.table[b].long()[index // P], index % P


@pytest.mark.parametrize("dtype,cache", KINDS)
def test_scores_that_climb(workspace, dtype, cache):
    """Scores that rise along the cache for half of the heads, by more than a power of 2^32 within
    some hundred keys, and fall for the others: sums are rescaled again and again."""
    lengths = [700, 300]

    def climb(pages):
        for b, n in enumerate(lengths):
            index = torch.arange(n)
            at = places(pages, b, index)
            k = pages.view(pages.k)
            k[at[0], at[1], :, 0] = (index * 0.5).to(cache)[:, None]
    for window, sinks in ((0, 0), (200, 10)):
        check_decode(lengths, 16, 8, 2, 64, dtype, cache, workspace, window, sinks, scale=1.0,
                     touch=climb)
        check_prompt([300, 33], lengths, 16, 8, 2, 64, dtype, workspace, window, sinks, scale=1.0,
                     touch=climb, cache=cache)


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("window,sinks", [(70, 0), (100, 5), (64, 130), (128, 64)])
def test_nothing_unseen_before_a_window(workspace, window, sinks, dtype, cache):
    """NaN in every key and value between the first tokens and the first one that a row sees."""
    lengths = [700, 300, 90]

    def junk(new):
        def touch(pages):
            for b, (n, length) in enumerate(zip(new, lengths)):
                index = torch.arange(sinks, max(sinks, length - n - window + 1))
                at = places(pages, b, index)
                for c in (pages.k, pages.v):
                    pages.view(c)[at[0], at[1]] = torch.full((), math.nan).to(cache)
        return touch
    check_decode(lengths, 16, 8, 2, 64, dtype, cache, workspace, window, sinks, touch=junk([1, 1, 1]))
    new = [150, 1, 40]
    check_prompt(new, lengths, 16, 8, 2, 128, dtype, workspace, window, sinks, touch=junk(new),
                 cache=cache)
    check_prompt(new, lengths, 16, 8, 2, 128, dtype, None, window, sinks, touch=junk(new), cache=cache)


@pytest.mark.parametrize("dtype,cache", KINDS)
def test_sequences_that_share_pages(workspace, dtype, cache):
    """A common beginning, and a page that stands twice in a sequence."""
    def share(table):
        table[1, :8] = table[0, :8]
        table[2, 3] = table[2, 1]
    check_decode([400, 300, 90], 32, 8, 2, 128, dtype, cache, workspace, table=share)
    check_prompt([40, 40, 20], [400, 300, 90], 32, 8, 2, 128, dtype, workspace, table=share, cache=cache)


@pytest.mark.parametrize("power", [95, -100])
def test_values_far_from_one(workspace, power):
    """bf16 values whose sums of 700 keys fit fp32 with room for weights of 2^16 (or 2^-16)."""
    def far(pages):
        pages.v *= 2.0 ** power
    for kw in ({}, {"window": 200, "sinks": 10}):
        check_decode([700, 300], 16, 8, 2, 64, BF16, BF16, workspace, touch=far, factor=5.0, **kw)
        check_prompt([300, 33], [700, 300], 16, 8, 2, 128, BF16, workspace, touch=far, factor=5.0, **kw)
