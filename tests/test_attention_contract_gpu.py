"""What the attention-layer calls promise at the edges of their contract."""
import math
import threading
from fractions import Fraction

import pytest
import torch

import attention_ref as R
from allreduce_residual_rmsnorm_gb300 import binding as B

pytestmark = pytest.mark.gpu
BF16, FP16, E4M3 = torch.bfloat16, torch.float16, torch.float8_e4m3fn


def ints(*x):
    return torch.tensor(x, dtype=torch.int32)


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


@pytest.fixture(scope="module")
def workspace(cuda_lib):
    return torch.empty(B.AR_ATTENTION_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")


# ------------------------------------------- starts that decrease or leave the rows

def with_rows(starts, tokens):
    """The sequences that have rows, by the header's words."""
    if any(lo > hi for lo, hi in zip(starts, starts[1:])):
        return
    for b, (lo, hi) in enumerate(zip(starts, starts[1:])):
        if 0 <= lo and hi <= tokens:
            yield b, lo, hi


def many_starts(n):
    """2048 sequences that all say 0 .. n, turn by turn with what runs back."""
    return [0, n] * 1024 + [0]


STARTS = [
    (40, [0, 40, 0, 40]), (40, [0, 15, 10, 30]), (40, [0, 50, 10, 30]), (40, [20, 10, 40, 40]),
    (40, [-1, 5, 20, 41]), (40, [3, 2, 1, 0]), (40, [-(1 << 31), (1 << 31) - 1, 0, 40]),
    (40, [0, 0, 40, 10, 40, 40]), (300, [0, 150, 20, 300, 300, 310]), (40, many_starts(40)),
    (300, [b % 7 * 40 for b in range(1001)]), (40, [-5, 0, 17, 40, 41]), (40, [-1, 41]),
    (300, [0, 150, 300, 300, 1 << 30]), (300, [0] * 1000 + [150] * 700 + [300] * 348 + [301])]


@pytest.mark.parametrize("T,starts", STARTS, ids=lambda x: str(x)[:40])
def test_starts_that_decrease_or_leave_the_rows(workspace, T, starts):
    S, H, K, D, P = len(starts) - 1, 4, 2, 64, 16
    lengths = [max(hi - lo, 0) + b % 5 if S < 50 else 3 for b, (lo, hi) in
               enumerate(zip([max(x, 0) for x in starts], [min(x, T) for x in starts[1:]]))]
    rows = list(with_rows(starts, T))
    for b, lo, hi in rows:
        lengths[b] = hi - lo + b % 5
    pages = R.Pages(lengths, P, K, D, BF16, seed=2, extra=1)
    q = torch.randn(T, H, D, generator=gen(3)).to(BF16)
    kc, vc, table, dev_lengths, _ = pages.cuda()
    dev = ints(*starts).cuda()
    parts = []
    for b, lo, hi in rows:
        parts.append((lo, hi, R.attention(q[lo:hi], pages.k, pages.v, pages.table[b:b + 1],
                                          pages.lengths[b:b + 1], [0, hi - lo], D ** -0.5, 0, 0)))
    dead = torch.ones(T, dtype=torch.bool)
    for work in (workspace, None):
        out = torch.full((T, H, D), 5.0, dtype=BF16, device="cuda")
        lse = torch.full((T, H), 5.0, device="cuda")
        B.ar_fusion_prompt_attention(q.cuda(), kc, vc, table, dev_lengths, dev, out, work, lse=lse)
        torch.cuda.synchronize()
        assert B.ar_fusion_attention_status() == (B.AR_OK, -1)
        for lo, hi, w in parts:
            dead[lo:hi] = False
            R.check_attention(out[lo:hi], lse[lo:hi], w, BF16, BF16, 0.0, splits=40)
        assert bool((out.cpu()[dead] == 5.0).all()) and bool((lse.cpu()[dead] == 5.0).all())
    # the append: the rows of those sequences to their places, and nothing else anywhere
    k = torch.randn(T, K, D, generator=gen(4)).to(BF16)
    want_k = pages.k.clone()
    for b, lo, hi in rows:
        for row in range(lo, hi):
            i = lengths[b] - (hi - row)
            want_k[int(pages.table[b, i // P]), i % P] = k[row]
    q_out = torch.full((T, H, D), 5.0, dtype=BF16, device="cuda")
    kc2, vc2 = kc.clone(), kc.clone()
    B.ar_fusion_rope_append(q.cuda(), k.cuda(), k.cuda(), kc2, vc2, table, dev_lengths, None, q_out,
                            starts=dev)
    torch.cuda.synchronize()
    same = lambda x, y: torch.equal(x.cpu().view(torch.int16), y.view(torch.int16))  # noqa: E731
    assert same(kc2, want_k) and same(vc2, want_k)
    want_q = q.clone()
    want_q[dead] = 5.0
    assert same(q_out, want_q)


# ------------------------------------------- threads that share a stream and a workspace

@pytest.mark.parametrize("native", [True, False])
def test_two_threads_on_one_stream_with_one_workspace(workspace, monkeypatch, native):
    """Split calls of other sizes and kinds, queued by two threads: each has its own answer."""
    if not native:
        monkeypatch.setattr(B, "_native", None)
    stream = torch.cuda.Stream()

    def job(lengths, new, H, K, seed):
        pages = R.Pages(lengths, 16, K, 64, BF16, seed=seed, junk=False)
        kc, vc, table, dev_lengths, _ = pages.cuda()
        T = sum(new) if new else len(lengths)
        q = torch.randn(T, H, 64, generator=gen(seed)).to(BF16).cuda()
        starts = None if new is None else ints(*(sum(new[:b]) for b in range(len(new) + 1))).cuda()

        def call(out):
            if new is None:
                B.ar_fusion_decode_attention(q, kc, vc, table, dev_lengths, out, workspace, stream=stream)
            else:
                B.ar_fusion_prompt_attention(q, kc, vc, table, dev_lengths, starts, out, workspace,
                                             stream=stream)
        return call, [torch.empty_like(q) for _ in range(300)]

    jobs = [job([3000, 700], None, 8, 2, 5), job([900, 40, 2000], [7, 40, 3], 4, 2, 6)]
    want = []
    for call, outs in jobs:
        torch.cuda.synchronize()
        call(outs[0])
        torch.cuda.synchronize()
        want.append(outs[0].clone())

    failed = []

    def work(call, outs):
        try:
            for out in outs:
                call(out)
        except Exception as e:      # noqa: BLE001 -- a thread's error must reach the test
            failed.append(e)
    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed and B.ar_fusion_attention_status() == (B.AR_OK, -1)
    for (_, outs), w in zip(jobs, want):
        assert all(torch.equal(out, w) for out in outs)


@pytest.mark.parametrize("native", [True, False])
@pytest.mark.parametrize("call", ["prompt", "product", "experts' product"])
def test_the_first_call_of_a_thread(workspace, monkeypatch, call, native):
    """A host thread that has made no CUDA call yet."""
    if not native:
        monkeypatch.setattr(B, "_native", None)
    n = 300
    if call == "prompt":
        pages = R.Pages([n], 16, 2, 64, BF16, junk=False)
        kc, vc, table, lengths, _ = pages.cuda()
        q = torch.randn(n, 4, 64, generator=gen(1)).to(BF16).cuda()
        starts = ints(0, n).cuda()
        make = lambda: torch.empty_like(q)                                       # noqa: E731
        run = lambda out: B.ar_fusion_prompt_attention(                          # noqa: E731
            q, kc, vc, table, lengths, starts, out, workspace)
    else:
        a, b = (torch.randint(0, 120, (m, 256), generator=gen(m), dtype=torch.uint8).cuda() for m in (n, 128))
        sa, sb = torch.ones(n, 2).cuda(), torch.ones(1, 2).cuda()
        make = lambda: torch.empty(n, 128, device="cuda")                        # noqa: E731
        run = lambda out: B.ar_fusion_matmul_fp8(a, sa, b, sb, out)              # noqa: E731
        if call != "product":
            offsets = ints(0, n).cuda()
            run = lambda out: B.ar_fusion_expert_matmul_fp8(                     # noqa: E731
                a, sa, b[None], sb[None], offsets, out)
    want, got = make(), make()
    run(want)
    torch.cuda.synchronize()
    failed = []

    def first():
        try:
            run(got)
        except Exception as e:      # noqa: BLE001 -- a thread's error must reach the test
            failed.append(e)
    t = threading.Thread(target=first)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not failed and torch.equal(got, want)


# ------------------------------------------- angles of far positions

PI = Fraction(314159265358979323846264338327950288419716939937510582097494, 10 ** 59)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("bits", [12, 24, 26, 28, 30, 31])
def test_angles_of_far_positions(cuda_lib, bits, interleaved):
    """Rows (1, 0) give cos and sin themselves, and where those are small the output's own rounding
    hides nothing.  The angle: half a turn off by 2^-25 and 2^-32, times pi 1.6 U; cos and sin by
    2 U; the products with 1 and 0 are exact."""
    T, D = 256, 128
    g = gen(bits)
    where = torch.randint(1 << (bits - 1), 1 << bits, (T,), generator=g)
    where[::2] *= -1
    where[:3] = torch.tensor([(1 << bits) - 1, -(1 << bits), 1 << (bits - 1)])
    f = 1e4 ** (-torch.arange(0, D, 2) / D)
    f[1] = -f[1]
    x = torch.zeros(T, 1, D)
    first = slice(0, D, 2) if interleaved else slice(0, D // 2)
    second = slice(1, D, 2) if interleaved else slice(D // 2, D)
    x[:, :, first] = 1.0
    pages = R.Pages([T], 16, 1, D, FP16, junk=False)
    kc, vc, table, lengths, _ = pages.cuda()
    dx = x.to(FP16).cuda()
    out = torch.empty_like(dx)
    B.ar_fusion_rope_append(dx, dx, dx, kc, vc, table, lengths, f.cuda(), out, starts=ints(0, T).cuda(),
                            positions=where.to(torch.int32).cuda(), interleaved=interleaved)
    exact = [Fraction(v) / PI for v in f.tolist()]
    half = torch.tensor([[float(p * e % 2) for e in exact] for p in where.tolist()], dtype=torch.float64)
    got = out.cpu().double()[:, 0]
    for part, want in ((first, torch.cos(math.pi * half)), (second, torch.sin(math.pi * half))):
        off = (got[:, part] - want).abs()
        tol = 4 * R.U + R.half_step(FP16) * want.abs() + 2.0 ** -25
        assert bool((off <= tol).all()), ((off - tol).amax() / R.U, int((off > tol).sum()))
    at = pages.table[0].long()[torch.arange(T) // 16]
    assert torch.equal(kc[at, torch.arange(T) % 16], out)


def test_a_frequency_that_is_not_finite_gives_nan(cuda_lib):
    pages = R.Pages([4], 16, 1, 16, BF16, junk=False)
    kc, vc, table, lengths, _ = pages.cuda()
    x = torch.ones(4, 1, 16, dtype=BF16, device="cuda")
    f = torch.tensor([1.0, math.inf, math.nan, -math.inf, 0.5, 0.0, 0.25, -1.0])
    B.ar_fusion_rope_append(x, x, x, kc, vc, table, lengths, f.cuda(), starts=ints(0, 4).cuda())
    bad = ~torch.isfinite(f)
    assert torch.equal(torch.isnan(x.cpu()[:, 0]), torch.cat([bad, bad]).expand(4, 16))


# ------------------------------------------- as many heads as there may be

def test_one_token_without_keys_and_with_many_heads(workspace):
    """2^27 query heads of 128 elements: 2^31 vectors of 16 bytes of zeros.  (The heads overlap, 16
    bytes apart, so that they need no 34 GB.)"""
    H, K, D = 1 << 27, 1 << 20, 128
    rows = torch.full((8 * H + D,), 3.0, dtype=BF16, device="cuda")
    q = rows.as_strided((1, H, D), (8 * H, 8, 1))
    out_rows = torch.full((8 * H + D,), 5.0, dtype=BF16, device="cuda")
    out = out_rows.as_strided((1, H, D), (8 * H, 8, 1))
    pages = torch.zeros(8 * (K + 8) + D, dtype=BF16, device="cuda")
    cache = pages.as_strided((1, 8, K, D), (8, 8, 8, 1))
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    B.ar_fusion_decode_attention(q, cache, cache, table, ints(0).cuda(), out, workspace)
    torch.cuda.synchronize()
    assert int((out_rows == 0).sum()) == 8 * H + D - 8 and bool((out_rows[8 * H + D - 8:] == 5.0).all())


# ------------------------------------------- small workspaces

def one_call(lengths, new, H, K, D, nbytes, seed=7):
    """out, and whether the workspace was written."""
    pages = R.Pages(lengths, 64, K, D, BF16, seed=seed, junk=False)
    kc, vc, table, dev_lengths, _ = pages.cuda()
    T = len(lengths) if new is None else sum(new)
    q = torch.randn(T, H, D, generator=gen(seed)).to(BF16)
    work = torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda") if nbytes else None
    out, lse = torch.empty_like(q).cuda(), torch.empty(T, H, device="cuda")
    starts = list(range(T + 1)) if new is None else [sum(new[:b]) for b in range(len(new) + 1)]
    if new is None:
        B.ar_fusion_decode_attention(q.cuda(), kc, vc, table, dev_lengths, out, work, lse=lse)
    else:
        B.ar_fusion_prompt_attention(q.cuda(), kc, vc, table, dev_lengths, ints(*starts).cuda(), out, work,
                                     lse=lse)
    torch.cuda.synchronize()
    want = R.attention(q, pages.k, pages.v, pages.table, pages.lengths, ints(*starts), D ** -0.5, 0, 0)
    R.check_attention(out, lse, want, BF16, BF16, 0.0, splits=40)
    return out, work is not None and bool((work != 255).any())


@pytest.mark.parametrize("D", [64, 128])
def test_a_workspace_of_a_few_blocks_is_not_used_for_many_items(cuda_lib, D):
    """700 tokens, 16 heads of their own: a block of whole items for each of 152 SMs, against three."""
    want, _ = one_call([700], [700], 16, 16, D, 0)
    got, used = one_call([700], [700], 16, 16, D, 1 << 20)
    assert not used and torch.equal(got, want)
    assert one_call([700], [700], 16, 16, D, 40 << 20)[1]


@pytest.mark.parametrize("lengths,H,K,nbytes,used", [
    ([20011], 8, 1, 200_000, True), ([20011, 3], 8, 2, 200_000, True), ([20011], 8, 1, 16_000, False),
    ([900] * 20, 8, 2, 200_000, False), ([5000], 33, 1, 60_000, True)])
def test_one_token_is_split_where_the_workspace_holds_more_than_the_items(cuda_lib, lengths, H, K, nbytes, used):
    assert one_call(lengths, None, H, K, 128, nbytes)[1] == used
