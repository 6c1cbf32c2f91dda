"""What the attention-layer calls promise at the edges of their contract."""
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
