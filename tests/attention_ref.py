"""Plain 64-bit implementations of the attention-layer operators on the CPU, from
their definitions, and the inputs that the tests share.  Test infrastructure: shares no
code with the package."""
import math

import torch

U = 2.0 ** -24
E4M3 = torch.float8_e4m3fn


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def turn(x, position, inv_freq, axis_of, interleaved):
    """x [T, heads, D] in 64 bits; position [axes, T]; axis_of [rot / 2]."""
    out = x.clone()
    half = len(axis_of)
    for m in range(half):
        a = position[axis_of[m]].double() * inv_freq[m].double()
        c, s = torch.cos(a)[:, None], torch.sin(a)[:, None]
        lo, hi = (2 * m, 2 * m + 1) if interleaved else (m, m + half)
        out[..., lo] = x[..., lo] * c - x[..., hi] * s
        out[..., hi] = x[..., hi] * c + x[..., lo] * s
    return out


def rows_of(starts, lengths, tokens, most):
    """(row, sequence, index) of each row of a sequence."""
    for b in range(len(lengths)):
        lo, hi = int(starts[b]), int(starts[b + 1])
        if lo < 0 or hi > tokens or lo > hi:
            continue
        n = min(max(int(lengths[b]), 0), most)
        for row in range(lo, hi):
            yield row, b, n - (hi - row)


def gathered(cache, scale, table_row, n):
    """[n, heads, D] in 64 bits of one sequence; entries of no page read as zeros."""
    pages, P, K, D = cache.shape
    out = torch.zeros(n, K, D, dtype=torch.float64)
    for i in range(0, n, P):
        p = int(table_row[i // P])
        if 0 <= p < pages:
            m = min(P, n - i)
            out[i:i + m] = cache[p, :m].to(torch.float32).double() * scale
    return out


def attention(q, k_cache, v_cache, table, lengths, starts, scale, window, sinks, kv_scale=(1.0, 1.0)):
    """out, lse, and for the tolerances: sum p |v| of each element, the largest
    scale * sum |q| |k| of each row and head, the number of keys seen, max |v|.  Rows of no
    sequence stay NaN."""
    T, H, D = q.shape
    K, P = k_cache.shape[2], k_cache.shape[1]
    G = H // K
    out = torch.full((T, H, D), math.nan, dtype=torch.float64)
    mags = torch.zeros(T, H, D, dtype=torch.float64)
    lse, reach, count, big = (torch.full((T, H), math.nan, dtype=torch.float64) for _ in range(4))
    cached = {}
    for row, b, i in rows_of(starts, lengths, T, table.shape[1] * P):
        if b not in cached:
            n = min(max(int(lengths[b]), 0), table.shape[1] * P)
            cached = {b: [gathered(c, s, table[b], n)
                          for c, s in zip((k_cache, v_cache), kv_scale)]}
        k, v = cached[b]
        j = torch.arange(i + 1 if i >= 0 else 0)
        if window:
            j = j[(j > i - window) | (j < sinks)]
        if len(j) == 0:
            out[row], lse[row], reach[row], count[row], big[row] = 0.0, -math.inf, 0.0, 0, 0.0
            continue
        kk = k[j].repeat_interleave(G, 1)                       # [n, H, D]
        vv = v[j].repeat_interleave(G, 1)
        x = q[row].double()
        s = scale * torch.einsum("hd,nhd->nh", x, kk)
        p = torch.softmax(s, 0)
        out[row] = torch.einsum("nh,nhd->hd", p, vv)
        mags[row] = torch.einsum("nh,nhd->hd", p, vv.abs())
        lse[row] = torch.logsumexp(s, 0)
        reach[row] = (scale * torch.einsum("hd,nhd->nh", x.abs(), kk.abs())).amax(0)
        count[row] = len(j)
        big[row] = vv.abs().amax((0, 2))
    return out, lse, mags, reach, count, big


def check_attention(got, got_lse, want, dtype, products, lost, splits=2):
    """got against attention()'s answer.  A score is a sum of up to 128 products and its scale, each
    addition off by at most a whole step (2 U) of the sum of magnitudes; exp2 and the
    exponent's own rounding add 4 U and 2 U |s|, and the rescaling of a running maximum
    as much again.  The weights are rounded to `products`, the type of the second
    product; sums of n keys add n steps.  `products` fp16 also loses up to 2^-25 of
    each weight below its normal range, `lost` next to a largest weight that is taken as 1
    (a largest weight of 2^14 in the kernel for one token: 2^-39; of 2^5 in that for prompts)."""
    out, lse, mags, reach, count, big = want
    live = ~torch.isnan(count)
    got, got_lse = got.double().cpu(), None if got_lse is None else got_lse.double().cpu()
    ds = (2 * 130 * U + 6 * U) * reach + 16 * U
    rel = 2 * ds + (2 * count + 16 * splits) * U + half_step(products)
    tol = rel[..., None] * mags + half_step(dtype) * out.abs() + 2.0 ** -133
    if products == torch.float16:
        tol = tol + (count * big * lost)[..., None]
    if dtype == torch.float16:
        tol = tol + 2.0 ** -25
    bad = ~((got - out).abs() <= tol) & live[..., None]
    assert not bad.any(), (bad.nonzero()[:4].tolist(), got[bad][:4], out[bad][:4], tol[bad][:4],
                           int(bad.sum()))
    if got_lse is not None:
        fine = live & torch.isfinite(lse)
        near = (got_lse - lse).abs() <= ds + (2 * count + 16 * splits) * U + 4 * U * lse.abs()
        assert bool(near[fine].all()), ((got_lse - lse)[fine & ~near][:4], lse[fine & ~near][:4])
        empty = live & torch.isinf(lse)
        assert torch.equal(got_lse[empty], lse[empty])


class Pages:
    """A paged cache with sequences of the given lengths: pages in any order, entries
    behind the last page of no page, and what no sequence holds full of NaN."""

    def __init__(self, lengths, P, K, D, dtype, seed=0, hnd=False, spare=2, junk=True, extra=0):
        g = torch.Generator()
        g.manual_seed(seed)
        self.lengths = torch.tensor(lengths, dtype=torch.int32)
        need = [-(-max(n, 0) // P) for n in lengths]
        pages = sum(need) + spare
        order = torch.randperm(pages, generator=g).tolist()
        self.table = torch.full((len(lengths), max([1] + need) + extra), -7, dtype=torch.int32)
        self.table[:, ::2] = 1 << 30
        shape = (pages, K, P, D) if hnd else (pages, P, K, D)
        self.scale = None
        self.scales = (1.0, 1.0)
        if dtype == E4M3:
            self.scale = torch.tensor([0.02, 0.015])
            self.scales = tuple(self.scale.double().tolist())
        fill = math.nan if junk else 0.0
        self.k, self.v = (torch.full(shape, fill).to(dtype) for _ in range(2))
        self.view = (lambda t: t.transpose(1, 2)) if hnd else (lambda t: t)
        for b, n in enumerate(need):
            for i in range(n):
                p = order.pop()
                self.table[b, i] = p
                m = min(P, lengths[b] - i * P)
                for t, s in zip((self.k, self.v), self.scales):
                    x = torch.randn(m, K, D, generator=g) / s
                    self.view(t)[p, :m] = x.clamp(-448, 448).to(dtype) if dtype == E4M3 else x.to(dtype)

    def cuda(self):
        """k, v (as [pages, P, K, D] views), table, lengths, scale on the GPU."""
        return (self.view(self.k.cuda()), self.view(self.v.cuda()), self.table.cuda(),
                self.lengths.cuda(), None if self.scale is None else self.scale.cuda())
