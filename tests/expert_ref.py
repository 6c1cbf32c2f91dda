"""Plain 64-bit implementations of the expert-layer operators on the CPU, from
their definitions, one row at a time where that is clearest.  Test
infrastructure: shares no code with the package."""
import math

import numpy as np
import torch

BLOCK = 128
FP8_MAX = 448.0
FLOOR = 2.0 ** -100


def route(logits, bias, topk, score, groups, kept, group_score, renorm, scale):
    """ids (int), weights (float64) of one call.  logits: any float tensor [T, E];
    score "softmax" / "sigmoid"; group_score "max" / "top2"."""
    x = logits.double().cpu().numpy()
    T, E = x.shape
    b = np.zeros(E) if bias is None else bias.double().cpu().numpy()
    ids = np.full((T, topk), -1, dtype=np.int64)
    w = np.zeros((T, topk))
    size = E // groups
    # exact order where all biases are one finite number: that of the logits
    flat = bool(np.isfinite(b).all() and (b == b[0]).all())
    for t in range(T):
        live = [e for e in range(E) if not (x[t, e] == -math.inf or b[e] == -math.inf)]
        if not live:
            continue
        with np.errstate(all="ignore"):
            if score == "softmax":
                top = np.fmax.reduce(x[t, live])
                ex = np.exp(x[t] - top)
                s = ex / np.sum(ex[live])
            else:
                s = 1.0 / (1.0 + np.exp(-x[t]))
            c = s + b
        rank = x[t] if flat else c

        def best_first(values):
            """Indices, largest first, NaN behind every number, lower index first."""
            return sorted(values, key=lambda iv: (iv[1] != iv[1], -iv[1] if iv[1] == iv[1] else 0.0,
                                                  iv[0]))
        left = live
        if groups > 1:
            value = []
            for g in range(groups):
                mine = [e for e in live if e // size == g]
                order = [i for i, _ in best_first([(e, rank[e]) for e in mine])]
                if not order:
                    continue
                if group_score == "max":
                    value.append((g, rank[order[0]]))
                else:
                    value.append((g, c[order[0]] + (c[order[1]] if len(order) > 1 else 0.0)))
            stay = {g for g, _ in best_first(value)[:kept]}
            left = [e for e in live if e // size in stay]
        chosen = [i for i, _ in best_first([(e, rank[e]) for e in left])][:topk]
        if renorm and chosen:
            # ratios of the scores by their logarithms: none is lost to underflow
            with np.errstate(all="ignore"):
                logs = x[t, chosen] if score == "softmax" else -np.logaddexp(0.0, -x[t, chosen])
                ratio = np.exp(logs - np.fmax.reduce(logs)) + 0.0 * s[chosen]
            ratio = ratio / ratio.sum()
        for j, e in enumerate(chosen):
            ids[t, j] = e
            w[t, j] = (ratio[j] if renorm else s[e]) * scale
    return ids, w


def plan(ids, first, experts):
    flat = np.asarray(ids).reshape(-1)
    position = np.full(flat.shape, -1, dtype=np.int64)
    offsets = [0]
    row = 0
    for e in range(first, first + experts):
        for slot in np.nonzero(flat == e)[0]:
            position[slot] = row
            row += 1
        offsets.append(row)
    return np.array(offsets), position.reshape(np.asarray(ids).shape)


def e4m3(code):
    """Bytes to the values they stand for, float64."""
    c = np.asarray(code, dtype=np.int64)
    sign = np.where(c & 0x80, -1.0, 1.0)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * np.exp2(e - 10.0))
    return np.where((c & 0x7F) == 0x7F, np.nan, sign * v)


def activate(x, act):
    x = x.double().cpu().numpy()
    if not act:
        return x
    h = x.shape[1] // 2
    with np.errstate(all="ignore"):
        return x[:, :h] / (1.0 + np.exp(-x[:, :h])) * x[:, h:]


def blocks(n):
    return -(-n // BLOCK)


def block_amax(y):
    """[rows, blocks]: the largest |y|, NaN passed over, at least 2^-100."""
    return np.stack([np.fmax.reduce(np.abs(np.concatenate(
        [y[:, i:i + BLOCK], np.full((y.shape[0], 1), FLOOR)], 1)), axis=1)
        for i in range(0, y.shape[1], BLOCK)], 1)


def spread(scale, n):
    """[.., blocks] to [.., n]."""
    return np.repeat(scale, BLOCK, axis=-1)[..., :n]


def matmul(a, sa, b, sb):
    """(out, bound): the product, and sum |a||b| of the scaled factors, float64.
    a, b: bytes; sa [rows, blocks], sb [col blocks, blocks]."""
    a, b = e4m3(a), e4m3(b)
    af = a * spread(np.asarray(sa, dtype=np.float64), a.shape[1])
    bf = b * spread(np.repeat(np.asarray(sb, dtype=np.float64), BLOCK, axis=0)[:b.shape[0]],
                    b.shape[1])
    return af @ bf.T, np.abs(af) @ np.abs(bf).T


def combine(rows, position, weights, add):
    """(out, bound) float64."""
    r = rows.double().cpu().numpy()
    T, k = position.shape
    out = np.zeros((T, r.shape[1])) if add is None else add.double().cpu().numpy().copy()
    bound = np.abs(out)
    p, w = position.cpu().numpy(), weights.double().cpu().numpy()
    for t in range(T):
        for j in range(k):
            if 0 <= p[t, j] < r.shape[0]:
                out[t] += w[t, j] * r[p[t, j]]
                bound[t] += np.abs(w[t, j] * r[p[t, j]])
    return out, bound


def half_step(dtype):
    return torch.finfo(dtype).eps / 2
