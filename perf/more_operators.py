"""The operators of an attention layer between two tensor-parallel epilogues:
rotating the new queries and keys and appending keys and values to a paged
cache, attention of one new token per sequence over that cache, and attention
of prompts (many new tokens per sequence) over it.

``listed()`` / ``draw()`` give cases, ``prepare()`` makes what a serving loop
has in hand before the call, ``run()`` is one pass.  With ``own`` false the
pass is plain torch arithmetic (32 bits; 64 for the angles of far positions),
with ``own`` true the calls of the library.  ``exact()`` gives the outputs from
the definitions in 64 bits.
"""
import math

import torch

own = False

FP8_MAX = 448.0
WORKSPACE = 32 << 20        # bytes that a serving loop keeps for the attention calls
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "fp16": 2, "e4m3": 1}


# ------------------------------------------------------------------- cases
#
# seqs sequences of `length` tokens down to length * (1 - spread), the new ones
# included: `new` of them down to new * (1 - new_spread).

def listed():
    return [
        # one decode step on a rank of eight (64 / 8 heads there): launch latency
        dict(name="append_decode", op="append", seqs=64, length=4096, spread=0.5, new=1,
             new_spread=0.0, heads=8, kv=1, dim=128, rot=128, axes=1, interleaved=False, page=64,
             dtype="bf16", cache="bf16"),
        # four long prompts
        dict(name="append_prompt", op="append", seqs=4, length=2048, spread=0.0, new=2048,
             new_spread=0.0, heads=32, kv=8, dim=128, rot=128, axes=1, interleaved=False, page=64,
             dtype="bf16", cache="bf16"),
        # an image among text: positions of time, height and width; 64 of 80 elements rotated
        # as neighbours, 8-bit cache, odd counts
        dict(name="append_axes_e4m3_odd", op="append", seqs=5, length=1501, spread=0.9, new=701,
             new_spread=0.8, heads=15, kv=5, dim=80, rot=64, axes=3, interleaved=True, page=32,
             dtype="fp16", cache="e4m3"),
        # a small batch on a rank of eight: latency
        dict(name="decode_small", op="decode", seqs=4, length=1003, spread=0.5, heads=8, kv=1,
             dim=128, page=16, window=0, sinks=0, dtype="bf16", cache="bf16"),
        # a batch of conversations of uneven lengths
        dict(name="decode_batch", op="decode", seqs=64, length=8000, spread=0.9, heads=32, kv=8,
             dim=128, page=64, window=0, sinks=0, dtype="bf16", cache="bf16"),
        # one long document
        dict(name="decode_long", op="decode", seqs=1, length=131072, spread=0.0, heads=64, kv=8,
             dim=128, page=64, window=0, sinks=0, dtype="bf16", cache="bf16"),
        # many conversations in an 8-bit cache
        dict(name="decode_e4m3", op="decode", seqs=128, length=4096, spread=0.5, heads=64, kv=8,
             dim=128, page=128, window=0, sinks=0, dtype="bf16", cache="e4m3"),
        # a layer with a sliding window, first tokens visible; 7 heads share a key, odd sizes
        dict(name="decode_window_odd", op="decode", seqs=33, length=5003, spread=0.99, heads=28,
             kv=4, dim=80, page=32, window=1000, sinks=5, dtype="fp16", cache="fp16"),
        # a long prompt
        dict(name="prompt_full", op="prompt", seqs=1, length=8192, spread=0.0, new=8192,
             new_spread=0.0, heads=32, kv=8, dim=128, page=64, window=0, sinks=0, dtype="bf16",
             cache="bf16"),
        # prompts in a layer with a sliding window, first tokens visible
        dict(name="prompt_window", op="prompt", seqs=3, length=5000, spread=0.4, new=5000,
             new_spread=0.4, heads=64, kv=8, dim=128, page=64, window=1024, sinks=4, dtype="bf16",
             cache="bf16"),
        # prompts in chunks: a few hundred new tokens behind a cached part; odd sizes
        dict(name="prompt_chunks_odd", op="prompt", seqs=13, length=3001, spread=0.8, new=401,
             new_spread=0.9, heads=14, kv=2, dim=64, page=16, window=0, sinks=0, dtype="fp16",
             cache="fp16"),
        # four drafted tokens of each sequence looked over at once, on a rank of eight: latency
        dict(name="prompt_drafted", op="prompt", seqs=8, length=1003, spread=0.5, new=4,
             new_spread=0.0, heads=8, kv=1, dim=128, page=16, window=0, sinks=0, dtype="bf16",
             cache="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "prompt", "prompt"])
    kv = rng.choice([1, 1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 4, 5, 7, 8, 8, 16])
    dim = rng.choice([64, 80, 96, 128, 128, 128])
    page = rng.choice([16, 16, 32, 64, 128])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    case = dict(op=op, heads=kv * group, kv=kv, dim=dim, page=page, dtype=dtype, cache=dtype,
                spread=round(rng.uniform(0.0, 0.95), 2))
    if op == "append":
        axes = rng.choice([1, 1, 3])
        case.update(new=rng.choice([1, _log(rng, 1, 2048)]), new_spread=round(rng.random(), 2),
                    rot=rng.choice([dim, dim, 32]), axes=axes, interleaved=rng.random() < 0.4,
                    cache=rng.choice([dtype, dtype, "e4m3"]))
        case["seqs"] = _log(rng, 1, max(1, min(128, 8192 * 48 // (case["new"] * kv * (group + 2)))))
        case["length"] = _log(rng, case["new"], max(case["new"], 131072 // case["seqs"]))
        return case
    if rng.random() < 0.35:
        case.update(window=_log(rng, 64, 2048), sinks=rng.choice([0, 4, _log(rng, 1, 64)]))
    else:
        case.update(window=0, sinks=0)
    if op == "decode":
        case["cache"] = rng.choice([dtype, dtype, "e4m3"])
        case["length"] = _log(rng, 1, 131072)
        most = 64 * 8000 * 4 // (case["length"] * kv)
        case["seqs"] = _log(rng, 1, max(1, min(256, most)))
        return case
    case["new"] = _log(rng, 2, 4096)
    case["length"] = case["new"] + rng.choice([0, 0, _log(rng, 1, 8192)])
    case["new_spread"] = round(rng.uniform(0.0, 0.9), 2)
    most = 8192 * 8192 * 32 // (2 * case["length"] * case["new"] * kv * group)
    case["seqs"] = _log(rng, 1, max(1, min(32, most)))
    return case


def _spread(most, spread, n):
    return [max(1, round(most * (1.0 - spread * i / max(1, n - 1)))) for i in range(n)]


def _sizes(case):
    """Tokens in the cache and new ones of each sequence."""
    n = case["seqs"]
    lengths = _spread(case["length"], case["spread"], n)
    new = _spread(case.get("new", 1), case.get("new_spread", 0.0), n)
    new = new[n // 2:] + new[:n // 2]
    return lengths, [min(a, b) for a, b in zip(new, lengths)]


# ------------------------------------------------------------------ inputs

def _sections(case):
    """Rotated pairs of each axis: a quarter for time, the rest shared."""
    pairs, axes = case["rot"] // 2, case["axes"]
    if axes == 1:
        return (pairs,)
    first = pairs // 4
    return (first, (pairs - first + 1) // 2, (pairs - first) // 2)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt, H, K, D, P = DT[case["dtype"]], case["heads"], case["kv"], case["dim"], case["page"]

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    lengths, new = _sizes(case)
    S = len(lengths)
    T = sum(new)
    per = -(-max(lengths) // P)                         # pages of the longest
    used = sum(-(-n // P) for n in lengths)
    pages = used + 3
    # the pages of a sequence lie anywhere; entries behind its last are of no page
    order = torch.randperm(pages, generator=g, device="cuda")[:used].to(torch.int32)
    length = torch.tensor(lengths, device="cuda")
    count = (length + P - 1) // P
    at = torch.arange(per, device="cuda")
    first = count.cumsum(0) - count
    table = torch.where(at < count[:, None], order[(first[:, None] + at).clamp_max(used - 1)], -1)
    starts = torch.tensor([sum(new[:i]) for i in range(S + 1)], device="cuda")
    k_cache, v_cache = (randn(pages, P, K, D) for _ in range(2))
    scale = None
    if case["cache"] == "e4m3":
        scale = torch.tensor([0.021, 0.013], device="cuda")
        k_cache, v_cache = ((x / s).clamp_(-FP8_MAX, FP8_MAX)
                            for x, s in zip((k_cache, v_cache), scale.tolist()))
    # a few channels of the keys are far above the rest
    loud = 1.0 + 4.0 * (torch.rand(D, generator=g, device="cuda") < 0.03)
    s = dict(case=case, page_table=table.to(torch.int32).contiguous(),
             lengths=length.to(torch.int32), starts=starts.to(torch.int32), kv_scale=scale,
             longest=max(new),
             k_cache=(k_cache * loud).to(DT[case["cache"]]) if scale is None
             else k_cache.to(DT[case["cache"]]), v_cache=v_cache.to(DT[case["cache"]]))
    if case["op"] == "append":
        # the output of one projection: queries, keys and values side by side
        qkv = (randn(T, H + 2 * K, D) * loud).to(dt)
        s.update(q=qkv[:, :H], k=qkv[:, H:H + K], v=qkv[:, H + K:],
                 q_out=torch.empty(T, H, D, dtype=dt, device="cuda"),
                 inv_freq=10000.0 ** (-torch.arange(0, case["rot"], 2, device="cuda")
                                      / case["rot"]), positions=None)
        if case["axes"] == 3:
            # a picture of 24 columns behind the text: time stands still
            row = torch.arange(T, device="cuda")
            s["positions"] = torch.stack([100 + row // 1000, 100 + row // 24 % 40,
                                          100 + row % 24]).to(torch.int32)
        return s
    s.update(q=(2.0 * randn(T, H, D)).to(dt),
             out=torch.empty(T, H, D, dtype=dt, device="cuda"),
             lse=torch.empty(T, H, device="cuda"),
             workspace=torch.empty(WORKSPACE, dtype=torch.uint8, device="cuda"))
    return s


# ------------------------------------------------------------ the plain forms

def _rotate(x, cos, sin, interleaved):
    """x [T, heads, D] in 32 bits, cos and sin [T, rot / 2]."""
    half = cos.shape[1]
    cos, sin = cos[:, None], sin[:, None]
    out = x.clone()
    a, b = ((x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if interleaved
            else (x[..., :half], x[..., half:2 * half]))
    first, second = a * cos - b * sin, b * cos + a * sin
    if interleaved:
        out[..., 0:2 * half:2], out[..., 1:2 * half:2] = first, second
    else:
        out[..., :half], out[..., half:2 * half] = first, second
    return out


def _rows(s):
    """Sequence and index in it of each new row."""
    starts = s["starts"].long()
    row = torch.arange(s["q"].shape[0], device=starts.device)
    seq = torch.searchsorted(starts, row, right=True) - 1
    return seq, s["lengths"].long()[seq] - starts[seq + 1] + row


def _plain_append(s):
    case, P = s["case"], s["case"]["page"]
    seq, index = _rows(s)
    where = index[None] if s["positions"] is None else s["positions"].long()
    axis = torch.repeat_interleave(
        torch.arange(case["axes"], device=seq.device),
        torch.tensor(_sections(case), device=seq.device), output_size=case["rot"] // 2)
    angle = where[axis].t().double() * s["inv_freq"].double()
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    q = _rotate(s["q"].float(), cos, sin, case["interleaved"])
    k = _rotate(s["k"].float(), cos, sin, case["interleaved"])
    v = s["v"].float()
    page = s["page_table"][seq, index // P].long()
    if s["kv_scale"] is None:
        s["k_cache"][page, index % P] = k.to(s["k_cache"].dtype)
        s["v_cache"][page, index % P] = v.to(s["v_cache"].dtype)
    else:
        k = (k / s["kv_scale"][0]).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
        v = (v / s["kv_scale"][1]).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
        s["k_cache"].view(torch.uint8)[page, index % P] = k.view(torch.uint8)
        s["v_cache"].view(torch.uint8)[page, index % P] = v.view(torch.uint8)
    return dict(q=q.to(s["q"].dtype), k_cache=s["k_cache"], v_cache=s["v_cache"])


def _gathered(s):
    """Keys and values [S, kv, length, D] in 32 bits."""
    table = s["page_table"].long().clamp_min(0)
    both = []
    for i, name in enumerate(("k_cache", "v_cache")):
        x = s[name][table] if s["kv_scale"] is None else (
            s[name].view(torch.uint8)[table].view(torch.float8_e4m3fn))
        x = x.float().flatten(1, 2).transpose(1, 2)
        both.append(x if s["kv_scale"] is None else x * s["kv_scale"][i])
    return both


def _plain_attention(s):
    case, H, K, D = s["case"], s["case"]["heads"], s["case"]["kv"], s["case"]["dim"]
    starts, lengths, n = s["starts"].long(), s["lengths"].long(), s["longest"]
    S, T, G = lengths.shape[0], s["q"].shape[0], H // K
    seq, index = _rows(s)
    inside = torch.arange(T, device=seq.device) - starts[seq]
    q = torch.zeros(S, n, H, D, device=seq.device)
    q[seq, inside] = s["q"].float()
    q = q.view(S, n, K, G, D).permute(0, 2, 3, 1, 4)             # [S, K, G, n, D]
    k, v = _gathered(s)
    score = (q.reshape(S, K, G * n, D) @ k.transpose(2, 3)) * (1.0 / math.sqrt(D))
    score = score.view(S, K, G, n, -1)
    i = (lengths - starts[1:] + starts[:-1])[:, None] + torch.arange(n, device=seq.device)
    j = torch.arange(score.shape[-1], device=seq.device)
    seen = j <= i[..., None]                                     # [S, n, L]
    if case["window"]:
        seen &= (j > i[..., None] - case["window"]) | (j < case["sinks"])
    seen &= j < lengths[:, None, None]
    score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    e = torch.exp(score.sub_(top))
    total = e.sum(-1, keepdim=True)
    out = (e.view(S, K, G * n, -1) @ v).view(S, K, G, n, D) / total
    lse = (top + torch.log(total)).squeeze(-1)
    out = out.permute(0, 3, 1, 2, 4).reshape(S, n, H, D)[seq, inside]
    lse = lse.permute(0, 3, 1, 2).reshape(S, n, H)[seq, inside]
    return dict(out=out.to(s["q"].dtype), lse=lse)


# ------------------------------------------------------------------- a pass

def run(s):
    case, op = s["case"], s["case"]["op"]
    if not own:
        return _plain_append(s) if op == "append" else _plain_attention(s)
    from allreduce_residual_rmsnorm_gb300 import binding as B
    if op == "append":
        B.ar_fusion_rope_append(
            s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["page_table"], s["lengths"],
            s["inv_freq"], s["q_out"], starts=s["starts"], positions=s["positions"],
            sections=_sections(case) if case["axes"] > 1 else None,
            interleaved=case["interleaved"], kv_scale=s["kv_scale"])
        return dict(q=s["q_out"], k_cache=s["k_cache"], v_cache=s["v_cache"])
    if op == "decode":
        B.ar_fusion_decode_attention(
            s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["lengths"], s["out"],
            s["workspace"], window=case["window"], sinks=case["sinks"], lse=s["lse"],
            kv_scale=s["kv_scale"])
    else:
        B.ar_fusion_prompt_attention(
            s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["lengths"], s["starts"],
            s["out"], s["workspace"], window=case["window"], sinks=case["sinks"], lse=s["lse"],
            kv_scale=s["kv_scale"])
    return dict(out=s["out"], lse=s["lse"])


def _seen(case, length, new):
    """(pairs of a new token and a key that it sees, keys that any of them sees)."""
    w, sinks = case["window"], case["sinks"]
    if not w:
        return new * (length - new) + new * (new + 1) // 2, length
    pairs = 0
    for i in range(length - new, length):
        low = max(0, i + 1 - w)                 # the window's first key
        pairs += i + 1 - low + min(sinks, low)
    low = max(0, length - new + 1 - w)
    return pairs, length - low + min(sinks, low)


def work(case):
    H, K, D = case["heads"], case["kv"], case["dim"]
    z, c = SIZE[case["dtype"]], SIZE[case["cache"]]
    lengths, new = _sizes(case)
    T = sum(new)
    if case["op"] == "append":
        return dict(bytes=T * D * (z * (2 * H + 2 * K) + c * 2 * K), flops=T * 3 * case["rot"] * (H + K))
    seen = [_seen(case, a, b) for a, b in zip(lengths, new)]
    return dict(bytes=T * H * (2 * D * z + 4) + sum(k for _, k in seen) * K * 2 * D * c,
                flops=4 * D * H * sum(p for p, _ in seen))


# ------------------------------------------------- the definitions in 64 bits

def _e4m3_grid(v):
    """64-bit values to the nearest E4M3 value, ties to even: a step is 2^-3 of the
    binade, and 2^-9 below 2^-6."""
    e = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6)))
    step = torch.exp2(e - 3)
    return (torch.round(v / step) * step).clamp(-FP8_MAX, FP8_MAX)


def exact(case, seed):
    s = prepare(case, seed)
    H, K, D, P = case["heads"], case["kv"], case["dim"], case["page"]
    lengths, new = _sizes(case)
    f64 = torch.float64
    if case["op"] == "append":
        q, k = s["q"].to(f64).clone(), s["k"].to(f64).clone()
        where = s["positions"]
        if where is None:
            where = torch.cat([torch.arange(a - b, a, device="cuda") for a, b in zip(lengths, new)])
            where = where[None]
        half, m = case["rot"] // 2, 0
        for axis, pairs in enumerate(_sections(case)):
            for _ in range(pairs):
                turn = torch.polar(torch.ones((), dtype=f64, device="cuda"),
                                   where[axis].to(f64) * s["inv_freq"][m].to(f64))
                lo, hi = (2 * m, 2 * m + 1) if case["interleaved"] else (m, m + half)
                for x in (q, k):
                    z = torch.complex(x[..., lo], x[..., hi]) * turn[:, None]
                    x[..., lo], x[..., hi] = z.real, z.imag
                m += 1
        caches = []
        table = s["page_table"].tolist()
        for i, (name, x) in enumerate((("k_cache", k), ("v_cache", s["v"].to(f64)))):
            c = s[name].to(f64)
            if s["kv_scale"] is not None:
                x = _e4m3_grid(x / s["kv_scale"][i].to(f64))
            row = 0
            for b, (length, n) in enumerate(zip(lengths, new)):
                at = length - n
                while at < length:                      # up to the end of its page
                    m = min(P - at % P, length - at)
                    c[table[b][at // P], at % P:at % P + m] = x[row:row + m]
                    row, at = row + m, at + m
            caches.append(c)
        return dict(q=q, k_cache=caches[0], v_cache=caches[1])
    if sum(a * b for a, b in zip(lengths, new)) * H > 1 << 32:
        return None
    out, lse = (torch.empty(sum(new), H, *d, dtype=f64, device="cuda") for d in ((D,), ()))
    row = 0
    for b, (length, n) in enumerate(zip(lengths, new)):
        own_pages = s["page_table"][b, :-(-length // P)].long()
        both = []
        for i, name in enumerate(("k_cache", "v_cache")):
            x = (s[name][own_pages] if s["kv_scale"] is None else
                 s[name].view(torch.uint8)[own_pages].view(torch.float8_e4m3fn).to(f64)
                 * s["kv_scale"][i].to(f64))
            both.append(x.reshape(-1, K, D)[:length])
        for r in range(0, n, 1024):                     # rows at a time
            m = min(1024, n - r)
            last = length - n + r + m                   # keys behind it are of later tokens
            i = torch.arange(last - m, last, device="cuda")[:, None]
            j = torch.arange(last, device="cuda")[None]
            hidden = j > i
            if case["window"]:
                hidden |= (i - j >= case["window"]) & (j >= case["sinks"])
            for h in range(H):
                key = both[0][:last, h * K // H].to(f64)
                value = both[1][:last, h * K // H].to(f64)
                z = s["q"][row + r:row + r + m, h].to(f64) @ key.t() / math.sqrt(D)
                z[hidden] = -math.inf
                lse[row + r:row + r + m, h] = torch.logsumexp(z, 1)
                out[row + r:row + r + m, h] = torch.softmax(z, 1) @ value
        row += n
    return dict(out=out, lse=lse)
