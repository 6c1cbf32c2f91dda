"""The attention-layer calls as they are used: between two fused calls, a prompt and then
decode steps over the same cache, queued one behind the other, captured, on other streams."""
import os
import subprocess
import sys

import pytest
import torch

import attention_ref as R
from allreduce_residual_rmsnorm_gb300 import binding as B

pytestmark = pytest.mark.gpu
BF16, U8 = torch.bfloat16, torch.uint8


class Layer:
    """The attention layer of one of two ranks: 8 query and 2 key heads of 64 here, hidden 512."""
    H, K, D, HIDDEN, PAGE = 8, 2, 64, 512, 16

    def __init__(self, lengths, room, seed, cache=BF16, window=0, sinks=0, workspace=None):
        g = torch.Generator()
        g.manual_seed(seed)
        self.S, self.window, self.sinks = len(lengths), window, sinks
        width = (self.H + 2 * self.K) * self.D
        codes = lambda *s: (100.0 * torch.randn(s, generator=g)).clamp(-448, 448).to(  # noqa: E731
            torch.float8_e4m3fn).view(U8).cuda()
        self.w_in, self.w_out = codes(width, self.HIDDEN), codes(self.HIDDEN, self.H * self.D)
        self.s_in = torch.full((-(-width // 128), self.HIDDEN // 128), 6e-4).cuda()
        self.s_out = torch.full((self.HIDDEN // 128, self.H * self.D // 128), 6e-4).cuda()
        need = [-(-n // self.PAGE) for n in room]
        order = torch.randperm(sum(need), generator=g).tolist()
        self.table = torch.zeros(self.S, max(need), dtype=torch.int32)
        for b, n in enumerate(need):
            self.table[b, :n] = torch.tensor([order.pop() for _ in range(n)])
        self.table = self.table.cuda()
        shape = (sum(need), self.PAGE, self.K, self.D)
        self.k, self.v = (torch.zeros(shape, dtype=BF16).to(cache).cuda() for _ in range(2))
        self.scale = None if cache == BF16 else torch.tensor([0.05, 0.03]).cuda()
        self.inv_freq = (1e4 ** (-torch.arange(0, self.D, 2) / self.D)).cuda()
        self.work = torch.empty(1 << 24, dtype=U8, device="cuda") if workspace is None else workspace

    def buffers(self, T):
        new = lambda *s, d=BF16: torch.empty(*s, dtype=d, device="cuda")  # noqa: E731
        h, width = self.HIDDEN, (self.H + 2 * self.K) * self.D
        return dict(q=new(T, h, d=U8), s=new(T, h // 128, d=torch.float32), qkv=new(T, width),
                    att=new(T, self.H, self.D), aq=new(T, h, d=U8), a_s=new(T, h // 128, d=torch.float32),
                    out=new(T, h), lse=new(T, self.H, d=torch.float32))

    def run(self, x, lengths, starts, b, sync=lambda: None):
        """x [T, hidden] -> a rank's partial [T, hidden]; starts None: one row each."""
        H, K, D, T = self.H, self.K, self.D, x.shape[0]
        B.ar_fusion_quant_blocks(x, b["q"], b["s"])
        sync()
        B.ar_fusion_matmul_fp8(b["q"], b["s"], self.w_in, self.s_in, b["qkv"])
        sync()
        qkv = b["qkv"].view(T, H + 2 * K, D)
        q, k, v = qkv[:, :H], qkv[:, H:H + K], qkv[:, H + K:]
        B.ar_fusion_rope_append(q, k, v, self.k, self.v, self.table, lengths, self.inv_freq,
                                starts=starts, kv_scale=self.scale)
        sync()
        more = dict(window=self.window, sinks=self.sinks, lse=b["lse"], kv_scale=self.scale)
        if starts is None:
            B.ar_fusion_decode_attention(q, self.k, self.v, self.table, lengths, b["att"], self.work, **more)
        else:
            B.ar_fusion_prompt_attention(q, self.k, self.v, self.table, lengths, starts, b["att"],
                                         self.work, **more)
        sync()
        B.ar_fusion_quant_blocks(b["att"].view(T, H * D), b["aq"], b["a_s"])
        sync()
        B.ar_fusion_matmul_fp8(b["aq"], b["a_s"], self.w_out, self.s_out, b["out"])
        sync()
        return b["out"]


class Model:
    """Two ranks' attention layers and the fused call on their partials, several tokens long."""

    def __init__(self, prompts, steps, seed=1, **kw):
        self.prompts, self.steps = prompts, steps
        room = [n + steps for n in prompts]
        self.ranks = [Layer(prompts, room, seed + r, **kw) for r in range(2)]
        S, T = len(prompts), sum(prompts)
        self.ws = B.ar_fusion_workspace_create(2, max(T, S, 16), Layer.HIDDEN, B.AR_DT_BF16)
        self.gamma = torch.ones(Layer.HIDDEN, dtype=BF16, device="cuda")
        g = torch.Generator()
        g.manual_seed(seed + 9)
        self.x = torch.randn(T, Layer.HIDDEN, generator=g).to(BF16).cuda()
        self.starts = torch.tensor([sum(prompts[:b]) for b in range(S + 1)], dtype=torch.int32).cuda()
        self.ends = self.starts[1:].long() - 1
        self.lengths = torch.tensor(prompts, dtype=torch.int32).cuda()
        self.wide = [r.buffers(T) for r in self.ranks]
        self.few = [r.buffers(S) for r in self.ranks]
        self.res, self.norm = torch.empty_like(self.x), torch.empty_like(self.x)
        self.row = torch.empty(S, Layer.HIDDEN, dtype=BF16, device="cuda")
        self.row_res = torch.empty_like(self.row)

    def prompt(self, sync=lambda: None):
        parts = [r.run(self.x, self.lengths, self.starts, b, sync) for r, b in zip(self.ranks, self.wide)]
        B.ar_fusion_run(self.ws, parts, self.x, self.gamma, 1e-6, B.PATTERNS["res_norm"],
                        residual_out=self.res, norm_out=self.norm)
        sync()
        self.row.copy_(self.norm[self.ends])

    def step(self, sync=lambda: None):
        self.lengths += 1
        parts = [r.run(self.row, self.lengths, None, b, sync) for r, b in zip(self.ranks, self.few)]
        B.ar_fusion_run(self.ws, parts, self.row, self.gamma, 1e-6, B.PATTERNS["res_norm"],
                        residual_out=self.row_res, norm_out=self.row)
        sync()
        return self.row.clone()

    def close(self):
        assert B.ar_fusion_workspace_status(self.ws)[0] == B.AR_OK
        assert B.ar_fusion_matmul_status() == (B.AR_OK, -1)
        assert B.ar_fusion_attention_status() == (B.AR_OK, -1)
        B.ar_fusion_workspace_destroy(self.ws)


@pytest.mark.parametrize("window,sinks", [(0, 0), (20, 3)])
def test_layers_without_a_wait_between_them(cuda_lib, window, sinks):
    a, b = (Model([40, 1, 130, 17], 12, window=window, sinks=sinks) for _ in range(2))
    a.prompt(torch.cuda.synchronize)
    want = [a.step(torch.cuda.synchronize) for _ in range(12)]
    b.prompt()
    got = [b.step() for _ in range(12)]
    torch.cuda.synchronize()
    assert torch.equal(a.norm, b.norm)
    for w, x in zip(want, got):
        assert torch.equal(w, x) and bool(torch.isfinite(x).all())
    for r, s in zip(a.ranks, b.ranks):
        assert torch.equal(r.k, s.k) and torch.equal(r.v, s.v)
    a.close()
    b.close()


def test_decode_steps_are_what_the_prompt_would_have_been(cuda_lib):
    """Rows appended one at a time and looked at by one-token calls, against one prompt of all rows,
    and against 64 bits on what the cache then holds."""
    n, more = 50, 14
    g = torch.Generator()
    g.manual_seed(5)
    rows = torch.randn(n + more, Layer.H + 2 * Layer.K, Layer.D, generator=g).to(BF16).cuda()
    one, two = (Layer([n], [n + more], 3) for _ in range(2))
    H, K = Layer.H, Layer.K

    def put(layer, lo, hi, starts):
        x = rows[lo:hi].clone()
        length = torch.tensor([hi], dtype=torch.int32).cuda()
        B.ar_fusion_rope_append(x[:, :H], x[:, H:H + K], x[:, H + K:], layer.k, layer.v, layer.table,
                                length, layer.inv_freq, starts=starts)
        return x[:, :H], length
    ends = lambda k: torch.tensor([0, k], dtype=torch.int32).cuda()  # noqa: E731
    q, length = put(one, 0, n + more, ends(n + more))
    whole = torch.empty(n + more, H, Layer.D, dtype=BF16, device="cuda")
    B.ar_fusion_prompt_attention(q, one.k, one.v, one.table, length, ends(n + more), whole, one.work)
    put(two, 0, n, ends(n))
    for i in range(n, n + more):
        qi, length = put(two, i, i + 1, None)
        out = torch.empty(1, H, Layer.D, dtype=BF16, device="cuda")
        B.ar_fusion_decode_attention(qi, two.k, two.v, two.table, length, out, two.work)
        assert torch.equal(qi, q[i:i + 1])
        want = R.attention(qi.cpu(), two.k.cpu(), two.v.cpu(), two.table.cpu(), length.cpu(), [0, 1],
                           Layer.D ** -0.5, 0, 0)
        R.check_attention(out, None, want, BF16, BF16, 0.0, splits=8)
        R.check_attention(whole[i:i + 1], None, want, BF16, BF16, 0.0, splits=8)
    assert torch.equal(one.k[one.table.long()], two.k[two.table.long()])


def test_decode_steps_in_one_graph_and_two_that_share_a_workspace(cuda_lib):
    a, b = Model([33, 70], 12), Model([33, 70], 12)
    work = b.ranks[0].work
    b.ranks[1].work = work                      # one behind the other on a stream: one is enough
    a.prompt()
    b.prompt()
    want = [a.step() for _ in range(12)]
    b.step()                                    # fills the launch caches
    graphs = []
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        before = b.lengths.clone()
        with torch.cuda.graph(graph, stream=s):
            b.step()
        assert torch.equal(before, b.lengths)   # captured, not run
        graphs.append(graph)
    for i in range(1, 12):
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        assert torch.equal(b.row, want[i])
    a.close()
    b.close()


def test_two_streams_at_once_with_a_workspace_each(cuda_lib):
    models = [Model([200, 31, 77], 10, seed=40 + i) for i in range(2)]
    alone = []
    for m in [Model([200, 31, 77], 10, seed=40 + i) for i in range(2)]:
        m.prompt()
        alone.append([m.step() for _ in range(10)])
        torch.cuda.synchronize()
        m.close()
    streams = [torch.cuda.Stream() for _ in models]
    got = [[], []]
    torch.cuda.synchronize()
    for m, s in zip(models, streams):
        with torch.cuda.stream(s):
            m.prompt()
    for _ in range(10):
        for i, (m, s) in enumerate(zip(models, streams)):
            with torch.cuda.stream(s):
                got[i].append(m.step())
    torch.cuda.synchronize()
    for g, w in zip(got, alone):
        assert all(torch.equal(x, y) for x, y in zip(g, w))
    for m in models:
        m.close()


def test_an_e4m3_cache_in_decode_steps(cuda_lib):
    layer = Layer([60, 5], [80, 30], 7, cache=torch.float8_e4m3fn)
    g = torch.Generator()
    g.manual_seed(2)
    starts = torch.tensor([0, 60, 65], dtype=torch.int32).cuda()
    lengths = torch.tensor([60, 5], dtype=torch.int32).cuda()
    x = torch.randn(65, Layer.H + 2 * Layer.K, Layer.D, generator=g).to(BF16).cuda()
    H, K = Layer.H, Layer.K
    B.ar_fusion_rope_append(None, x[:, H:H + K], x[:, H + K:], layer.k, layer.v, layer.table, lengths,
                            layer.inv_freq, starts=starts, kv_scale=layer.scale)
    for i in range(10):
        lengths += 1
        row = torch.randn(2, Layer.HIDDEN, generator=g).to(BF16).cuda()
        b = layer.buffers(2)
        layer.run(row, lengths, None, b)
        q = b["qkv"].view(2, H + 2 * K, Layer.D)[:, :H]         # rotated in place
        want = R.attention(q.cpu(), layer.k.cpu(), layer.v.cpu(), layer.table.cpu(), lengths.cpu(),
                           [0, 1, 2], Layer.D ** -0.5, 0, 0, layer.scale.double().tolist())
        R.check_attention(b["att"], b["lse"], want, BF16, torch.float16, 2.0 ** -39, splits=8)


def test_calls_on_a_given_stream_and_through_ctypes(cuda_lib, monkeypatch):
    """The stream argument, and the binding's own marshalling against the built module's."""
    lengths, new = [70, 9, 200], [5, 9, 1]
    pages = R.Pages(lengths, 16, 2, 64, BF16)
    kc, vc, table, dev_lengths, _ = pages.cuda()
    starts = torch.tensor([0, 5, 14, 15], dtype=torch.int32).cuda()
    work = torch.empty(1 << 24, dtype=U8, device="cuda")
    g = torch.Generator()
    g.manual_seed(1)
    q = torch.randn(15, 8, 64, generator=g).to(BF16).cuda()
    f = (1e4 ** (-torch.arange(0, 64, 2) / 64)).cuda()
    where = torch.randint(0, 99, (2, 15), generator=g, dtype=torch.int32).cuda()
    side = torch.cuda.Stream()

    def calls(stream):
        k, v, q_out = kc.clone(), vc.clone(), torch.empty_like(q)
        outs = [torch.empty(15, 8, 64, dtype=BF16, device="cuda"), torch.empty(15, 8, device="cuda"),
                torch.empty(3, 8, 64, dtype=BF16, device="cuda"), torch.empty(3, 8, device="cuda")]
        torch.cuda.synchronize()
        B.ar_fusion_rope_append(q, q[:, :2], q[:, 2:4], k, v, table, dev_lengths, f, q_out, starts=starts,
                                positions=where, sections=[20, 12], stream=stream)
        B.ar_fusion_prompt_attention(q_out, k, v, table, dev_lengths, starts, outs[0], work, lse=outs[1],
                                     window=50, sinks=2, stream=stream)
        B.ar_fusion_decode_attention(q_out[:3], k, v, table, dev_lengths, outs[2], work, lse=outs[3],
                                     scale=0.2, stream=stream)
        torch.cuda.synchronize()
        return [q_out, k.nan_to_num(), v.nan_to_num(), *outs]
    want = calls(None)
    for s in (side, side.cuda_stream):
        assert all(torch.equal(x, y) for x, y in zip(want, calls(s)))
    monkeypatch.setattr(B, "_native", None)
    assert all(torch.equal(x, y) for x, y in zip(want, calls(side)))


def test_caches_past_32_bits(cuda_lib):
    """Pages whose elements lie beyond 2^32 bytes and 2^31 elements."""
    P, K, D, pages = 64, 8, 128, 36000                          # 4.7 GB each
    kc, vc = (torch.empty(pages, P, K, D, dtype=BF16, device="cuda") for _ in range(2))
    at = [pages - 1, 3, pages - 2, 17000]
    g = torch.Generator()
    g.manual_seed(4)
    small = [torch.randn(len(at), P, K, D, generator=g).to(BF16) for _ in range(2)]
    index = torch.tensor(at).cuda()
    for c, s in zip((kc, vc), small):
        c[index] = s.cuda()
    n = P * 3 + 40
    table, local = torch.tensor([at], dtype=torch.int32), torch.tensor([[0, 1, 2, 3]])
    lengths = torch.tensor([n], dtype=torch.int32)
    q = torch.randn(10, 16, D, generator=g).to(BF16)
    work = torch.empty(1 << 25, dtype=U8, device="cuda")
    starts = torch.tensor([0, 10], dtype=torch.int32)
    out = torch.empty(10, 16, D, dtype=BF16, device="cuda")
    one = torch.empty(1, 16, D, dtype=BF16, device="cuda")
    B.ar_fusion_prompt_attention(q.cuda(), kc, vc, table.cuda(), lengths.cuda(), starts.cuda(), out, work)
    B.ar_fusion_decode_attention(q[9:].cuda(), kc, vc, table.cuda(), lengths.cuda(), one, work)
    want = R.attention(q, *small, local, lengths, starts, D ** -0.5, 0, 0)
    R.check_attention(out, None, want, BF16, BF16, 0.0, splits=8)
    R.check_attention(one, None, [w[9:] for w in want], BF16, BF16, 0.0, splits=8)
    new = torch.randn(10, K, D, generator=g).to(BF16).cuda()
    B.ar_fusion_rope_append(None, new, new, kc, vc, table.cuda(), lengths.cuda(), None, starts=starts.cuda())
    assert torch.equal(kc[at[3], 30:40], new) and torch.equal(vc[at[3], 30:40], new)


FIRST_CALLS = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import torch
import test_attention_layer_chain_gpu as C
m = C.Model([20, 3], 4)
s = torch.cuda.Stream()
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph, stream=s):
    m.ranks[0].run(m.x, m.lengths, m.starts, m.wide[0])
    m.ranks[0].run(m.row, m.lengths, None, m.few[0])
m.row.fill_(0.5)
graph.replay()
torch.cuda.synchronize()
got = [m.wide[0]["out"].clone(), m.few[0]["out"].clone()]
m.ranks[0].run(m.x, m.lengths, m.starts, m.wide[0])
m.ranks[0].run(m.row, m.lengths, None, m.few[0])
torch.cuda.synchronize()
assert torch.equal(got[0], m.wide[0]["out"]) and torch.equal(got[1], m.few[0]["out"])
m.close()
"""


def test_first_calls_of_a_process_under_capture(cuda_lib):
    tests = os.path.dirname(os.path.abspath(__file__))
    code = FIRST_CALLS.format(root=os.path.dirname(tests), tests=tests)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-2000:]
