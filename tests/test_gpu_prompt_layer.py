"""The prompt's operators together, as serving takes a batch through a layer's
attention: norms with rotation and append, the prompts' attention, the attention
of later chunks over the cache, then single tokens by the decode attention.

Tolerance. The reference is 64 bits throughout, from the projections on; the
calls round q and k once (u each, half a step) before the attention, which takes
them as they are. A score is off by at most (2 u + u^2 + a few 2^-20) sum_i
|q_i||k_i| scale =: d, so the weights are off by e^(2 d) - 1 relative, and by
w = u where they enter the product; sums over n keys by (n / 16 + 400) 2^-22.
Then one rounding of the output."""
import math

import pytest

import gpu_common as gc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    gc.require_gpu()
    gc.build_all()


class Layer:
    """Projections of whole sequences, their cache and the calls."""

    def __init__(self, lens, hq, hk, dim, kind, page=16, seed=0):
        import torch
        import awq_int4_moe_gb300 as awq
        self.t, self.awq = torch, awq
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.dt = {"f16": torch.float16, "bf16": torch.bfloat16}[kind]
        self.u = 2.0 ** -11 if kind == "f16" else 2.0 ** -8
        self.lens, self.hq, self.hk, self.dim, self.page = lens, hq, hk, dim, page
        most = max(lens)
        self.x = [torch.randn((n, hq + 2 * hk, dim), generator=g, device="cuda").to(self.dt) for n in lens]
        self.qw, self.kw = ((1 + 0.2 * torch.randn(dim, generator=g, device="cuda")).to(self.dt) for _ in range(2))
        angle = torch.arange(most, device="cuda", dtype=torch.float64)[:, None] * \
            10000.0 ** (-torch.arange(0, dim, 2, device="cuda", dtype=torch.float64) / dim)
        self.table = torch.cat([angle.cos(), angle.sin()], 1).float()
        per = -(-most // page)
        self.kc, self.vc = (torch.zeros((len(lens) * per + 1, page, hk, dim), device="cuda", dtype=self.dt) for _ in range(2))
        order = torch.randperm(len(lens) * per, generator=g, device="cuda")
        self.pages = order.view(len(lens), per).int()
        self.ws = torch.zeros(awq.prompt_attention_workspace_bytes(dim), dtype=torch.uint8, device="cuda")
        self.ws1 = torch.zeros(awq.paged_attention_workspace_bytes(dim), dtype=torch.uint8, device="cuda")
        self.st = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.done = [0] * len(lens)

    def ints(self, values, kind="int32"):
        return self.t.tensor(values, dtype=getattr(self.t, kind), device="cuda")

    def step(self, news, how):
        """Takes news[b] more tokens of each sequence; returns the output by sequence."""
        t, awq = self.t, self.awq
        x = t.cat([self.x[b][self.done[b]:self.done[b] + n] for b, n in enumerate(news)])
        where = [(b, p) for b, n in enumerate(news) for p in range(self.done[b], self.done[b] + n)]
        q, k, v = x[:, :self.hq], x[:, self.hq:self.hq + self.hk], x[:, self.hq + self.hk:]
        b, p = self.ints([w[0] for w in where], "int64"), self.ints([w[1] for w in where], "int64")
        slots = self.pages[b, p // self.page].long() * self.page + p % self.page
        awq.qk_norm_rope_append(q, k, v, self.qw, self.kw, 1e-6, p.int(), self.table, slots, self.kc, self.vc, self.st)   # q in place
        self.done = [d + n for d, n in zip(self.done, news)]
        cu = [0]
        for n in news:
            cu.append(cu[-1] + n)
        out = t.empty((len(where), self.hq, self.dim), device="cuda", dtype=self.dt)
        if how == "prompt":
            kk = self.kc.view(-1, self.hk, self.dim)[slots]               # the turned keys, packed
            awq.prompt_attention(q, kk, v, self.ints(cu), out, self.ws, self.st)
        elif how == "chunk":
            awq.chunk_attention(q, self.kc, self.vc, self.pages, self.ints(cu), self.ints(self.done), out, self.ws, self.st)
        else:
            awq.paged_attention(q, self.kc, self.vc, self.pages, self.ints(self.done), out, self.ws1, self.st)
        t.cuda.synchronize()
        assert int(self.st) == 0
        return [out[cu[i]:cu[i + 1]] for i in range(len(news))]

    def turned(self, x, w):
        t = self.t
        x = x.double()
        y = x / (x.square().mean(2, keepdim=True) + 1e-6).sqrt() * w.double()
        half = self.dim // 2
        row = self.table[: len(x)].double()[:, None]
        a, b, cos, sin = y[..., :half], y[..., half:], row[..., :half], row[..., half:]
        return t.cat([a * cos - b * sin, b * cos + a * sin], 2)

    def check(self, b, got):
        """got: the output of every token of sequence b."""
        t, n = self.t, self.lens[b]
        q = self.turned(self.x0[b][:, :self.hq], self.qw).view(n, self.hk, -1, self.dim)
        k = self.turned(self.x0[b][:, self.hq:self.hq + self.hk], self.kw)
        v = self.x0[b][:, self.hq + self.hk:].double()
        scale = self.dim ** -0.5
        s = t.einsum("ihgd,nhd->hgin", q, k) * scale
        s.masked_fill_(t.ones(n, n, dtype=t.bool, device="cuda").triu(1), -math.inf)
        prob = s.softmax(3)
        want = t.einsum("hgin,nhd->ihgd", prob, v).reshape(n, self.hq, self.dim)
        size = t.einsum("hgin,nhd->ihgd", prob, v.abs()).reshape(n, self.hq, self.dim)
        d = (2 * self.u + self.u ** 2 + 2.0 ** -18) * scale * float(t.einsum("ihgd,nhd->hgin", q.abs(), k.abs()).max())
        tol = want.abs() * self.u + (math.expm1(2 * d) + self.u + (n / 16 + 400) * 2.0 ** -22) * size + 2.0 ** -24
        err = (got.double() - want).abs()
        assert bool((err <= tol).all()), (b, float((err - tol).max()))

    def whole(self, steps):
        self.x0 = [x.clone() for x in self.x]
        outs = [[] for _ in self.lens]
        for news, how in steps:
            for o, part in zip(outs, self.step(news, how)):
                o.append(part)
        assert self.done == self.lens
        for b, o in enumerate(outs):
            self.check(b, self.t.cat(o))


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("heads,dim", [((20, 4), 128), ((6, 2), 64), ((4, 1), 256)])
def test_a_batch_from_its_prompts_to_its_last_token(kind, heads, dim):
    """Prompts, a mixed batch (a chunk of one, a token of another, drafted ones of
    a third, none of the last), then tokens one at a time by both attentions."""
    lens = [333, 40, 150, 17]
    layer = Layer(lens, *heads, dim, kind)
    layer.whole([([200, 35, 130, 13], "prompt"), ([130, 1, 5, 0], "chunk"), ([1, 1, 1, 1], "decode"), ([1, 1, 1, 1], "chunk"),
                 ([1, 2, 13, 2], "chunk")])


def test_every_split_of_a_prompt_gives_the_same_answer():
    """One prompt in one call, in chunks of one size and of another: the same
    tolerance of the same 64-bit answer."""
    for steps in ([([700], "prompt")], [([700], "chunk")], [([256], "prompt"), ([256], "chunk"), ([188], "chunk")],
                  [([1], "prompt"), ([698], "chunk"), ([1], "decode")]):
        Layer([700], 10, 2, 128, "f16", seed=4).whole(steps)


def test_two_streams_with_a_workspace_each():
    """Calls that run at the same time, each with its own workspace, have the
    bits of calls made alone."""
    import torch
    import awq_int4_moe_gb300 as awq
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    cu = torch.tensor([0, 700, 1000, 3500], dtype=torch.int32, device="cuda")
    calls = []
    for i in range(2):
        q, k, v = (torch.randn((3500, h, 128), generator=g, device="cuda").half() for h in (8, 2, 2))
        calls.append((q, k, v, cu, torch.empty_like(q), torch.zeros(awq.prompt_attention_workspace_bytes(128), dtype=torch.uint8,
                                                                   device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")))
    alone = []
    for c in calls:
        awq.prompt_attention(*c)
        torch.cuda.synchronize()
        alone.append(c[4].clone())
        c[4].zero_()
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s in zip(calls, streams):
            awq.prompt_attention(*c, stream=s)
    torch.cuda.synchronize()
    for c, a in zip(calls, alone):
        assert torch.equal(c[4], a) and int(c[6]) == 0


def test_two_graphs_share_a_workspace():
    """A serving step of each of two batches (append and chunk attention),
    captured with one workspace, replayed in turn with growing lengths."""
    import torch
    import awq_int4_moe_gb300 as awq
    hq, hk, dim, page, per = 8, 2, 128, 16, 160
    ws = torch.zeros(awq.prompt_attention_workspace_bytes(dim), dtype=torch.uint8, device="cuda")
    w = torch.ones(dim, device="cuda", dtype=torch.float16)
    table = torch.cat([torch.ones(per * page, dim // 2, device="cuda"), torch.zeros(per * page, dim // 2, device="cuda")], 1)
    g = torch.Generator(device="cuda")
    g.manual_seed(5)

    class Batch:
        def __init__(self, news, lens):
            n = sum(news)
            self.x = torch.randn((n, hq + 2 * hk, dim), generator=g, device="cuda").half()
            cu = [0]
            for m in news:
                cu.append(cu[-1] + m)
            self.cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
            self.b = torch.repeat_interleave(torch.arange(len(news), device="cuda"), torch.tensor(news, device="cuda"))
            self.i = torch.arange(n, device="cuda") - self.cu[self.b].long()
            self.news = torch.tensor(news, dtype=torch.int32, device="cuda")
            self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
            self.kc, self.vc = (torch.randn((len(news) * per, page, hk, dim), generator=g, device="cuda").half() for _ in range(2))
            self.pages = torch.randperm(len(news) * per, generator=g, device="cuda").view(len(news), per).int()
            self.q = torch.empty((n, hq, dim), device="cuda", dtype=torch.float16)
            self.out, self.st = torch.empty_like(self.q), torch.zeros(1, dtype=torch.int32, device="cuda")

        def step(self):
            self.lens += self.news
            at = (self.lens - self.news)[self.b].long() + self.i
            slots = self.pages[self.b, at // page].long() * page + at % page
            x = self.x
            awq.qk_norm_rope_append(x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:], w, w, 1e-6, at.int(), table, slots, self.kc, self.vc,
                                    self.st, q_out=self.q)
            awq.chunk_attention(self.q, self.kc, self.vc, self.pages, self.cu, self.lens, self.out, ws, self.st)

    batches = [Batch([1, 40, 3], [900, 5, 2000]), Batch([200, 1], [0, 1500])]
    keep = [(b.lens.clone(), b.kc.clone(), b.vc.clone()) for b in batches]
    want = []
    for b in batches:
        outs = []
        for _ in range(4):
            b.step()
            torch.cuda.synchronize()
            outs.append(b.out.clone())
        want.append(outs)
    graphs = []
    for b in batches:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            b.step()
        graphs.append(graph)
    for b, kept in zip(batches, keep):
        for t, k in zip((b.lens, b.kc, b.vc), kept):
            t.copy_(k)
    for i in range(4):
        for b, graph in zip(batches, graphs):
            graph.replay()
        torch.cuda.synchronize()
        for b, outs in zip(batches, want):
            assert torch.equal(b.out, outs[i]) and int(b.st) == 0
