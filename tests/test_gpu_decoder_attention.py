"""awq_paged_attention against 64-bit results.

Tolerances. A score is a dot product of D terms in fp32 and one scaling: it is
off by at most d = (D + 8) 2^-23 scale |q||k|, so a weight by 2 d relative
(numerator and sum), plus 2^-20 for the exponential and the split of the
weights into 16-bit terms (2^-12 more where a weight is one fp16 term: bf16
queries over an e4m3 cache), plus the fp32 sums: at most n / 16 + 64 + 320
additions in a row (a lane's units, the merges, the joined pieces) at 2^-24
each. Errors of weights move the output by at most their size times the largest
|v|; then one rounding (u as in the norm's tests)."""
import math

import pytest

import gpu_common as gc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    gc.require_gpu()
    gc.build_all()


def torch():
    return gc.torch_mod()


def dtype_of(name):
    t = torch()
    return {"f16": t.float16, "bf16": t.bfloat16, "e4m3": t.float8_e4m3fn}[name]


_WS = {}


def workspace(dim):
    """One workspace for all calls at a head size: zero-filled once."""
    import awq_int4_moe_gb300 as awq
    size = awq.paged_attention_workspace_bytes(dim)
    if size not in _WS:
        _WS[size] = torch().zeros(size, dtype=torch().uint8, device="cuda")
    return _WS[size]


class Case:
    def __init__(self, lens, hq, hk, dim, kind, cache, page, heads_first=False, seed=0, q_std=1.0, spare=2):
        t = torch()
        g = t.Generator(device="cuda")
        g.manual_seed(seed)
        self.lens, self.hq, self.hk, self.dim, self.kind, self.page = lens, hq, hk, dim, kind, page
        need = [-(-n // page) for n in lens]
        pages = sum(need) + spare
        shape = (pages, hk, page, dim) if heads_first else (pages, page, hk, dim)
        std = 40.0 if cache == "e4m3" else 1.0
        self.kc, self.vc = ((t.randn(shape, generator=g, device="cuda") * std).to(dtype_of(cache)) for _ in range(2))
        if heads_first:
            self.kc, self.vc = self.kc.transpose(1, 2), self.vc.transpose(1, 2)
        self.scales = (0.025, 0.03) if cache == "e4m3" else (1.0, 1.0)
        order = t.randperm(pages, generator=g, device="cuda").int().cpu()
        self.table = t.full((len(lens), max(1, max(need, default=1))), -5, dtype=t.int32)    # unneeded entries: no page
        at = 0
        for i, n in enumerate(need):
            self.table[i, :n] = order[at:at + n]
            at += n
        self.free = order[at:]
        self.table = self.table.cuda()
        self.seq = t.tensor(lens, dtype=t.int32, device="cuda")
        self.q = (t.randn((len(lens), hq, dim), generator=g, device="cuda") * q_std).to(dtype_of(kind))
        self.scale = dim ** -0.5

    def call(self, **over):
        import awq_int4_moe_gb300 as awq
        t = torch()
        out = t.full_like(self.q, 9.0)
        lse = t.full((len(self.lens), self.hq), 9.0, device="cuda")
        st = t.zeros(1, dtype=t.int32, device="cuda")
        a = dict(q=self.q, k_cache=self.kc, v_cache=self.vc, page_table=self.table, seq_lens=self.seq, out=out,
                 workspace=workspace(self.dim), dev_status=st, scale=self.scale, lse=lse, k_scale=self.scales[0],
                 v_scale=self.scales[1])
        a.update(over)
        awq.paged_attention(**a)
        t.cuda.synchronize()
        return a["out"], a["lse"], int(st)

    def rows(self, b):
        """k, v of a sequence, 64 bits: [tokens][KV heads][dim]."""
        t = torch()
        n = self.lens[b]
        pages = self.table[b, : -(-n // self.page)].long()
        take = lambda c, s: c.float()[pages].reshape(-1, self.hk, self.dim)[:n].double() * s  # noqa: E731
        return take(self.kc, self.scales[0]), take(self.vc, self.scales[1]) if n else t.zeros(0)

    def check(self, out, lse, sequences=None):
        t = torch()
        u = 2.0 ** -11 if self.kind == "f16" else 2.0 ** -8
        for b in range(len(self.lens)) if sequences is None else sequences:
            n = self.lens[b]
            if n == 0:
                assert bool((out[b] == 0).all()) and bool((lse[b] == -math.inf).all())
                continue
            k, v = self.rows(b)
            group = self.hq // self.hk
            q = self.q[b].double().view(self.hk, group, self.dim)
            s = t.einsum("hgd,nhd->hgn", q, k) * self.scale
            want = t.einsum("hgn,nhd->hgd", t.softmax(s, 2), v).reshape(self.hq, self.dim)
            size = float(q.norm(dim=2).max() * k.norm(dim=2).max()) * self.scale
            d = (self.dim + 8) * 2.0 ** -23 * size
            sums = (n / 16 + 384) * 2.0 ** -24
            one = 2.0 ** -12 if self.kind == "bf16" and self.kc.dtype == t.float8_e4m3fn else 0.0
            tol = want.abs() * u + (2 * d + 2.0 ** -20 + one + 2 * sums) * float(v.abs().max()) + 2.0 ** -25
            err = (out[b].double() - want).abs()
            assert bool((err <= tol).all()), f"sequence {b}: {float((err - tol).max())} over {float(tol.min())}"
            ref = t.logsumexp(s, 2).view(-1)
            err = (lse[b].double() - ref).abs()
            assert bool((err <= d + 2.0 ** -20 + sums + 2.0 ** -22 * ref.abs()).all()), f"lse {b}: {float(err.max())}"


def run(*args, **kw):
    c = Case(*args, **kw)
    out, lse, st = c.call()
    assert st == 0
    c.check(out, lse)
    return c


EDGES = [1, 15, 16, 17, 0, 63, 64, 65, 2, 1000, 0, 129]
TYPES = [("f16", "f16"), ("bf16", "bf16"), ("f16", "e4m3"), ("bf16", "e4m3")]


@pytest.mark.parametrize("kind,cache", TYPES)
@pytest.mark.parametrize("dim", [16, 64, 80, 96, 128, 144, 256])
@pytest.mark.parametrize("group", [1, 5, 8, 9, 16])
def test_types_and_heads(kind, cache, dim, group):
    run(EDGES, 2 * group, 2, dim, kind, cache, 16, seed=dim + group)


@pytest.mark.parametrize("dim", [8, 72, 136, 200])
def test_head_sizes_of_half_a_step(dim):
    run(EDGES, 6, 2, dim, "f16", "f16", 16, seed=dim)


@pytest.mark.parametrize("group", [17, 24, 40])
@pytest.mark.parametrize("kind,cache", TYPES)
def test_many_heads_of_one(group, kind, cache):
    run([33, 0, 700], group, 1, 128, kind, cache, 16, seed=group)


@pytest.mark.parametrize("page", [1, 3, 5, 16, 24, 64, 256])
@pytest.mark.parametrize("heads_first", [False, True])
def test_pages(page, heads_first):
    run(EDGES, 8, 2, 128, "f16", "f16", page, heads_first, seed=page)
    run(EDGES, 8, 2, 128, "bf16", "e4m3", page, heads_first, seed=page)


@pytest.mark.parametrize("lens", [[1], [16], [17], [0], [0, 0, 5], [5000], [40000], [3, 20000, 1, 64], [77] * 300])
def test_lengths(lens):
    run(lens, 8, 2, 128, "f16", "f16", 16, seed=len(lens))
    run(lens, 8, 1, 64, "bf16", "e4m3", 32, seed=len(lens))


def test_more_sequences_than_threads_and_lengths_in_shared_memory():
    lens = [(i * 37) % 90 for i in range(1500)]
    c = Case(lens, 4, 2, 64, "f16", "f16", 16)
    out, lse, st = c.call()
    assert st == 0
    c.check(out, lse, range(0, 1500, 7))


def test_peaked_scores():
    run(EDGES, 8, 2, 128, "f16", "f16", 16, q_std=60.0)
    run(EDGES, 16, 1, 128, "bf16", "bf16", 16, q_std=60.0)
    run(EDGES, 8, 2, 128, "bf16", "e4m3", 16, q_std=1e6)       # past fp16's range before the scale
    run(EDGES, 8, 2, 128, "bf16", "e4m3", 16, q_std=1e-30)


@pytest.mark.parametrize("kind,cache", TYPES)
@pytest.mark.parametrize("scale", [0.0, -0.0, -0.1, 1e-40])
def test_scales_of_zero_and_below(kind, cache, scale):
    c = Case(EDGES, 8, 2, 128, kind, cache, 16)
    c.scale = scale
    out, lse, st = c.call()
    assert st == 0
    c.scale = abs(scale)                                       # what the tolerances take
    if scale < 0:
        c.q = -c.q
    c.check(out, lse)


def test_query_of_zeros_with_a_small_cache_scale():
    c = Case(EDGES, 8, 2, 128, "bf16", "e4m3", 16)
    c.q.zero_()
    c.scales = (1e-8, 0.03)
    out, lse, st = c.call()
    assert st == 0
    c.check(out, lse)


@pytest.mark.parametrize("kind,cache", TYPES)
def test_many_small_weights_beside_a_large_one(kind, cache):
    """Token 0 outweighs each other one by 2^26.6 and has values of 0: the output
    is what the other 2,499 leave. A weight in fp16 is off by at most 2^-25 of
    2^7 times the largest one, which adds 2^-32 per token to the tolerance
    (nothing for a bf16 cache). Segments outnumber the warps, so that whole
    ones are in a single warp."""
    t = torch()
    n, few = 2500, [0, 77, 159]
    c = Case([n] * 160, 8, 8, 64, kind, cache, 64, spare=0)
    first = c.table[:, 0].long()
    raw = t.zeros(c.kc.shape, device="cuda")
    raw[first, 0, :, 0] = 11.0 / c.scales[0]
    c.kc.copy_(raw.to(c.kc.dtype))
    raw.fill_(400.0 if cache == "e4m3" else 12.0)
    raw[first, 0] = 0.0
    c.vc.copy_(raw.to(c.vc.dtype))
    c.q.zero_()
    c.q[:, :, 0] = 13.4
    out, lse, st = c.call()
    assert st == 0
    u = 2.0 ** -11 if kind == "f16" else 2.0 ** -8
    for b in few:
        k, v = c.rows(b)
        s = t.einsum("hd,nhd->hn", c.q[b].double(), k) * c.scale
        want = t.einsum("hn,nhd->hd", t.softmax(s, 1), v)
        relative = u + 2 * (64 + 8) * 2.0 ** -23 * float(s.max()) + 2.0 ** -20 + 2 * (n / 16 + 384) * 2.0 ** -24
        relative += 2.0 ** -12 if kind == "bf16" and cache == "e4m3" else 0.0
        tol = want * relative + 2.0 ** -25 + (0.0 if cache == "bf16" else n * 2.0 ** -32 * float(v.max()))
        err = (out[b].double() - want).abs()
        assert float(tol.max()) < 0.1 * float(want.min()) and bool((err <= tol).all()), float((err - tol).max())


@pytest.mark.parametrize("kind,cache", TYPES)
def test_values_past_the_end_do_not_matter(kind, cache):
    """NaN and infinities in free pages and in the places after a sequence's
    last token; the result has the same bits as with zeros there."""
    t = torch()
    results = []
    for bad in (0.0, float("nan"), 448.0 if cache == "e4m3" else float("inf")):
        c = Case([1, 17, 50, 0, 111], 8, 2, 128, kind, cache, 16, seed=4)
        for plane in (c.kc, c.vc):
            raw = plane.float()
            raw[c.free.long().cuda()] = bad
            for b, n in enumerate(c.lens):
                if n % 16:
                    raw[c.table[b, n // 16].long(), n % 16:] = bad
            plane.copy_(raw.to(plane.dtype) if cache != "e4m3" else raw.to(t.float8_e4m3fn))
        out, lse, st = c.call()
        assert st == 0
        c.check(out, lse)
        results.append((out, lse))
    for out, lse in results[1:]:
        assert bool((out == results[0][0]).all()) and bool((lse == results[0][1]).all())


def test_non_finite_values_inside():
    t = torch()
    c = Case([40, 40, 40], 8, 2, 128, "f16", "f16", 16, seed=4)
    c.vc[c.table[0, 1].long(), 3, 0, 5] = float("nan")         # one V element: its column, its heads
    c.kc[c.table[1, 1].long(), 3, 1] = float("nan")            # one K row: its heads
    out, lse, st = c.call()
    assert st == 0
    assert bool(out[0, :4, 5].isnan().all()) and int(out[0].isnan().sum()) == 4
    assert bool(out[1, 4:].isnan().all()) and bool(lse[1, 4:].isnan().all()) and not bool(out[1, :4].isnan().any())
    c.check(out, lse, [2])


def test_same_bits_every_time_and_on_a_side_stream():
    t = torch()
    c = Case([3000, 5, 900, 0, 12000], 10, 2, 128, "f16", "f16", 16)
    first = c.call()
    for _ in range(5):
        again = c.call()
        assert bool((again[0] == first[0]).all()) and bool((again[1] == first[1]).all())
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    again = c.call(stream=side)
    assert bool((again[0] == first[0]).all())


def test_strides_of_q_out_and_table():
    t = torch()
    c = Case([100, 7], 8, 2, 128, "f16", "f16", 16)
    want, _, _ = c.call()
    wide = t.zeros((2, 12, 192), device="cuda", dtype=t.float16)
    q = wide[:, 2:10, :128]
    q.copy_(c.q)
    out = t.full((8, 2, 128), 9.0, device="cuda", dtype=t.float16).transpose(0, 1)
    table = t.full((2, 40), -5, dtype=t.int32, device="cuda")
    table[:, : c.table.shape[1]] = c.table
    got, _, st = c.call(q=q, out=out, page_table=table[:, : c.table.shape[1]])
    assert st == 0 and bool((got == want).all())
    got, lse, st = c.call(lse=None)
    assert st == 0 and lse is None and bool((got == want).all())


def test_shared_pages():
    """Two sequences whose first pages are the same ones."""
    c = Case([64, 70], 4, 2, 64, "f16", "f16", 16)
    c.table[1, :4] = c.table[0, :4]
    out, lse, st = c.call()
    assert st == 0
    c.check(out, lse)


def test_bad_pages_and_lengths_are_reported():
    import awq_int4_moe_gb300 as awq
    t = torch()
    for bad in (-1, 1 << 30):
        c = Case([40, 200, 33], 8, 2, 128, "f16", "f16", 16)
        c.table[1, 3] = bad
        out, lse, st = c.call()
        assert st == awq.ERR_BAD_INDEX
        c.check(out, lse, [0, 2])
    for bad in (-1, 13 * 16 + 1):
        c = Case([40, 200, 33], 8, 2, 128, "f16", "f16", 16)
        c.table[:] = c.table.clamp(min=0)
        c.seq[1] = bad
        out, lse, st = c.call()
        assert st == awq.ERR_BAD_INDEX
        c.check(out, lse, [0, 2])
    out, lse, st = Case([40, 200, 33], 8, 2, 128, "f16", "f16", 16).call()      # the workspace is ready again
    assert st == 0


def test_cache_past_32_bit_offsets():
    t = torch()
    c = Case([50], 8, 8, 128, "f16", "f16", 16)
    pages = 140000                               # 2.3 G elements a plane
    big = [t.zeros((pages, 16, 8, 128), device="cuda", dtype=t.float16) for _ in range(2)]
    n = c.table.shape[1]
    for plane, small in zip(big, (c.kc, c.vc)):
        plane[pages - n:] = small[c.table[0].long()]
    far = t.arange(pages - n, pages, device="cuda", dtype=t.int32)[None]
    want, wl, _ = c.call()
    got, gl, st = c.call(k_cache=big[0], v_cache=big[1], page_table=far)
    assert st == 0 and bool((got == want).all()) and bool((gl == wl).all())


def test_graph_capture_with_new_lengths():
    t = torch()
    import awq_int4_moe_gb300 as awq
    c = Case([900, 40, 333], 8, 2, 128, "f16", "f16", 16)
    out, st = t.empty_like(c.q), t.zeros(1, dtype=t.int32, device="cuda")
    lse = t.empty((3, 8), device="cuda")
    ws = workspace(128)

    def go():
        awq.paged_attention(c.q, c.kc, c.vc, c.table, c.seq, out, ws, st, scale=c.scale, lse=lse)

    go()
    t.cuda.synchronize()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        go()
    for lens in ([900, 40, 333], [1, 0, 17], [500, 40, 300]):
        c.seq.copy_(t.tensor(lens, dtype=t.int32))
        c.lens = lens
        graph.replay()
        t.cuda.synchronize()
        assert int(st) == 0
        c.check(out, lse)


@pytest.mark.parametrize("kind,cache", TYPES)
def test_weights_of_tokens_that_cancel(kind, cache):
    """Two tokens with weights of any 24 bits and values that nearly cancel: the
    rounding of the weights shows. Scores are one product each, so a weight's
    error is that of the score's scaling (8 roundings of |s| log2 e <= 1.5), of
    the exponential and of its two 16-bit terms: 2^-20 with fp16, and 2^-17 (8 +
    8 bits and the sign of the second term) with bf16."""
    t = torch()
    n, dim, heads = 2, 64, 8
    c = Case([n] * 40, heads, 1, dim, kind, cache, 16, seed=7)
    g = t.Generator(device="cuda")
    g.manual_seed(8)
    first = c.table[:, 0].long()
    k, v = t.zeros(c.kc.shape, device="cuda"), t.zeros(c.vc.shape, device="cuda")
    k[first, 1, 0, 0] = 8.0                                      # token 0 scores 0
    c.kc.copy_(k.to(c.kc.dtype))
    c.scales = (1.0, 1.0)
    c.scale = 0.125
    c.q.zero_()
    c.q[:, :, 0] = -t.rand((len(c.lens), 1), generator=g, device="cuda").to(c.q.dtype)    # token 1 between -1 and 0
    weight = t.exp(c.q[:, 0, 0].double())
    v[first, 1, 0] = t.randn((len(c.lens), dim), generator=g, device="cuda")
    c.vc.copy_(v.to(c.vc.dtype))
    v[first, 0, 0] = (-weight[:, None] * c.vc[first, 1, 0].double()).float()
    c.vc.copy_(v.to(c.vc.dtype))
    out, lse, st = c.call()
    assert st == 0
    u = 2.0 ** -11 if kind == "f16" else 2.0 ** -8
    split = 2.0 ** -17 if cache == "bf16" else 2.0 ** -20
    fine = 0
    for b in range(len(c.lens)):
        keys, values = c.rows(b)
        s = t.einsum("hd,nhd->hn", c.q[b].double(), keys.expand(n, heads, dim)) * c.scale
        p = t.softmax(s, 1)
        want = t.einsum("hn,nhd->hd", p, values.expand(n, heads, dim))
        size = t.einsum("hn,nhd->hd", p, values.abs().expand(n, heads, dim))
        tol = want.abs() * u + (split + 8 * 1.5 * 2.0 ** -24 + 8 * 2.0 ** -24) * size + 2.0 ** -25
        err = (out[b].double() - want).abs()
        assert bool((err <= tol).all()), f"sequence {b}: {float((err / tol).max())} times the tolerance"
        fine += int((tol < 2.0 ** -13 * size).sum())
    assert cache == "bf16" or fine > 100                       # outputs at which one fp16 term would show


@pytest.mark.parametrize("kind,cache", TYPES)
def test_strides_of_dimensions_of_one_are_not_used(kind, cache):
    """One sequence, KV head and page: the strides between them carry nothing,
    so odd ones change neither the result nor what is accepted."""
    t = torch()
    c = Case([13], 1, 1, 64, kind, cache, 16, spare=0)
    want, wl, st = c.call()
    assert st == 0

    def odd(x, *dims):
        strides = list(x.stride())
        for d in dims:
            assert x.shape[d] == 1
            strides[d] = 67
        return x.as_strided(x.shape, strides)

    out = t.full_like(c.q, 9.0)
    got, gl, st = c.call(q=odd(c.q, 0, 1), k_cache=odd(c.kc, 0, 2), v_cache=odd(c.vc, 0), out=odd(out, 0, 1))
    assert st == 0 and t.equal(got, want) and t.equal(gl, wl)
    c = Case([1], 1, 1, 64, kind, cache, 1, spare=0)           # pages of one token
    want, wl, st = c.call()
    got, gl, st = c.call(k_cache=odd(c.kc, 0, 1, 2), v_cache=odd(c.vc, 1))
    assert st == 0 and t.equal(got, want) and t.equal(gl, wl)
    c.check(got, gl)


@pytest.mark.parametrize("kind,cache", TYPES)
@pytest.mark.parametrize("group,hk", [(17, 3), (24, 4), (40, 2)])
def test_many_heads_of_several(kind, cache, group, hk):
    """More than one tile of query heads and more than one KV head."""
    run([33, 0, 700, 1], group * hk, hk, 128, kind, cache, 16, seed=group)
    run([90, 5], group * hk, hk, 64, kind, cache, 5, seed=group)


@pytest.mark.parametrize("kind,cache", TYPES)
@pytest.mark.parametrize("page", [1, 5, 16, 48])
@pytest.mark.parametrize("k_first", [False, True])
def test_planes_of_different_strides(kind, cache, page, k_first):
    """K's pages with heads before tokens and V's with tokens before heads, and
    the other way round."""
    c = Case(EDGES, 8, 2, 128, kind, cache, page, heads_first=k_first, seed=page)
    other = c.vc.transpose(1, 2).contiguous().transpose(1, 2) if not k_first else c.vc.contiguous()
    assert c.page == 1 or other.stride() != c.kc.stride()
    out, lse, st = c.call(v_cache=other)
    assert st == 0
    c.check(out, lse)
    want, wl, _ = c.call()
    assert bool((out == want).all()) and bool((lse == wl).all())


@pytest.mark.parametrize("kind,cache", [("f16", "f16"), ("bf16", "bf16")])
def test_sums_of_few_tokens(kind, cache):
    """As check(), with the additions that a few units make in a row: a chain of
    products per unit, the units of a warp, at most 24 parts of a block and 8
    pieces of a segment cut between blocks, and the two bf16 terms' own 2^-17."""
    t = torch()
    c = Case([1, 2, 7, 16, 40, 64], 8, 2, 64, kind, cache, 16, seed=3)
    out, lse, st = c.call()
    assert st == 0
    u = 2.0 ** -11 if kind == "f16" else 2.0 ** -8
    for b, n in enumerate(c.lens):
        k, v = c.rows(b)
        q = c.q[b].double().view(2, 4, 64)
        s = t.einsum("hgd,nhd->hgn", q, k) * c.scale
        want = t.einsum("hgn,nhd->hgd", t.softmax(s, 2), v).reshape(8, 64)
        d = (64 + 8) * 2.0 ** -23 * float(q.norm(dim=2).max() * k.norm(dim=2).max()) * c.scale
        sums = (n + 40) * 2.0 ** -24
        split = 2.0 ** -20 if cache == "f16" else 2.0 ** -17
        tol = want.abs() * u + (2 * d + split + 2 * sums) * float(v.abs().max()) + 2.0 ** -25
        err = (out[b].double() - want).abs()
        assert bool((err <= tol).all()), f"sequence {b}: {float((err / tol).max())} times the tolerance"


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_values_that_are_not_finite_stay_in_their_column(kind, bad):
    """NaN or infinite there, whichever; every other output keeps its bits."""
    t = torch()
    c = Case([40, 700, 17], 8, 2, 128, kind, kind, 16, seed=4)
    want, wl, _ = c.call()
    c.vc[c.table[0, 1].long(), 3, 0, 5] = bad
    c.vc[c.table[1, 40].long(), 0, 1, 9] = bad
    out, lse, st = c.call()
    assert st == 0
    hit = t.zeros_like(out, dtype=t.bool)
    hit[0, :4, 5] = True
    hit[1, 4:, 9] = True
    assert bool((out.isfinite() != hit).all())
    assert bool((out == want)[~hit].all()) and bool((lse == wl).all())
