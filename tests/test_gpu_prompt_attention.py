"""awq_prompt_attention and awq_chunk_attention against 64-bit results.

Tolerances. A score is a dot product of D terms, added by the tensor core in
fp32 in steps of 16 that may truncate, and one scaling: it is off by at most d =
(D + 16) 2^-22 scale |q||k|. So a weight is off by 2 d relative, 2^-20 for the
exponential, and by its rounding to the tensor core's type where it is
multiplied with v: half a step, w = 2^-11 (fp16) or 2^-8 (bf16), or for fp16
2^-32 of the largest weight where it is that small. Sums over n keys: n / 16 + 400
additions in a row (tensor core, tiles, joined pieces) at 2^-23 each. Errors of
weights move the output by at most their size times sum_j p_j |v_j|; then one
rounding (u, half a step of the output's type)."""
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
    size = awq.prompt_attention_workspace_bytes(dim)
    if size not in _WS:
        _WS[size] = torch().zeros(size, dtype=torch().uint8, device="cuda")
    return _WS[size]


class Case:
    """A batch of sequences (tokens, new ones); cache None: whole prompts, packed."""

    def __init__(self, lens, news, hq, hk, dim, kind, cache=None, page=16, heads_first=False, seed=0, q_std=1.0, behind=0, spare=2):
        t = torch()
        g = t.Generator(device="cuda")
        g.manual_seed(seed)
        self.packed = cache is None
        self.lens, self.news = lens, lens if news is None else news
        self.hq, self.hk, self.dim, self.kind, self.page = hq, hk, dim, kind, page
        self.core = "f16" if cache == "e4m3" else kind                    # the tensor core's type
        self.cu = [0]
        for n in self.news:
            self.cu.append(self.cu[-1] + n)
        self.rows = self.cu[-1] + behind
        self.cu_t = t.tensor(self.cu, dtype=t.int32, device="cuda")
        self.q = (t.randn((self.rows, hq, dim), generator=g, device="cuda") * q_std).to(dtype_of(kind))
        self.scale = dim ** -0.5
        self.scales = (0.025, 0.03) if cache == "e4m3" else (1.0, 1.0)
        if self.packed:
            self.k, self.v = (t.randn((self.rows, hk, dim), generator=g, device="cuda").to(dtype_of(kind)) for _ in range(2))
            return
        need = [-(-n // page) for n in lens]
        pages = sum(need) + spare
        shape = (pages, hk, page, dim) if heads_first else (pages, page, hk, dim)
        std = 40.0 if cache == "e4m3" else 1.0
        self.kc, self.vc = ((t.randn(shape, generator=g, device="cuda") * std).to(dtype_of(cache)) for _ in range(2))
        if heads_first:
            self.kc, self.vc = self.kc.transpose(1, 2), self.vc.transpose(1, 2)
        order = t.randperm(pages, generator=g, device="cuda").int().cpu()
        self.table = t.full((len(lens), max(1, max(need, default=1))), -5, dtype=t.int32)    # unneeded entries: no page
        at = 0
        for i, n in enumerate(need):
            self.table[i, :n] = order[at:at + n]
            at += n
        self.free = order[at:]
        self.table = self.table.cuda()
        self.seq = t.tensor(lens, dtype=t.int32, device="cuda")

    def call(self, **over):
        import awq_int4_moe_gb300 as awq
        t = torch()
        st = t.zeros(1, dtype=t.int32, device="cuda")
        a = dict(q=self.q, cu_seqlens=self.cu_t, out=t.full((self.rows, self.hq, self.dim), 9.0, device="cuda", dtype=dtype_of(self.kind)),
                 workspace=workspace(self.dim), dev_status=st, scale=self.scale,
                 lse=t.full((self.rows, self.hq), 9.0, device="cuda"))
        if self.packed:
            a.update(k=self.k, v=self.v)
        else:
            a.update(k_cache=self.kc, v_cache=self.vc, page_table=self.table, seq_lens=self.seq, k_scale=self.scales[0],
                     v_scale=self.scales[1])
        a.update(over)
        (awq.prompt_attention if self.packed else awq.chunk_attention)(**a)
        t.cuda.synchronize()
        return a["out"], a["lse"], int(st)

    def kv(self, b):
        """k, v of a sequence, 64 bits: [tokens][KV heads][dim]."""
        n = self.lens[b]
        if self.packed:
            at = self.cu[b]
            return self.k[at:at + n].double(), self.v[at:at + n].double()
        pages = self.table[b, : -(-n // self.page)].long()
        take = lambda c, s: c.float()[pages].reshape(-1, self.hk, self.dim)[:n].double() * s  # noqa: E731
        return take(self.kc, self.scales[0]), take(self.vc, self.scales[1])

    def check(self, out, lse, sequences=None):
        t = torch()
        u = 2.0 ** -11 if self.kind == "f16" else 2.0 ** -8
        w = 2.0 ** -11 if self.core == "f16" else 2.0 ** -8
        for b in range(len(self.lens)) if sequences is None else sequences:
            n, new, at = self.lens[b], self.news[b], self.cu[b]
            if new == 0:
                continue
            first = n - new                                              # position of the first new token
            empty = max(0, min(new, -first))                             # rows before the cache's first token
            got, got_lse = out[at:at + new], lse[at:at + new]
            assert bool((got[:empty] == 0).all()) and bool((got_lse[:empty] == -math.inf).all())
            if empty == new:
                continue
            k, v = self.kv(b)
            group = self.hq // self.hk
            q = self.q[at + empty:at + new].double().view(new - empty, self.hk, group, self.dim)
            s = t.einsum("ihgd,nhd->hgin", q, k) * self.scale
            hidden = t.arange(n, device="cuda") > first + t.arange(empty, new, device="cuda")[:, None]
            s.masked_fill_(hidden, -math.inf)
            p = t.softmax(s, 3)
            want = t.einsum("hgin,nhd->ihgd", p, v).reshape(new - empty, self.hq, self.dim)
            size = t.einsum("hgin,nhd->ihgd", p, v.abs()).reshape(new - empty, self.hq, self.dim)
            d = (self.dim + 16) * 2.0 ** -22 * float(q.norm(dim=3).max() * k.norm(dim=2).max()) * abs(self.scale)
            sums = (n / 16 + 400) * 2.0 ** -23
            small = n * 2.0 ** -32 * float(v.abs().max()) if self.core == "f16" else 0.0
            tol = want.abs() * u + (2 * d + 2.0 ** -20 + w + 2 * sums) * size + small + 2.0 ** -25
            err = (got[empty:].double() - want).abs()
            assert bool((err <= tol).all()), f"sequence {b}: {float((err - tol).max())} over {float(tol.min())}, at {(err - tol).argmax()}"
            ref = t.logsumexp(s, 3).permute(2, 0, 1).reshape(new - empty, self.hq)
            err = (got_lse[empty:].double() - ref).abs()
            assert bool((err <= d + 2.0 ** -20 + sums + 2.0 ** -22 * ref.abs()).all()), f"lse {b}: {float(err.max())}"
        behind = slice(self.cu[-1], self.rows)
        assert bool((out[behind] == 9.0).all()) and bool((lse[behind] == 9.0).all())      # left as they were


def run(*args, **kw):
    c = Case(*args, **kw)
    out, lse, st = c.call()
    assert st == 0
    c.check(out, lse)
    return c


TYPES = [("f16", "f16"), ("bf16", "bf16"), ("f16", "e4m3"), ("bf16", "e4m3")]
PROMPTS = [1, 0, 2, 15, 64, 127, 128, 129, 300, 0]
CHUNKS = ([1, 15, 16, 17, 130, 700, 64, 1000, 5, 0], [1, 1, 5, 17, 3, 200, 64, 9, 0, 0])


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [128, 64, 256])
def test_one_tile(kind, dim):
    run([16], None, 1, 1, dim, kind)
    run([128], None, 1, 1, dim, kind)
    run([100], [100], 2, 1, dim, kind, kind)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [8, 16, 64, 72, 80, 96, 128, 136, 200, 256])
@pytest.mark.parametrize("group", [1, 5, 8])
def test_prompts(kind, dim, group):
    run(PROMPTS, None, 2 * group, 2, dim, kind, seed=dim + group, behind=3)


@pytest.mark.parametrize("kind,cache", TYPES)
@pytest.mark.parametrize("dim", [16, 64, 80, 128, 144, 256])
@pytest.mark.parametrize("group", [1, 5, 16])
def test_chunks(kind, cache, dim, group):
    run(*CHUNKS, 2 * group, 2, dim, kind, cache, seed=dim + group, behind=3)


@pytest.mark.parametrize("group", [17, 40, 129, 300])
def test_many_heads_of_one(group):
    run([33, 0, 300], None, group, 1, 64, "f16")
    run([33, 500, 300], [2, 1, 30], group, 1, 64, "bf16", "e4m3")


@pytest.mark.parametrize("page", [1, 3, 16, 24, 64, 128, 200, 256])
@pytest.mark.parametrize("heads_first", [False, True])
def test_pages(page, heads_first):
    run(*CHUNKS, 8, 2, 128, "f16", "f16", page, heads_first, seed=page)
    run(*CHUNKS, 8, 2, 128, "bf16", "e4m3", page, heads_first, seed=page)


@pytest.mark.parametrize("kind,cache", TYPES)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("news", [1, 7, 40, 300])
def test_long_contexts_are_cut_and_joined(kind, cache, dim, news):
    run([20000], [news], 4, 1, dim, kind, cache, 64, seed=news)
    run([3, 9000, 1, 12345], [1, news, 1, news], 8, 2, dim, kind, cache, 64, seed=news)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("lens", [[1], [2000], [4100], [1500, 1, 700, 1300], [77] * 150])
def test_lengths_of_prompts(dim, lens):
    run(lens, None, 8, 2, dim, "bf16", seed=len(lens))


def test_more_sequences_than_threads():
    lens = [(i * 37) % 90 for i in range(1500)]
    run(lens, None, 4, 2, 64, "f16")
    run(lens, [min(n, 1 + i % 3) for i, n in enumerate(lens)], 4, 2, 64, "f16", "f16")


def test_more_new_tokens_than_the_cache_has():
    """Rows before the cache's first token see nothing: zeros and -infinity."""
    for dim in (64, 128, 256):
        run([5, 0, 130, 40], [9, 4, 400, 300], 6, 2, dim, "f16", "f16")
    run([5, 0, 130, 40], [9, 4, 400, 300], 6, 2, 128, "bf16", "e4m3")


def test_peaked_scores():
    run(PROMPTS, None, 8, 2, 128, "f16", q_std=60.0)
    run(PROMPTS, None, 8, 2, 128, "bf16", q_std=60.0)
    run(*CHUNKS, 8, 2, 128, "bf16", "e4m3", q_std=1e6)                    # past fp16's range before the scale
    run(*CHUNKS, 8, 2, 128, "bf16", "e4m3", q_std=1e-30)


@pytest.mark.parametrize("kind,cache", TYPES + [("f16", None), ("bf16", None)])
@pytest.mark.parametrize("scale", [0.0, -0.0, -0.1, 1e-40])
def test_scales_of_zero_and_below(kind, cache, scale):
    c = Case(CHUNKS[0], CHUNKS[1] if cache else None, 8, 2, 128, kind, cache)
    c.scale = scale
    out, lse, st = c.call()
    assert st == 0
    c.check(out, lse)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_rising_scores_raise_the_maximum_again_and_again(kind):
    """Key j's score grows with j in steps past every threshold."""
    for dim in (64, 128, 256):
        c = Case([2000], None, 4, 1, dim, kind)
        c.k.zero_()
        c.k[:, :, 0] = torch().arange(2000, device="cuda")[:, None].to(c.k.dtype)
        c.q.zero_()
        c.q[:, :, 0] = 1.0
        out, lse, st = c.call()
        assert st == 0
        c.check(out, lse)


@pytest.mark.parametrize("kind,cache", TYPES + [("f16", None), ("bf16", None)])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_values_that_a_row_does_not_see_do_not_reach_it(kind, cache, dim):
    """NaN and infinities in the last tokens: rows before them have the same bits
    as with zeros there, rows that see them have NaN in their columns alone."""
    t = torch()
    results = []
    lens, news = [300, 90], [40, 30]
    for bad in (0.0, float("nan"), 448.0 if cache == "e4m3" else float("inf")):
        c = Case(lens, news if cache else None, 4, 2, dim, kind, cache, seed=4)
        for b in range(2):
            for back in (1, 7, 20):
                j = lens[b] - back
                if cache is None:
                    c.k[c.cu[b] + j, 1] = bad
                    c.v[c.cu[b] + j, :, 5] = bad
                    c.v[c.cu[b] + j, 0, dim - 1] = bad
                else:
                    page, at = c.table[b, j // 16].long(), j % 16
                    for plane, where in ((c.kc, (page, at, 1)), (c.vc, (page, at, slice(None), 5)), (c.vc, (page, at, 0, dim - 1))):
                        raw = plane.float()
                        raw[where] = bad
                        plane.copy_(raw.to(plane.dtype))
        out, lse, st = c.call()
        assert st == 0
        results.append((out, lse))
    for i, (out, lse) in enumerate(results[1:]):
        finite = i == 1 and cache == "e4m3"                               # (e4m3 has no infinity: its largest value)
        for b in range(2):
            end = c.cu[b + 1]
            before = slice(c.cu[b], end - 20)
            assert bool((out[before] == results[0][0][before]).all()) and bool((lse[before] == results[0][1][before]).all())
            seen = out[end - 20:end]
            if finite:
                assert bool(seen.isfinite().all())
                continue
            head0 = seen[:, :2]                                          # KV head 0: K is finite, V's columns 5 and the last are not
            where = t.zeros(dim, dtype=t.bool, device="cuda")
            where[5] = where[dim - 1] = True
            assert bool(head0[:, :, where].isnan().all()) and bool(head0[:, :, ~where].isfinite().all())
            assert bool(lse[end - 20:end, :2].isfinite().all())


def test_values_past_the_end_do_not_matter():
    """NaN in free pages and in the places after a sequence's last token."""
    results = []
    for cache in ("f16", "e4m3"):
        for bad in (0.0, float("nan")):
            c = Case([1, 17, 50, 0, 111], [1, 5, 50, 0, 2], 8, 2, 128, "f16", cache, 16, seed=4)
            for plane in (c.kc, c.vc):
                raw = plane.float()
                raw[c.free.long().cuda()] = bad
                for b, n in enumerate(c.lens):
                    if n % 16:
                        raw[c.table[b, n // 16].long(), n % 16:] = bad
                plane.copy_(raw.to(plane.dtype))
            out, lse, st = c.call()
            assert st == 0
            c.check(out, lse)
            results.append((out, lse))
        assert bool((results[-1][0] == results[-2][0]).all()) and bool((results[-1][1] == results[-2][1]).all())


def test_same_bits_every_time_and_on_a_side_stream():
    t = torch()
    for c in (Case([3000, 5, 900, 0, 12000], [300, 5, 1, 0, 20], 10, 2, 128, "f16", "f16", 16), Case([3000, 1, 500], None, 8, 2, 128, "bf16")):
        first = c.call()
        for _ in range(5):
            again = c.call()
            assert bool((again[0] == first[0]).all()) and bool((again[1] == first[1]).all())
        side = t.cuda.Stream()
        side.wait_stream(t.cuda.current_stream())
        again = c.call(stream=side)
        assert bool((again[0] == first[0]).all())


def test_strides_of_everything():
    t = torch()
    c = Case([100, 7], None, 8, 2, 128, "f16")
    want, want_lse, _ = c.call()
    wide = t.zeros((c.rows, 12, 192), device="cuda", dtype=t.float16)
    for part, of in ((wide[:, 0:8, :128], c.q), (wide[:, 8:10, :128], c.k), (wide[:, 10:12, 64:], c.v)):
        part.copy_(of)
    out = t.full((8, c.rows, 128), 9.0, device="cuda", dtype=t.float16).transpose(0, 1)
    got, lse, st = c.call(q=wide[:, 0:8, :128], k=wide[:, 8:10, :128], v=wide[:, 10:12, 64:], out=out)
    assert st == 0 and bool((got == want).all()) and bool((lse == want_lse).all())
    got, lse, st = c.call(lse=None)
    assert st == 0 and lse is None and bool((got == want).all())
    shared = c.k[:, :1].expand(-1, 2, -1)                               # one KV head for both, by a stride of 0
    got, _, st = c.call(k=shared)
    other = Case([100, 7], None, 8, 2, 128, "f16")
    other.k = shared.contiguous()
    assert st == 0
    other.check(got, other.call()[1])


def test_shared_pages():
    """Two sequences whose first pages are the same ones."""
    c = Case([64, 70], [3, 40], 4, 2, 64, "f16", "f16", 16)
    c.table[1, :4] = c.table[0, :4]
    out, lse, st = c.call()
    assert st == 0
    c.check(out, lse)


def test_graph_replays_with_other_lengths():
    t = torch()
    c = Case([900, 40, 300], [100, 1, 20], 8, 2, 128, "f16", "f16", 16)
    out, lse, _ = c.call()
    g = t.cuda.CUDAGraph()
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    import awq_int4_moe_gb300 as awq
    st = t.zeros(1, dtype=t.int32, device="cuda")
    with t.cuda.graph(g):
        awq.chunk_attention(c.q, c.kc, c.vc, c.table, c.cu_t, c.seq, out, workspace(128), st, scale=c.scale, lse=lse)
    for lens in ([900, 40, 300], [500, 17, 21], [100, 0, 299]):
        c.lens = lens
        c.seq.copy_(t.tensor(lens, dtype=t.int32))
        out.fill_(9.0)
        lse.fill_(9.0)
        g.replay()
        t.cuda.synchronize()
        assert int(st) == 0
        c.check(out, lse)


def test_bad_pages_lengths_and_bounds_are_reported():
    import awq_int4_moe_gb300 as awq
    t = torch()
    for cache in ("f16", "e4m3"):
        for bad in (-1, 1 << 30):
            c = Case([40, 200, 33], [4, 50, 33], 8, 2, 128, "f16", cache, 16)
            c.table[1, 3] = bad
            out, lse, st = c.call()
            assert st == awq.ERR_BAD_INDEX
            c.check(out, lse, [0, 2])
    for bad in (-1, 13 * 16 + 1):
        c = Case([40, 200, 33], [4, 50, 33], 8, 2, 128, "f16", "f16", 16)
        c.table[:] = c.table.clamp(min=0)
        c.seq[1] = bad
        out, lse, st = c.call()
        assert st == awq.ERR_BAD_INDEX
        c.check(out, lse, [0, 2])
    for cu in ([-3, 40, 60, 93], [0, 40, 30, 93], [0, 40, 60, 94], [0, 1 << 30, 60, 93]):
        c = Case([40, 20, 33], None, 8, 2, 128, "f16")
        out, lse, st = c.call(cu_seqlens=t.tensor(cu, dtype=t.int32, device="cuda"))
        assert st == awq.ERR_BAD_INDEX
    out, lse, st = c.call()                                             # the workspace is ready again
    assert st == 0
    c.check(out, lse)


def test_cache_past_32_bit_offsets():
    t = torch()
    c = Case([50], [20], 8, 8, 128, "f16", "f16", 16)
    pages = 140000                               # 2.3 G elements a plane
    big = [t.zeros((pages, 16, 8, 128), device="cuda", dtype=t.float16) for _ in range(2)]
    far = t.tensor([pages - 1, 139000, 131072 + 7, 135000], device="cuda")
    for plane, of in zip(big, (c.kc, c.vc)):
        plane[far] = of[c.table[0].long()]
    want, _, _ = c.call()
    got, lse, st = c.call(k_cache=big[0], v_cache=big[1], page_table=far[None].int())
    assert st == 0 and bool((got == want).all())


@pytest.mark.parametrize("kind,cache", TYPES)
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_values_that_some_rows_do_not_see_in_cut_units(kind, cache, dim):
    """Long contexts, cut between blocks, and one that is not: the last token's value
    and all places behind it not finite. Only the last token's rows see that, the
    others keep every bit."""
    t = torch()
    c = Case([9000, 20000, 130, 257], [3, 200, 130, 1], 8, 2, dim, kind, cache, page=16, seed=dim)
    before, lse, st = c.call()
    assert st == 0
    c.check(before, lse)
    bad = t.full((), math.nan, device="cuda").to(c.vc.dtype)
    last = []
    for b, n in enumerate(c.lens):
        page, place = int(c.table[b, (n - 1) // 16]), (n - 1) % 16
        c.vc[page, place, :, 5:9] = bad
        c.vc[page, place + 1:] = bad
        c.kc[page, place + 1:] = bad
        last.append(c.cu[b + 1] - 1)
    out, lse2, st = c.call()
    assert st == 0 and t.equal(lse, lse2)
    rows = t.zeros(c.rows, dtype=t.bool, device="cuda")
    rows[last] = True
    assert t.equal(out[~rows], before[~rows])
    assert bool(out[rows][:, :, 5:9].isnan().all())
    keep = t.ones(dim, dtype=t.bool, device="cuda")
    keep[5:9] = False
    assert t.equal(out[rows][:, :, keep], before[rows][:, :, keep])


@pytest.mark.parametrize("cache", [None, "f16"])
def test_rows_before_the_first_sequence_and_repeated_heads_of_q(cache):
    """Bounds that begin past 0 leave the rows before them; a query that is the same
    for all heads, by a stride of 0."""
    t = torch()
    c = Case([200, 31], None if cache is None else [40, 31], 4, 2, 128, "f16", cache, seed=3)
    shift = 7
    c.q = c.q[:, :1].expand(-1, 4, -1)
    want, want_lse, st = c.call()
    assert st == 0
    c.check(want, want_lse)
    pad = lambda x: t.cat([x.new_full((shift,) + x.shape[1:], math.nan), x])  # noqa: E731
    c.q, c.rows, c.cu_t = pad(c.q), c.rows + shift, c.cu_t + shift
    if cache is None:
        c.k, c.v = pad(c.k), pad(c.v)
    out, lse, st = c.call()
    assert st == 0 and bool((out[:shift] == 9).all()) and bool((lse[:shift] == 9).all())
    # (a stride of 0 takes the rows of q one by one, a copy of its own in boxes: the same numbers)
    assert t.equal(out[shift:], want) and t.equal(lse[shift:], want_lse)
