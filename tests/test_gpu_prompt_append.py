"""awq_qk_norm_rope_append against 64-bit results.

Tolerances. A head's sum of squares is a sum of up to D fp32 terms, its root and
the two scalings a handful of roundings: y is off by at most (D + 16) 2^-24
relative (half of the sum's error, as it goes under a root, and 8 roundings). A
turned element is two products of such values: off by at most that, and 4
roundings, times |a cos| + |b sin|. Then one rounding (u, half a step of the
type); e4m3 rounds to within 2^-4 relative, or 2^-10 absolute where it is
subnormal, after the scale's two roundings."""
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


class Case:
    def __init__(self, tokens, hq, hk, dim, rotary, kind, cache, page=16, interleaved=False, heads_first=False, seed=0, std=3.0, unused=0,
                 eps=1e-6):
        t = torch()
        g = t.Generator(device="cuda")
        g.manual_seed(seed)
        dt = dtype_of(kind)
        self.tokens, self.hq, self.hk, self.dim, self.rotary, self.kind, self.cache = tokens, hq, hk, dim, rotary, kind, cache
        self.page, self.interleaved, self.unused, self.eps = page, interleaved, unused, eps
        self.q, self.k, self.v = ((t.randn((tokens, h, dim), generator=g, device="cuda") * std).to(dt) for h in (hq, hk, hk))
        self.qw, self.kw = ((1 + 0.3 * t.randn(dim, generator=g, device="cuda")).to(dt) for _ in range(2))
        self.positions = t.randint(0, 500, (tokens,), generator=g, device="cuda").int()
        angle = t.arange(500, device="cuda", dtype=t.float64)[:, None] * \
            1000.0 ** (-t.arange(0, max(rotary, 1), 2, device="cuda", dtype=t.float64)[: rotary // 2] / max(rotary, 1))
        self.table = t.cat([angle.cos(), angle.sin()], 1).float()
        pages = -(-tokens // page) + 2
        shape = (pages, hk, page, dim) if heads_first else (pages, page, hk, dim)
        self.kc, self.vc = (t.full(shape, 7.0, device="cuda").to(dtype_of(cache)) for _ in range(2))
        if heads_first:
            self.kc, self.vc = self.kc.transpose(1, 2), self.vc.transpose(1, 2)
        self.scales = (0.03, 0.05) if cache == "e4m3" else (1.0, 1.0)
        self.slots = t.randperm(pages * page, generator=g, device="cuda")[:tokens]
        self.slots[tokens - unused:] = -1

    def call(self, **over):
        import awq_int4_moe_gb300 as awq
        t = torch()
        st = t.zeros(1, dtype=t.int32, device="cuda")
        a = dict(q=self.q, k=self.k, v=self.v, q_weight=self.qw, k_weight=self.kw, eps=self.eps, positions=self.positions,
                 cos_sin=self.table, slots=self.slots, k_cache=self.kc, v_cache=self.vc, dev_status=st, q_out=t.empty_like(self.q),
                 interleaved=self.interleaved, k_scale=self.scales[0], v_scale=self.scales[1])
        a.update(over)
        awq.qk_norm_rope_append(**a)
        t.cuda.synchronize()
        return a["q"] if a["q_out"] is None else a["q_out"], int(st)

    def turned(self, x, w):
        """The normed and turned heads in 64 bits, and how far they may be off."""
        t = torch()
        x = x.double()
        y = x / (x.square().mean(2, keepdim=True) + self.eps).sqrt() * w.double()
        half = self.rotary // 2
        i = t.arange(half, device="cuda")
        a, b = (2 * i, 2 * i + 1) if self.interleaved else (i, i + half)
        row = self.table[self.positions.long()].double()
        cos, sin = row[:, None, :half], row[:, None, half:]
        z, size = y.clone(), y.abs()
        z[..., a], z[..., b] = y[..., a] * cos - y[..., b] * sin, y[..., b] * cos + y[..., a] * sin
        s = size.clone()
        s[..., a] = size[..., a] * cos.abs() + size[..., b] * sin.abs()
        s[..., b] = size[..., b] * cos.abs() + size[..., a] * sin.abs()
        return z, s * (self.dim + 24) * 2.0 ** -24

    def rounded(self, got, want, tol, scale=1.0):
        """got: as fp32; want in 64 bits."""
        if scale == 1.0:
            u = 2.0 ** -11 if self.kind == "f16" else 2.0 ** -8
            return bool(((got.double() - want).abs() <= tol * (1 + u) + want.abs() * u + 2.0 ** -25).all())
        top = 448.0
        want = (want / scale).clamp(-top, top)
        tol = tol / scale + want.abs() * 2.0 ** -22
        return bool(((got.double() - want).abs() <= tol * 1.1 + want.abs() * 2.0 ** -4 + 2.0 ** -10).all())

    def check(self, q_out):
        t = torch()
        assert self.rounded(q_out.float(), *self.turned(self.q, self.qw))
        kept = self.tokens - self.unused
        page, at = self.slots[:kept] // self.page, self.slots[:kept] % self.page
        z, tol = self.turned(self.k, self.kw)
        kf, vf = self.kc.float(), self.vc.float()
        s = self.scales if self.cache == "e4m3" else (1.0, 1.0)
        assert self.rounded(kf[page, at], z[:kept], tol[:kept], s[0])
        assert self.rounded(vf[page, at], self.v.double()[:kept], t.zeros((), device="cuda"), s[1])
        untouched = t.ones(kf.shape[:2], dtype=t.bool, device="cuda")
        untouched[page, at] = False
        assert bool((kf[untouched] == 7.0).all()) and bool((vf[untouched] == 7.0).all())


def run(*args, **kw):
    c = Case(*args, **kw)
    q, st = c.call()
    assert st == 0
    c.check(q)
    return c


TYPES = [("f16", "f16"), ("bf16", "bf16"), ("f16", "e4m3"), ("bf16", "e4m3")]


@pytest.mark.parametrize("kind,cache", TYPES)
@pytest.mark.parametrize("dim,rotary", [(64, 64), (80, 80), (96, 48), (128, 128), (128, 64), (256, 256), (256, 64), (1024, 1024), (512, 32),
                                        (64, 0), (576, 64), (8, 8), (6, 2), (1, 0), (77, 38), (1000, 500)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_heads(kind, cache, dim, rotary, interleaved):
    run(17, 5, 2, dim, rotary, kind, cache, interleaved=interleaved, seed=dim + rotary)


@pytest.mark.parametrize("tokens", [1, 2, 33, 1300, 3001])
@pytest.mark.parametrize("heads", [(1, 1), (20, 4), (40, 8), (7, 1), (64, 8)])
def test_tokens_and_head_counts(tokens, heads):
    run(tokens, *heads, 128, 128, "f16", "f16", seed=tokens)
    run(tokens, *heads, 128, 64, "bf16", "e4m3", interleaved=True, seed=tokens)


@pytest.mark.parametrize("tokens", [10, 2000])
@pytest.mark.parametrize("dim,rotary", [(1024, 1024), (1024, 64), (321, 64)])
def test_long_heads(tokens, dim, rotary):
    run(tokens, 6, 1, dim, rotary, "bf16", "bf16")
    run(tokens, 6, 1, dim, rotary, "f16", "e4m3", interleaved=True)


@pytest.mark.parametrize("page", [1, 3, 16, 64])
@pytest.mark.parametrize("heads_first", [False, True])
def test_pages_and_unused_tokens(page, heads_first):
    run(50, 8, 2, 128, 128, "f16", "f16", page, heads_first=heads_first, unused=7)
    run(50, 8, 2, 128, 128, "bf16", "e4m3", page, heads_first=heads_first, unused=50)


def test_strides_and_in_place():
    t = torch()
    for kind, dim, at in (("f16", 128, 0), ("bf16", 96, 3)):             # 3: rows at odd addresses
        c = Case(40, 8, 2, dim, dim, kind, kind)
        want, _ = c.call()
        k_want = c.kc.clone()
        wide = t.zeros((40, 12, dim + 40), device="cuda", dtype=c.q.dtype)
        parts = wide[:, 0:8, at:at + dim], wide[:, 8:10, at:at + dim], wide[:, 10:12, at:at + dim]
        for part, of in zip(parts, (c.q, c.k, c.v)):
            part.copy_(of)
        c.kc.fill_(7.0)
        got, st = c.call(q=parts[0], k=parts[1], v=parts[2], q_out=None)
        assert st == 0
        c.check(got)
        c.check(want)
        if at == 0:
            assert bool((got == want).all()) and bool((c.kc == k_want).all())


def test_weights_at_odd_addresses():
    t = torch()
    c = Case(9, 4, 2, 64, 64, "f16", "f16")
    w = t.empty(65, device="cuda", dtype=t.float16)
    w[1:] = c.qw
    got, st = c.call(q_weight=w[1:])
    assert st == 0
    c.check(got)


def test_small_and_large_heads():
    t = torch()
    c = Case(8, 2, 1, 128, 128, "bf16", "bf16")
    c.q[0] = 0.0                                                         # eps alone
    c.q[1] = 1e-20
    c.q[2] = 1e18
    c.q[3] = 3e38                                                        # the sum of squares passes fp32's range
    got, st = c.call()
    assert st == 0 and bool((got[0] == 0).all()) and bool((got[3] == 0).all())
    keep = [0, 1, 2, 4, 5, 6, 7]
    z, tol = c.turned(c.q, c.qw)
    assert c.rounded(got.float()[keep], z[keep], tol[keep])
    c = Case(8, 2, 1, 128, 128, "f16", "f16", eps=0.0)
    c.q[2, 1, 5] = math.nan
    got, st = c.call()
    assert st == 0 and bool(got[2, 1].isnan().all()) and int(got.isnan().sum()) == 128


def test_bad_positions_and_slots_are_reported():
    import awq_int4_moe_gb300 as awq
    t = torch()
    for bad in (-1, 500):
        c = Case(12, 4, 2, 64, 64, "f16", "f16")
        good = c.positions.clone()
        c.positions[3] = bad
        out = t.full_like(c.q, 9.0)
        _, st = c.call(q_out=out)
        assert st == awq.ERR_BAD_INDEX and bool((out[3] == 9.0).all())
        c.positions = good
        assert c.rounded(out.float()[[0, 11]], *(x[[0, 11]] for x in c.turned(c.q, c.qw)))
    c = Case(12, 4, 2, 64, 64, "f16", "f16")
    c.slots[3] = c.kc.shape[0] * c.page
    out = t.full_like(c.q, 9.0)
    _, st = c.call(q_out=out)
    assert st == awq.ERR_BAD_INDEX and bool((out[3] == 9.0).all())


def test_same_bits_as_the_append_where_the_norm_is_one():
    """Rows of mean square 1 - eps, weights of 1: awq_rope_append's outputs to within the norm's roundings."""
    t = torch()
    import awq_int4_moe_gb300 as awq
    c = Case(20, 4, 2, 64, 64, "f16", "f16", eps=0.0)
    for x in (c.q, c.k):
        x.copy_(t.where(x > 0, 1.0, -1.0))
    c.qw.fill_(1.0)
    c.kw.fill_(1.0)
    got, _ = c.call()
    k_got = c.kc.clone()
    out, st = t.empty_like(c.q), t.zeros(1, dtype=t.int32, device="cuda")
    awq.rope_append(c.q, c.k, c.v, c.positions, c.table, c.slots, c.kc, c.vc, st, q_out=out)
    t.cuda.synchronize()
    assert int(st) == 0
    # y is off by at most 2^-22 of 1: one step of fp16 where a sum lies next to a border
    assert bool(((got.float() - out.float()).abs() <= 2.0 ** -10 * 1.5).all())
    assert bool(((k_got.float() - c.kc.float()).abs() <= 2.0 ** -10 * 1.5).all())


def test_graph_replay():
    import awq_int4_moe_gb300 as awq
    t = torch()
    c = Case(30, 8, 2, 128, 128, "f16", "f16")
    want, _ = c.call()
    out, st = t.empty_like(c.q), t.zeros(1, dtype=t.int32, device="cuda")
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        awq.qk_norm_rope_append(c.q, c.k, c.v, c.qw, c.kw, c.eps, c.positions, c.table, c.slots, c.kc, c.vc, st, q_out=out)
    out.zero_()
    g.replay()
    t.cuda.synchronize()
    assert int(st) == 0 and bool((out == want).all())
