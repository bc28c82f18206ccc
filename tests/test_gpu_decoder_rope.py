"""awq_rope_append against 64-bit results.

Tolerances: an output is one rounding (u of its type, as in the norm's tests)
of a cos - b sin, whose fp32 evaluation is off by at most 2^-22 (|a| + |b|);
an e4m3 element by half its spacing, 2^-4 relative or 2^-10, in units of the
scale; copies are exact."""
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


def table(positions, rotary):
    t = torch()
    f = 10000.0 ** (-t.arange(0, rotary, 2, device="cuda", dtype=t.float64) / max(rotary, 1))
    a = t.arange(positions, device="cuda", dtype=t.float64)[:, None] * f
    return t.cat([a.cos(), a.sin()], 1).float()


def turned(x, row, inter):
    """64-bit rotation and the bound's |a| + |b|."""
    t = torch()
    half = row.shape[1] // 2
    c, s = row[:, None, :half].double(), row[:, None, half:].double()
    i = t.arange(half, device="cuda")
    lo, hi = (2 * i, 2 * i + 1) if inter else (i, i + half)
    a, b = x[..., lo], x[..., hi]
    y, size = x.clone(), t.zeros_like(x)
    y[..., lo], y[..., hi] = a * c - b * s, b * c + a * s
    size[..., lo] = size[..., hi] = a.abs() + b.abs()
    return y, size


def make_cache(pages, page, heads, dim, kind, heads_first):
    t = torch()
    shape = (pages, heads, page, dim) if heads_first else (pages, page, heads, dim)
    c = t.full(shape, 3.0, device="cuda").to(dtype_of(kind))
    return c.transpose(1, 2) if heads_first else c


def close(got, want, size, kind, scale=1.0):
    u = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "e4m3": 2.0 ** -4}[kind]
    low = scale * 2.0 ** -10 if kind == "e4m3" else 2.0 ** -25
    err = (got.double() * scale - want).abs()
    tol = want.abs() * u + (1 + u) * 2.0 ** -22 * size + low + want.abs() * 2.0 ** -22
    assert bool((err <= tol).all()), float((err - tol).max())


def run(tokens, hq, hk, dim, rotary, inter, kind, cache, page, heads_first, fused=True, in_place=False, seed=0):
    import awq_int4_moe_gb300 as awq
    t = torch()
    g = t.Generator(device="cuda")
    g.manual_seed(seed)
    dt = dtype_of(kind)
    if fused:                                   # cut from one product's output
        qkv = t.randn((tokens, hq + 2 * hk, dim), generator=g, device="cuda").to(dt)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    else:                                       # heads before tokens
        q, k, v = (t.randn((h, tokens, dim), generator=g, device="cuda").to(dt).transpose(0, 1) for h in (hq, hk, hk))
    pages = -(-tokens // page) + 2
    kc, vc = (make_cache(pages, page, hk, dim, cache, heads_first) for _ in range(2))
    cs = table(500, rotary)
    pos = t.randint(0, 500, (tokens,), generator=g, device="cuda").int()
    slots = t.randperm(pages * page, generator=g, device="cuda")[:tokens]
    slots[::4] = -1                              # unused tokens
    scales = (0.03, 0.05) if cache == "e4m3" else (1.0, 1.0)
    st = t.zeros(1, dtype=t.int32, device="cuda")
    q0, k0, v0 = q.double(), k.double(), v.double()
    q_out = None if in_place else t.full((tokens, hq, dim), 9.0, device="cuda", dtype=dt)
    awq.rope_append(q, k, v, pos, cs, slots, kc, vc, st, q_out=q_out, interleaved=inter, k_scale=scales[0],
                    v_scale=scales[1])
    t.cuda.synchronize()
    assert int(st) == 0
    row = cs[pos.long()]
    qr, qs = turned(q0, row, inter)
    kr, ks = turned(k0, row, inter)
    close(q if in_place else q_out, qr, qs, kind)
    used = slots >= 0
    place = slots[used]
    flat = (lambda c: c.float().reshape(pages * page, hk, dim))
    close(flat(kc)[place], kr[used], ks[used], cache, scales[0])
    close(flat(vc)[place], v0[used], t.zeros_like(v0[used]), cache, scales[1])
    rest = t.ones(pages * page, dtype=t.bool, device="cuda")
    rest[place] = False
    assert bool((flat(kc)[rest] == 3.0).all()) and bool((flat(vc)[rest] == 3.0).all())


@pytest.mark.parametrize("kind,cache", [("f16", "f16"), ("bf16", "bf16"), ("f16", "e4m3"), ("bf16", "e4m3")])
@pytest.mark.parametrize("hq,hk,dim,rotary,inter", [
    (20, 4, 128, 128, False), (8, 8, 128, 64, True), (5, 1, 80, 40, False), (4, 2, 96, 48, True), (3, 3, 64, 64, True),
    (2, 1, 256, 256, False), (7, 1, 72, 24, False), (2, 2, 20, 20, True), (3, 1, 13, 6, False), (3, 1, 13, 6, True),
    (2, 1, 100, 0, False), (40, 8, 576, 64, False)])
def test_rope_append(hq, hk, dim, rotary, inter, kind, cache):
    run(9, hq, hk, dim, rotary, inter, kind, cache, 4, False)


@pytest.mark.parametrize("tokens,page,heads_first,fused", [(1, 1, False, True), (2, 16, True, True), (33, 7, True, False),
                                                           (300, 64, False, False)])
def test_rope_append_layouts(tokens, page, heads_first, fused):
    run(tokens, 6, 2, 128, 128, False, "f16", "f16", page, heads_first, fused, seed=tokens)
    run(tokens, 6, 2, 128, 128, True, "bf16", "e4m3", page, heads_first, fused, in_place=True, seed=tokens)


def test_indexes_outside_write_nothing():
    import awq_int4_moe_gb300 as awq
    t = torch()
    for bad_pos, bad_slot in ((-1, 0), (50, 0), (0, 8), (0, 1 << 40)):
        q = t.randn((3, 2, 64), device="cuda").half()
        k, v = t.randn((3, 1, 64), device="cuda").half(), t.randn((3, 1, 64), device="cuda").half()
        kc, vc = make_cache(2, 4, 1, 64, "f16", False), make_cache(2, 4, 1, 64, "f16", False)
        pos = t.tensor([1, bad_pos, 3], dtype=t.int32, device="cuda")
        slots = t.tensor([2, bad_slot, 6], device="cuda")
        st = t.zeros(1, dtype=t.int32, device="cuda")
        out = t.full_like(q, 9.0)
        awq.rope_append(q, k, v, pos, table(50, 64), slots, kc, vc, st, q_out=out)
        t.cuda.synchronize()
        assert int(st) == awq.ERR_BAD_INDEX
        assert bool((out[1] == 9.0).all()) and bool((out[0] != 9.0).any())
        flat = vc.reshape(8, 64)
        assert bool((flat[2] == v[0, 0]).all()) and bool((flat[6] == v[2, 0]).all())
        assert all(bool((flat[i] == 3.0).all()) for i in (0, 1, 3, 4, 5, 7))


def test_cache_past_32_bit_offsets():
    import awq_int4_moe_gb300 as awq
    t = torch()
    pages = 140000                               # x 16 tokens x 8 heads x 128: 2.3 G elements
    kc = t.zeros((pages, 16, 8, 128), device="cuda", dtype=t.float16)
    vc = t.zeros_like(kc)
    qkv = t.randn((2, 12, 128), device="cuda").half()
    q, k, v = qkv[:, :4], qkv[:, 4:12], qkv[:, 4:12]
    slots = t.tensor([pages * 16 - 1, 5], device="cuda")
    pos = t.tensor([7, 8], dtype=t.int32, device="cuda")
    st = t.zeros(1, dtype=t.int32, device="cuda")
    awq.rope_append(q, k, v, pos, table(10, 128), slots, kc, vc, st, q_out=t.empty((2, 4, 128), device="cuda").half())
    t.cuda.synchronize()
    assert int(st) == 0
    assert bool((vc[-1, 15] == v[0]).all()) and bool((vc[0, 5] == v[1]).all())


def test_saturation_and_nan_into_e4m3():
    import awq_int4_moe_gb300 as awq
    t = torch()
    v = t.zeros((1, 1, 64), device="cuda").half()
    v[0, 0, :4] = t.tensor([1000.0, -1000.0, float("nan"), float("inf")])
    kc, vc = make_cache(1, 1, 1, 64, "e4m3", False), make_cache(1, 1, 1, 64, "e4m3", False)
    z = t.zeros((1, 1, 64), device="cuda").half()
    st = t.zeros(1, dtype=t.int32, device="cuda")
    awq.rope_append(z, z.clone(), v, t.zeros(1, dtype=t.int32, device="cuda"), table(1, 64),
                    t.zeros(1, dtype=t.int64, device="cuda"), kc, vc, st, q_out=z.clone())
    got = vc.float().flatten()
    assert float(got[0]) == 448.0 and float(got[1]) == -448.0 and bool(got[2].isnan()) and float(got[3]) == 448.0


@pytest.mark.parametrize("kind,cache", [("f16", "f16"), ("bf16", "e4m3")])
def test_strides_of_dimensions_of_one_are_not_used(kind, cache):
    """One token, KV head and page of one token: the same bits whatever the
    strides behind them."""
    import awq_int4_moe_gb300 as awq
    t = torch()
    g = t.Generator(device="cuda")
    g.manual_seed(5)
    q, k, v = (t.randn((1, 1, 64), generator=g, device="cuda").to(dtype_of(kind)) for _ in range(3))
    pos, slots = t.tensor([3], dtype=t.int32, device="cuda"), t.zeros(1, dtype=t.int64, device="cuda")
    found = []
    for strides in ((64, 64, 64), (67, 71, 73)):
        heads = lambda x: x.as_strided((1, 1, 64), (strides[0], strides[1], 1))  # noqa: E731
        plane = lambda x: x.as_strided((1, 1, 1, 64), (*strides, 1))  # noqa: E731
        kc, vc = make_cache(1, 1, 1, 64, cache, False), make_cache(1, 1, 1, 64, cache, False)
        out, st = t.full_like(q, 9.0), t.zeros(1, dtype=t.int32, device="cuda")
        awq.rope_append(heads(q), heads(k), heads(v), pos, table(10, 64), slots, plane(kc), plane(vc), st, q_out=heads(out),
                        k_scale=0.5 if cache == "e4m3" else 1.0, v_scale=0.5 if cache == "e4m3" else 1.0)
        t.cuda.synchronize()
        assert int(st) == 0 and bool((out != 9.0).any())
        found.append((out, kc.float(), vc.float()))
    assert all(t.equal(a, b) for a, b in zip(*found))


@pytest.mark.parametrize("kind,cache", [("f16", "f16"), ("bf16", "bf16"), ("f16", "e4m3"), ("bf16", "e4m3")])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("tokens,hq,hk,dim,rotary", [
    (1300, 20, 4, 128, 128), (2500, 32, 8, 128, 128), (1300, 7, 1, 100, 40), (1217, 5, 2, 13, 6), (1300, 3, 1, 80, 0),
    (1300, 2, 1, 576, 64), (1216, 1, 1, 1024, 1024)])
def test_rope_append_of_prompts(tokens, hq, hk, dim, rotary, inter, kind, cache):
    """From 8 tokens per multiprocessor on a token has two warps, which go over
    its rows in several turns."""
    run(tokens, hq, hk, dim, rotary, inter, kind, cache, 16, False, seed=tokens + dim)


@pytest.mark.parametrize("inter", [False, True])
def test_rope_append_of_more_rows_than_a_block_holds(inter):
    run(9, 64, 8, 128, 128, inter, "f16", "f16", 4, False)      # 80 rows, 32 at once
    run(9, 90, 5, 128, 64, inter, "bf16", "e4m3", 4, True, in_place=True)
    run(1300, 24, 4, 128, 64, inter, "bf16", "bf16", 4, True, in_place=True)


@pytest.mark.parametrize("page", [5, 16])
@pytest.mark.parametrize("kind,cache", [("f16", "f16"), ("bf16", "e4m3")])
def test_rope_append_with_planes_of_different_layouts(page, kind, cache, monkeypatch):
    turns = iter([True, False])
    real = make_cache
    monkeypatch.setitem(globals(), "make_cache", lambda pages, page, heads, dim, kind, first: real(pages, page, heads, dim, kind, next(turns)))
    run(33, 6, 2, 128, 128, False, kind, cache, page, None)
