"""awq_fp8_gemm against 64-bit results.

Tolerances. Products of e4m3 values are exact in fp32. A block of 128 is added
in four steps of 32 products with fp32 results: below 2^-17 of the sum of the
products' magnitudes. Blocks are scaled and added in fp32, 2^-24 each. With S
the sum of all scaled magnitudes: (2^-17 + (blocks + 4) 2^-23) S, and one
rounding of the output."""
import pytest

import gpu_common as gc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    gc.require_gpu()
    gc.build_all()


def torch():
    return gc.torch_mod()


def operands(m, n, k, seed=0, lda=None, ldb=None):
    """e4m3 values and scales; the last block's rows and columns are partly there."""
    t = torch()
    g = t.Generator(device="cuda")
    g.manual_seed(seed)
    kb, nb = -(-k // 128), -(-n // 128)
    fill = 448.0                                 # past K: must not be read into the sum
    a = t.full((m, lda or -(-k // 16) * 16), fill, device="cuda").to(t.float8_e4m3fn)
    b = t.full((n, ldb or -(-k // 16) * 16), fill, device="cuda").to(t.float8_e4m3fn)
    a[:, :k] = (t.randn((m, k), generator=g, device="cuda") * 60).clamp(-448, 448).to(t.float8_e4m3fn)
    b[:, :k] = (t.randn((n, k), generator=g, device="cuda") * 60).clamp(-448, 448).to(t.float8_e4m3fn)
    sa = t.exp(t.randn((m, kb), generator=g, device="cuda")) * 0.01
    sb = t.exp(t.randn((nb, kb), generator=g, device="cuda")) * 0.001
    return a[:, :k], sa, b[:, :k], sb


def check(a, sa, b, sb, out):
    t = torch()
    k, n = a.shape[1], b.shape[0]
    ad = a.float().double() * sa.double().repeat_interleave(128, 1)[:, :k]
    bd = b.float().double() * sb.double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    want, size = ad @ bd.t(), ad.abs() @ bd.abs().t()
    u = 2.0 ** -11 if out.dtype == t.float16 else 2.0 ** -8
    tol = want.abs() * u + (2.0 ** -17 + (sa.shape[1] + 4) * 2.0 ** -23) * size + 2.0 ** -25
    err = (out.double() - want).abs()
    bad = err > tol
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()}, worst {float((err / tol).max())}, first {bad.nonzero()[0].tolist()}"


def run(m, n, k, kind="f16", pad=0, seed=0):
    import awq_int4_moe_gb300 as awq
    t = torch()
    a, sa, b, sb = operands(m, n, k, seed)
    dt = {"f16": t.float16, "bf16": t.bfloat16}[kind]
    wide = t.full((m, n + pad), 9.0, device="cuda", dtype=dt)
    st = t.zeros(1, dtype=t.int32, device="cuda")
    awq.fp8_gemm(a, sa, b, sb, wide[:, :n], st)
    t.cuda.synchronize()
    assert int(st) == 0
    check(a, sa, b, sb, wide[:, :n])
    assert bool((wide[:, n:] == 9.0).all())


@pytest.mark.parametrize("m", [1, 2, 15, 16, 17, 32, 33, 63, 64, 65, 96, 127, 128, 129, 200, 256, 300])
def test_token_counts(m):
    run(m, 640, 2560, "f16", seed=m)
    run(m, 131, 384, "bf16", pad=3, seed=m)


@pytest.mark.parametrize("n", [1, 7, 8, 64, 127, 128, 129, 255, 256, 257, 2560, 3584])
def test_output_sizes(n):
    run(5, n, 512, "f16", seed=n)
    run(150, n, 512, "bf16", pad=8, seed=n)


@pytest.mark.parametrize("k", [1, 15, 16, 31, 32, 100, 127, 128, 129, 144, 256, 1000, 1024, 4240, 16384])
def test_depths(k):
    run(3, 256, k, "f16", seed=k)
    run(40, 200, k, "bf16", seed=k)
    run(190, 300, k, "f16", seed=k)


@pytest.mark.parametrize("m,n,k", [(1, 16384, 2560), (16, 5120, 8192), (1024, 2560, 2560), (2100, 5001, 1040), (4096, 4096, 512),
                                   (8191, 2560, 256)])
def test_large(m, n, k):
    run(m, n, k, "bf16", seed=m)


def test_strided_operands_and_misaligned_output():
    import awq_int4_moe_gb300 as awq
    t = torch()
    for m in (4, 50, 140):
        a, sa, b, sb = operands(m, 300, 640, lda=1024, ldb=688)
        flat = t.full((m * 303 + 5,), 9.0, device="cuda", dtype=t.float16)
        out = flat[3:3 + m * 303].view(m, 303)[:, :300]
        st = t.zeros(1, dtype=t.int32, device="cuda")
        awq.fp8_gemm(a, sa, b, sb, out, st)
        t.cuda.synchronize()
        assert int(st) == 0
        check(a, sa, b, sb, out)
        assert bool((flat[:3] == 9.0).all()) and bool((flat[-2:] == 9.0).all())


@pytest.mark.parametrize("m,n,k", [(1, 40, 1001), (1, 1, 77), (64, 1, 48), (200, 1, 1000)])
def test_single_rows_of_any_depth(m, n, k):
    import awq_int4_moe_gb300 as awq
    t = torch()
    a, sa, b, sb = operands(m, n, k)
    a, b = (x.contiguous() if x.shape[0] == 1 else x for x in (a, b))
    out, st = t.empty((m, n), device="cuda", dtype=t.float16), t.zeros(1, dtype=t.int32, device="cuda")
    awq.fp8_gemm(a, sa, b, sb, out, st)
    t.cuda.synchronize()
    assert int(st) == 0
    check(a, sa, b, sb, out)


def test_scales_of_zero_and_extremes():
    import awq_int4_moe_gb300 as awq
    t = torch()
    for m in (3, 150):
        a, sa, b, sb = operands(m, 256, 512)
        sa[0] = 0
        sb[1] = 0
        sa[1] *= 1e-20
        sb[0] *= 1e20
        out, st = t.empty((m, 256), device="cuda", dtype=t.bfloat16), t.zeros(1, dtype=t.int32, device="cuda")
        awq.fp8_gemm(a, sa, b, sb, out, st)
        t.cuda.synchronize()
        assert bool((out[0] == 0).all()) and bool((out[:, 128:] == 0).all())
        check(a, sa, b, sb, out)


def test_nan_stays_in_its_row_or_column():
    import awq_int4_moe_gb300 as awq
    t = torch()
    for m in (3, 40, 150):
        a, sa, b, sb = operands(m, 256, 512)
        a.view(t.uint8)[1, 5] = 0x7F
        b.view(t.uint8)[200, 6] = 0xFF
        out, st = t.empty((m, 256), device="cuda", dtype=t.float16), t.zeros(1, dtype=t.int32, device="cuda")
        awq.fp8_gemm(a, sa, b, sb, out, st)
        t.cuda.synchronize()
        nan = out.isnan()
        assert bool(nan[1].all()) and bool(nan[:, 200].all()) and int(nan.sum()) == 256 + m - 1


def test_same_bits_every_time():
    import awq_int4_moe_gb300 as awq
    t = torch()
    for m in (1, 60, 100, 700):
        a, sa, b, sb = operands(m, 640, 2560)
        st = t.zeros(1, dtype=t.int32, device="cuda")
        outs = []
        for _ in range(3):
            out = t.empty((m, 640), device="cuda", dtype=t.float16)
            awq.fp8_gemm(a, sa, b, sb, out, st)
            outs.append(out)
        t.cuda.synchronize()
        assert all(bool((o == outs[0]).all()) for o in outs[1:])


def test_weight_past_32_bit_offsets():
    import awq_int4_moe_gb300 as awq
    t = torch()
    n, k = 270000, 8192                          # 2.2 GB of weight
    b = t.zeros((n, k), device="cuda", dtype=t.uint8).view(t.float8_e4m3fn)
    a, sa, tail, sb1 = operands(2, 128, k)
    b[n - 48:] = tail[:48]
    sb = t.ones((-(-n // 128), k // 128), device="cuda") * 0.001
    out, st = t.empty((2, n), device="cuda", dtype=t.float16), t.zeros(1, dtype=t.int32, device="cuda")
    awq.fp8_gemm(a, sa, b, sb, out, st)
    t.cuda.synchronize()
    assert int(st) == 0
    check(a, sa, tail[:48].contiguous(), sb[:1], out[:, n - 48:])
    assert bool((out[:, : n - 48] == 0).all())


@pytest.mark.parametrize("m,n,k", [
    (1, 40960, 640), (20, 39100, 640), (30, 50000, 144), (50, 40001, 640), (64, 39000, 272),      # weights on the M side
    (200, 5120, 700), (1100, 1280, 700), (129, 9800, 400), (1025, 1400, 2560)])                 # tiles of 128 x 128
def test_tiles_of_one_block_and_several_k_blocks(m, n, k):
    """More tiles than clusters that run at once: a block per tile, which goes
    on to further tiles where there are more than blocks."""
    run(m, n, k, "bf16", pad=3, seed=m)
    run(m, n, k, "f16", seed=m + 1)
