"""awq_add_rmsnorm and awq_quantize_fp8 against 64-bit results.

Tolerances. u is half a unit in the last place of the output type, relative to
a normal value: 2^-11 (fp16), 2^-8 (bf16), 2^-4 (e4m3); the spacing below the
smallest normal adds 2^-25 (fp16) or 2^-10 of a group's scale (e4m3). The
fp32 part: a sum of squares added in a tree and at most 32 terms a thread,
a square root, a division and two products, below 2^-18 relative."""
import pytest

import gpu_common as gc

pytestmark = pytest.mark.gpu
F32 = 2.0 ** -18


@pytest.fixture(scope="module", autouse=True)
def _built():
    gc.require_gpu()
    gc.build_all()


def torch():
    return gc.torch_mod()


def dtype_of(name):
    return {"f16": torch().float16, "bf16": torch().bfloat16}[name]


def unit(name):
    return 2.0 ** -11 if name == "f16" else 2.0 ** -8


def data(seed, *shape):
    g = torch().Generator(device="cuda")
    g.manual_seed(seed)
    return torch().randn(shape, generator=g, device="cuda")


def check_groups(y, q, scales):
    """q, scales against 64-bit rows y."""
    t = torch()
    n, h = y.shape
    for j, c in enumerate(range(0, h, 128)):
        part = y[:, c:c + 128]
        want = part.abs().amax(1).clamp(min=1e-12) / 448
        got = scales[:, j].double()
        assert bool(((got - want).abs() <= F32 * want).all())
        back = q[:, c:c + 128].double() * got[:, None]
        tol = part.abs() * (2.0 ** -4 + 2 * F32) + got[:, None] * 2.0 ** -10
        assert bool(((back - part).abs() <= tol).all()), f"group {j}"
        assert bool(t.isfinite(back).all())


def reference(x, residual, w, eps):
    r = x.double() + (residual.double() if residual is not None else 0.0)
    return r, r / (r.square().mean(1, keepdim=True) + eps).sqrt() * w.double()


def run_norm(rows, hidden, kind, residual, outputs, pad, seed=0, scale=1.0):
    import awq_int4_moe_gb300 as awq
    t = torch()
    dt = dtype_of(kind)
    wide = t.zeros((rows, hidden + pad), device="cuda", dtype=dt)
    x = wide[:, :hidden]
    x.copy_(data(seed, rows, hidden) * scale)
    w = (1 + 0.3 * data(seed + 1, hidden)).to(dt)
    res = (data(seed + 2, rows, hidden) * scale).to(dt) if residual else None
    res_out = t.empty_like(res) if residual else None
    out = t.full((rows, hidden + pad), 7.0, device="cuda", dtype=dt)
    q = t.zeros((rows, hidden + pad), device="cuda", dtype=t.uint8).view(t.float8_e4m3fn)
    sc = t.full((rows, (hidden + 127) // 128), -1.0, device="cuda")
    awq.add_rmsnorm(x, w, 1e-6, residual=res, residual_out=res_out, out=out[:, :hidden] if "y" in outputs else None,
                    out_q=q[:, :hidden] if "q" in outputs else None, out_scales=sc if "q" in outputs else None)
    t.cuda.synchronize()
    r, y = reference(x, res, w, 1e-6)
    u = unit(kind)
    if residual:
        assert bool(((res_out.double() - r).abs() <= r.abs() * u + 2.0 ** -25).all())
    if "y" in outputs:
        assert bool(((out[:, :hidden].double() - y).abs() <= y.abs() * (u + F32) + 2.0 ** -25).all())
        assert bool((out[:, hidden:] == 7.0).all())          # nothing past the row
    if "q" in outputs:
        check_groups(y, q[:, :hidden], sc)
        assert int(q.view(t.uint8)[:, hidden:].sum()) == 0


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("rows,hidden,pad", [
    (1, 2560, 0), (1, 1, 0), (3, 2, 1), (5, 127, 0), (5, 128, 0), (5, 129, 3), (2, 1000, 0), (7, 1024, 8), (3, 1032, 0),
    (4, 4095, 0), (4, 4104, 8), (2, 8192, 0), (2, 8200, 0), (2, 16384, 0), (1, 16385, 0), (2, 32768, 0), (1, 32767, 2),
    (1, 24000, 0), (130, 640, 5), (1000, 128, 0), (2500, 1280, 0), (1400, 5120, 8), (700, 16384, 0), (5000, 96, 3),
    (900, 1500, 1)])
def test_norm_sizes(rows, hidden, pad, kind):
    run_norm(rows, hidden, kind, True, "yq", pad)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("outputs", ["y", "q", "yq"])
def test_norm_outputs(residual, outputs):
    run_norm(9, 2560, "f16", residual, outputs, 0, seed=5)
    run_norm(9, 333, "bf16", residual, outputs, 0, seed=6)


@pytest.mark.parametrize("scale", [1e-6, 100.0])
def test_norm_ranges(scale):
    run_norm(4, 2560, "f16", True, "yq", 0, seed=9, scale=scale)
    run_norm(4, 2560, "bf16", True, "yq", 0, seed=10, scale=scale * scale)


def test_norm_in_place():
    import awq_int4_moe_gb300 as awq
    t = torch()
    x, res, w = (data(i, 6, 1280).half() for i in range(3))
    w = w[0].contiguous()
    r, y = reference(x, res, w, 1e-5)
    awq.add_rmsnorm(x, w, 1e-5, residual=res, residual_out=res, out=x)
    t.cuda.synchronize()
    assert bool(((res.double() - r).abs() <= r.abs() * 2.0 ** -11 + 2.0 ** -25).all())
    assert bool(((x.double() - y).abs() <= y.abs() * (2.0 ** -11 + F32) + 2.0 ** -25).all())


@pytest.mark.parametrize("hidden", [2560, 333])
def test_norm_zero_rows_and_non_finite_values(hidden):
    import awq_int4_moe_gb300 as awq
    t = torch()
    x = data(3, 4, hidden).half()
    x[0] = 0
    x[1, 5] = float("nan")
    x[2, 5] = float("inf")
    w = t.ones(hidden, device="cuda", dtype=t.float16)
    out, q = t.empty_like(x), t.empty((4, hidden), device="cuda", dtype=t.float8_e4m3fn)
    sc = t.empty((4, (hidden + 127) // 128), device="cuda")
    awq.add_rmsnorm(x, w, 1e-6, out=out, out_q=q, out_scales=sc)
    t.cuda.synchronize()
    assert bool((out[0] == 0).all()) and bool((q[0].float() == 0).all())
    assert bool(((sc[0] - 1e-12 / 448).abs() <= 1e-20).all())
    assert bool(out[1].isnan().all()) and bool(q[1].float().isnan().all())
    # an infinite element makes the row's mean infinite: 0 elsewhere, NaN there
    assert bool(out[2, 5].isnan()) and int(out[2].isnan().sum()) == 1 and bool((out[2][~out[2].isnan()] == 0).all())
    run = reference(x[3:], None, w, 1e-6)[1]
    assert bool(((out[3:].double() - run).abs() <= run.abs() * (2.0 ** -11 + F32) + 2.0 ** -25).all())


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("rows,cols,pad", [(1, 1, 0), (1, 128, 0), (3, 130, 0), (2, 255, 1), (48, 4096, 0), (5, 257, 7),
                                           (700, 384, 128), (2, 70000, 0), (3, 8192, 8)])
def test_quantize(rows, cols, pad, kind):
    import awq_int4_moe_gb300 as awq
    t = torch()
    wide = t.full((rows, cols + pad), 9.0, device="cuda").to(dtype_of(kind))
    x = wide[:, :cols]
    x.copy_(data(cols, rows, cols) * t.exp(2 * data(cols + 1, cols)))
    x[0, : cols // 2] = 0
    q = t.zeros((rows, cols + pad), device="cuda", dtype=t.uint8).view(t.float8_e4m3fn)
    sc = t.empty((rows, (cols + 127) // 128), device="cuda")
    awq.quantize_fp8(x, q[:, :cols], sc)
    t.cuda.synchronize()
    check_groups(x.double(), q[:, :cols], sc)
    assert int(q.view(t.uint8)[:, cols:].sum()) == 0
    # the largest magnitude of a group is the largest code
    top = q[:, :cols].float().abs()
    assert float(top[-1, :128].max()) == 448.0


@pytest.mark.parametrize("rows,cols,pad", [(17000, 1024, 0), (8001, 2560, 8), (3001, 2563, 2), (40, 200001, 0), (500, 40960, 0)])
def test_quantize_of_many_rows(rows, cols, pad):
    import awq_int4_moe_gb300 as awq
    t = torch()
    wide = t.full((rows, cols + pad), 9.0, device="cuda").bfloat16()
    x = wide[:, :cols]
    x.copy_(data(cols, rows, cols))
    q = t.zeros((rows, cols + pad), device="cuda", dtype=t.uint8).view(t.float8_e4m3fn)
    sc = t.full((rows, (cols + 127) // 128), -1.0, device="cuda")
    awq.quantize_fp8(x, q[:, :cols], sc)
    t.cuda.synchronize()
    check_groups(x.double(), q[:, :cols], sc)
    assert int(q.view(t.uint8)[:, cols:].sum()) == 0


@pytest.mark.parametrize("cols", [256, 250])
def test_quantize_non_finite(cols):
    import awq_int4_moe_gb300 as awq
    t = torch()
    x = data(1, 2, cols).bfloat16()
    x[0, 3], x[1, 4] = float("nan"), float("-inf")
    q, sc = t.empty((2, cols), device="cuda", dtype=t.float8_e4m3fn), t.empty((2, 2), device="cuda")
    awq.quantize_fp8(x, q, sc)
    t.cuda.synchronize()
    assert bool(q[0, 3].float().isnan()) and int(q[0].float().isnan().sum()) == 1      # its group's others as ever
    assert float(sc[1, 0]) == float("inf") and bool(q[1, 4].float().isnan())
    check_groups(x[1:, 128:].double(), q[1:, 128:], sc[1:, 1:])


def test_rows_past_32_bit_offsets():
    import awq_int4_moe_gb300 as awq
    t = torch()
    rows, cols = 70000, 32768                    # 2.3 G elements
    x = t.zeros((rows, cols), device="cuda", dtype=t.float16)
    x[-1] = data(8, cols).half()
    w = t.ones(cols, device="cuda", dtype=t.float16)
    q, sc = t.empty((rows, cols), device="cuda", dtype=t.float8_e4m3fn), t.empty((rows, cols // 128), device="cuda")
    awq.quantize_fp8(x, q, sc)
    check_groups(x[-1:].double(), q[-1:], sc[-1:])
    awq.add_rmsnorm(x, w, 1e-6, out_q=q, out_scales=sc)
    check_groups(reference(x[-1:], None, w, 1e-6)[1], q[-1:], sc[-1:])


def test_same_bits_on_a_side_stream():
    import awq_int4_moe_gb300 as awq
    t = torch()
    x, w = data(1, 40, 2560).half(), data(2, 2560).half()
    a, b = t.empty_like(x), t.empty_like(x)
    awq.add_rmsnorm(x, w, 1e-6, out=a)
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    awq.add_rmsnorm(x, w, 1e-6, out=b, stream=side)
    t.cuda.synchronize()
    assert bool((a == b).all())


@pytest.mark.parametrize("rows", [2 ** 31 - 1, 2 ** 31 - 3])
def test_norm_of_as_many_rows_as_there_can_be(rows):
    """One column: every y is the weight, with the sign of x (x^2 + eps is x^2 in
    fp32 for the magnitudes taken)."""
    import awq_int4_moe_gb300 as awq
    t = torch()
    x = t.full((rows, 1), 4.0, device="cuda", dtype=t.float16)
    x[-2:] = t.tensor([[-8.0], [16.0]])
    out = t.zeros((rows, 1), device="cuda", dtype=t.float16)
    awq.add_rmsnorm(x, t.full((1,), 3.0, device="cuda", dtype=t.float16), 1e-9, out=out)
    t.cuda.synchronize()
    assert out[-2:].flatten().tolist() == [-3.0, 3.0]
    assert all(bool((part == 3.0).all()) for part in out[:-2].split(1 << 28))


def test_stride_of_a_single_row_is_not_used():
    """The same accesses, so the same bits, whatever the stride behind the only row."""
    import awq_int4_moe_gb300 as awq
    t = torch()
    for seed in range(8):
        x, res = (data(seed + 10 * i, 1, 2560).half() for i in range(2))
        w = (1 + 0.3 * data(seed + 20, 2560)).half()
        odd = lambda r: r.as_strided((1, r.shape[1]), (r.shape[1] + 5, 1))  # noqa: E731
        sums = []
        for view in (lambda r: r, odd):
            ro, out = t.empty_like(x), t.empty_like(x)
            q, sc = t.empty((1, 2560), device="cuda", dtype=t.float8_e4m3fn), t.empty((1, 20), device="cuda")
            awq.add_rmsnorm(view(x), w, 1e-6, residual=view(res), residual_out=view(ro), out=view(out), out_q=view(q), out_scales=sc)
            q2, sc2 = t.empty_like(q), t.empty_like(sc)
            awq.quantize_fp8(view(x), view(q2), sc2)
            sums.append((ro, out, q.view(t.uint8), sc, q2.view(t.uint8), sc2))
        t.cuda.synchronize()
        assert all(t.equal(a, b) for a, b in zip(*sums))


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("rows,hidden,pad", [
    # unaligned rows of 4097 to 16384 columns: four chunks a thread
    (3, 4097, 0), (700, 6001, 0), (2, 8191, 3), (3, 8192, 5), (2, 8193, 0), (400, 12000, 1), (2, 16383, 0),
    # aligned rows of 257 to 512 columns: two chunks a lane
    (5, 264, 0), (900, 384, 8), (3, 512, 0),
    # more rows than the grid's warps: a row per warp that goes on to a second and a third
    (9733, 128, 0), (25000, 256, 0), (10001, 384, 0), (12000, 1000, 0), (11000, 100, 3), (10007, 300, 1)])
def test_norm_of_the_other_forms(rows, hidden, pad, kind):
    run_norm(rows, hidden, kind, True, "yq", pad, seed=rows)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("rows,cols,pad", [(10000, 256, 0), (4000, 2560, 0), (16384, 400, 8), (3000, 515, 2), (9728, 1, 1), (5001, 130, 0),
                                           (30001, 384, 0)])
def test_quantize_with_two_steps_a_warp(rows, cols, pad, kind):
    """From 64 steps per multiprocessor on, below 400 of them or where rows are
    short."""
    import awq_int4_moe_gb300 as awq
    t = torch()
    wide = t.full((rows, cols + pad), 9.0, device="cuda").to(dtype_of(kind))
    x = wide[:, :cols]
    x.copy_(data(cols, rows, cols))
    q = t.zeros((rows, cols + pad), device="cuda", dtype=t.uint8).view(t.float8_e4m3fn)
    sc = t.full((rows, (cols + 127) // 128), -1.0, device="cuda")
    awq.quantize_fp8(x, q[:, :cols], sc)
    t.cuda.synchronize()
    check_groups(x.double(), q[:, :cols], sc)
    assert int(q.view(t.uint8)[:, cols:].sum()) == 0
