"""The decoder operators' C ABI and binding without a GPU: every declared
symbol is exported, and what the host can see to be wrong is refused before any
CUDA call."""
import ctypes as C
import os
import re

import pytest

import awq_int4_moe_gb300 as awq
from awq_int4_moe_gb300 import decoder as d

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "awq_decoder.h")
P = 0x10000000          # a 256-byte aligned non-null address; never dereferenced on these paths
OK, INVALID, SHAPE, ALIGN = awq.OK, awq.ERR_INVALID_ARG, awq.ERR_UNSUPPORTED_SHAPE, awq.ERR_MISALIGNED


@pytest.fixture(scope="module", autouse=True)
def _built():
    import awq_int4_moe_gb300.build as b
    b.build()


def test_every_declared_symbol_is_exported():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"AWQ_API\s+[\w\s\*]*?\b(awq_\w+)\s*\(", text))
    assert names == {"awq_add_rmsnorm", "awq_quantize_fp8", "awq_rope_append", "awq_paged_attention",
                     "awq_paged_attention_workspace_bytes", "awq_fp8_gemm"}
    for n in names:
        assert hasattr(awq.lib(), n), n


def test_constants_match_the_header():
    text = open(HEADER).read()
    for name, value in (("AWQ_DTYPE_F16", d.DTYPE_F16), ("AWQ_DTYPE_BF16", d.DTYPE_BF16), ("AWQ_DTYPE_E4M3", d.DTYPE_E4M3)):
        assert re.search(rf"{name} = {value}\b", text)
    assert f"#define AWQ_FP8_BLOCK {d.FP8_BLOCK}" in text
    assert awq.status_string(awq.ERR_BAD_INDEX) != "unknown status"


def norm(**over):
    a = dict(x=P, ldx=2560, residual=P, ldr=2560, residual_out=P, ldro=2560, weight=P, eps=1e-6, out=P, ldo=2560, out_q=P,
             ldq=2560, out_scales=P, rows=4, hidden=2560, dtype=0)
    a.update(over)
    return awq.lib().awq_add_rmsnorm(*a.values(), None)


@pytest.mark.parametrize("over,code", [
    (dict(rows=0), OK), (dict(rows=0, x=None, weight=None), OK), (dict(rows=-1), INVALID), (dict(hidden=0), SHAPE),
    (dict(hidden=32769), SHAPE), (dict(dtype=2), INVALID), (dict(dtype=-1), INVALID), (dict(x=None), INVALID),
    (dict(weight=None), INVALID), (dict(out=None, out_q=None, out_scales=None), INVALID), (dict(out_q=None), INVALID),
    (dict(out_scales=None), INVALID), (dict(ldx=2559), INVALID), (dict(ldr=2559), INVALID), (dict(ldro=2559), INVALID),
    (dict(ldo=2559), INVALID), (dict(ldq=2559), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(x=P + 1), ALIGN), (dict(residual=P + 1), ALIGN), (dict(out=P + 1), ALIGN),
    (dict(weight=P + 1), ALIGN), (dict(residual_out=P + 1), ALIGN), (dict(out_scales=P + 2), ALIGN)])
def test_norm_refusals(over, code):
    assert norm(**over) == code


@pytest.mark.parametrize("over,code", [
    (dict(rows=0), OK), (dict(rows=0, x=None), OK), (dict(rows=-1), INVALID), (dict(cols=0), INVALID), (dict(dtype=2), INVALID),
    (dict(x=None), INVALID), (dict(q=None), INVALID), (dict(scales=None), INVALID), (dict(ldx=99), INVALID),
    (dict(ldq=99), INVALID), (dict(x=P + 1), ALIGN), (dict(scales=P + 1), ALIGN)])
def test_quantize_refusals(over, code):
    a = dict(x=P, ldx=100, q=P, ldq=100, scales=P, rows=3, cols=100, dtype=1)
    a.update(over)
    assert awq.lib().awq_quantize_fp8(*a.values(), None) == code


def plane(data=P, scale=1.0, page=2048, token=128, head=64):
    return d.KvPlane(data, page, token, head, scale)


def cache(k=None, v=None, dtype=0, pages=8, page=16, heads=2, dim=64):
    return d.KvCache(k or plane(), v or plane(), dtype, pages, page, heads, dim)


def heads(data=P, tok=512, head=64):
    return d.Heads(data, tok, head)


CACHE_REFUSALS = [
    (dict(cache=None), INVALID), (dict(cache=cache(dtype=1)), INVALID), (dict(cache=cache(dtype=3)), INVALID),
    (dict(cache=cache(pages=0)), INVALID), (dict(cache=cache(page=0)), INVALID), (dict(cache=cache(heads=0)), INVALID),
    (dict(cache=cache(dim=0)), SHAPE), (dict(cache=cache(k=plane(data=None))), INVALID),
    (dict(cache=cache(v=plane(data=None))), INVALID), (dict(cache=cache(k=plane(scale=0.5))), INVALID),
    (dict(cache=cache(dtype=2, v=plane(scale=0.0))), INVALID), (dict(cache=cache(dtype=2, v=plane(scale=-1.0))), INVALID),
    (dict(cache=cache(dtype=2, k=plane(scale=float("nan")))), INVALID),
    (dict(cache=cache(dtype=2, k=plane(scale=float("inf")))), INVALID),
    (dict(cache=cache(k=plane(page=-1))), INVALID), (dict(cache=cache(k=plane(data=P + 1))), ALIGN),
    (dict(dtype=2), INVALID)]


def rope(**over):
    a = dict(q=heads(), q_out=heads(), k=heads(), v=heads(), positions=P, cos_sin=P, top=100, rotary=64, inter=0, slots=P,
             cache=cache(), tokens=4, q_heads=4, dtype=0, status=P)
    a.update(over)
    return awq.lib().awq_rope_append(*a.values(), None)


@pytest.mark.parametrize("over,code", CACHE_REFUSALS + [
    (dict(tokens=0), OK), (dict(tokens=0, q=None, positions=None), OK), (dict(tokens=-1), INVALID), (dict(q_heads=0), INVALID),
    (dict(top=0), INVALID), (dict(rotary=63), SHAPE), (dict(rotary=66), SHAPE), (dict(rotary=-2), SHAPE),
    (dict(cache=cache(dim=1025)), SHAPE), (dict(q=None), INVALID), (dict(q_out=heads(data=None)), INVALID),
    (dict(k=heads(tok=-1)), INVALID), (dict(v=heads(head=-1)), INVALID), (dict(positions=None), INVALID),
    (dict(slots=None), INVALID), (dict(cos_sin=None), INVALID), (dict(status=None), INVALID), (dict(q=heads(data=P + 1)), ALIGN),
    (dict(positions=P + 2), ALIGN), (dict(slots=P + 4), ALIGN), (dict(cos_sin=P + 4), ALIGN), (dict(status=P + 1), ALIGN)])
def test_rope_refusals(over, code):
    assert rope(**over) == code


def test_quantize_refuses_rows_that_32_bits_do_not_count():
    assert awq.lib().awq_quantize_fp8(P, 1 << 31, P, 1 << 31, P, 3, (1 << 30) + 1, 1, None) == SHAPE


def attention(**over):
    a = dict(q=heads(), cache=cache(), table=P, stride=10, pages=10, lens=P, batch=3, q_heads=4, dtype=0, scale=0.1,
             out=heads(), lse=P, ws=P, ws_bytes=1 << 26, status=P)
    a.update(over)
    return awq.lib().awq_paged_attention(*a.values(), None)


@pytest.mark.parametrize("over,code", CACHE_REFUSALS + [
    (dict(batch=0), OK), (dict(batch=0, q=None, table=None), OK), (dict(batch=-1), INVALID), (dict(q_heads=0), INVALID),
    (dict(pages=0), INVALID), (dict(q_heads=5), SHAPE), (dict(cache=cache(dim=264)), SHAPE), (dict(cache=cache(dim=60)), SHAPE),
    (dict(cache=cache(dtype=2, dim=72)), SHAPE), (dict(q=None), INVALID), (dict(out=heads(data=None)), INVALID),
    (dict(table=None), INVALID), (dict(lens=None), INVALID), (dict(ws=None), INVALID), (dict(status=None), INVALID),
    (dict(stride=9), INVALID), (dict(q=heads(data=P + 8)), ALIGN), (dict(q=heads(tok=516)), ALIGN),
    (dict(out=heads(head=68)), ALIGN), (dict(cache=cache(k=plane(data=P + 2))), ALIGN),
    (dict(cache=cache(v=plane(page=2052))), ALIGN), (dict(cache=cache(dtype=2, k=plane(token=136))), ALIGN),
    (dict(table=P + 2), ALIGN), (dict(lens=P + 2), ALIGN), (dict(lse=P + 2), ALIGN), (dict(ws=P + 128), ALIGN),
    (dict(status=P + 2), ALIGN), (dict(ws_bytes=1000), awq.ERR_WORKSPACE_TOO_SMALL),
    (dict(batch=4096, pages=1 << 27, stride=1 << 27), SHAPE), (dict(batch=1 << 30, pages=64, stride=64), SHAPE),
    (dict(ws_bytes=awq.paged_attention_workspace_bytes(64) - 1), awq.ERR_WORKSPACE_TOO_SMALL)])
def test_attention_refusals(over, code):
    assert attention(**over) == code


@pytest.mark.parametrize("scale", [float("nan"), float("inf"), -float("inf")])
def test_attention_refuses_a_scale_that_is_not_finite(scale):
    assert attention(scale=scale) == INVALID


def test_attention_workspace():
    assert awq.paged_attention_workspace_bytes(0) == awq.paged_attention_workspace_bytes(264) == 0
    assert awq.paged_attention_workspace_bytes(12) == 0
    sizes = [awq.paged_attention_workspace_bytes(n) for n in range(8, 257, 8)]
    assert sizes == sorted(sizes) and sizes[0] > 0


def gemm(**over):
    a = dict(a=P, lda=512, a_scales=P, b=P, ldb=512, b_scales=P, out=P, ldo=256, M=4, N=256, K=512, dtype=0, status=P)
    a.update(over)
    return awq.lib().awq_fp8_gemm(*a.values(), None)


@pytest.mark.parametrize("over,code", [
    (dict(M=0), OK), (dict(N=0), OK), (dict(M=0, a=None), OK), (dict(M=-1), INVALID), (dict(N=-1), INVALID), (dict(K=0), INVALID),
    (dict(dtype=2), INVALID), (dict(a=None), INVALID), (dict(b=None), INVALID), (dict(a_scales=None), INVALID),
    (dict(b_scales=None), INVALID), (dict(out=None), INVALID), (dict(status=None), INVALID), (dict(lda=511), INVALID),
    (dict(ldb=500), INVALID), (dict(ldo=255), INVALID), (dict(lda=520), ALIGN), (dict(ldb=520), ALIGN), (dict(a=P + 8), ALIGN),
    (dict(b=P + 1), ALIGN), (dict(a_scales=P + 2), ALIGN), (dict(b_scales=P + 2), ALIGN), (dict(out=P + 1), ALIGN),
    (dict(status=P + 2), ALIGN)])
def test_gemm_refusals(over, code):
    assert gemm(**over) == code


@pytest.mark.parametrize("size", [dict(M=(1 << 30) + 1), dict(N=(1 << 30) + 1, ldo=1 << 31), dict(K=(1 << 30) + 1, lda=1 << 31, ldb=1 << 31)])
def test_gemm_refuses_sizes_that_32_bits_do_not_count(size):
    assert gemm(**size) == SHAPE


def test_binding_checks_types_shapes_and_devices():
    import torch
    f16, f32, i32, f8 = torch.float16, torch.float32, torch.int32, torch.float8_e4m3fn
    x, w = torch.zeros(4, 256, dtype=f16), torch.zeros(256, dtype=f16)
    with pytest.raises(ValueError, match="CUDA"):
        awq.add_rmsnorm(x, w, 1e-6, out=x)
    with pytest.raises(TypeError, match="x: expected float16 or bfloat16"):
        awq.add_rmsnorm(x.float(), w, 1e-6, out=x)
    with pytest.raises(ValueError, match="2 dimensions"):
        awq.quantize_fp8(w, w, w)
    with pytest.raises(TypeError, match="x: expected a tensor, got NoneType"):
        awq.quantize_fp8(None, w, w)
    q, c = torch.zeros(1, 2, 64, dtype=f16), torch.zeros(1, 1, 1, 64, dtype=f16)
    with pytest.raises(ValueError, match="q: must be a CUDA device tensor, got one on cpu"):
        awq.paged_attention(q, c, c, None, None, None, None, None)
    with pytest.raises(TypeError, match="q: expected float16 or bfloat16, got float32"):
        awq.rope_append(q.float(), None, None, None, None, None, c, c, None)
    with pytest.raises(ValueError, match="3 dimensions"):
        awq.rope_append(q[0], None, None, None, None, None, c, c, None)
    with pytest.raises(ValueError, match="CUDA"):
        awq.fp8_gemm(torch.zeros(4, 256).to(f8), torch.zeros(4, 2), torch.zeros(8, 256).to(f8), torch.zeros(1, 2),
                     torch.zeros(4, 8, dtype=f16), torch.zeros(1, dtype=i32))


def test_binding_names_the_argument_that_is_no_query():
    import torch
    c = torch.zeros(1, 1, 1, 64, dtype=torch.float16)
    with pytest.raises(TypeError, match="q: expected a tensor, got list"):
        awq.paged_attention([1.0], c, c, None, None, None, None, None)
    with pytest.raises(ValueError, match="q: must be a CUDA device tensor"):
        awq.paged_attention(torch.zeros(1, 2, 0, dtype=torch.float16), c, c, None, None, None, None, None)


def test_attention_workspace_of_sizes_that_32_bits_do_not_hold():
    for dim in ((1 << 32) + 64, -(1 << 32) + 64, 1 << 31):
        assert awq.paged_attention_workspace_bytes(dim) == 0
