"""The prompt's operators' C ABI and binding without a GPU: every declared symbol
is exported, and what the host can see to be wrong is refused before any CUDA
call."""
import os
import re

import pytest

import awq_int4_moe_gb300 as awq
from awq_int4_moe_gb300 import decoder as d

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "awq_prompt.h")
P = 0x10000000          # a 256-byte aligned non-null address; never dereferenced on these paths
OK, INVALID, SHAPE, ALIGN, SMALL = awq.OK, awq.ERR_INVALID_ARG, awq.ERR_UNSUPPORTED_SHAPE, awq.ERR_MISALIGNED, awq.ERR_WORKSPACE_TOO_SMALL


@pytest.fixture(scope="module", autouse=True)
def _built():
    import awq_int4_moe_gb300.build as b
    b.build()


def test_every_declared_symbol_is_exported():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"AWQ_API\s+[\w\s\*]*?\b(awq_\w+)\s*\(", text))
    assert names == {"awq_prompt_attention", "awq_prompt_attention_workspace_bytes", "awq_chunk_attention", "awq_qk_norm_rope_append"}
    for n in names:
        assert hasattr(awq.lib(), n), n
        assert hasattr(awq, n[4:]), n


def heads(data=P, tok=512, head=64):
    return d.Heads(data, tok, head)


def plane(data=P, scale=1.0, page=2048, token=128, head=64):
    return d.KvPlane(data, page, token, head, scale)


def cache(k=None, v=None, dtype=0, pages=8, page=16, heads=2, dim=64):
    return d.KvCache(k or plane(), v or plane(), dtype, pages, page, heads, dim)


def prompt(**over):
    a = dict(q=heads(), k=heads(), v=heads(), cu=P, batch=3, tokens=50, q_heads=4, kv_heads=2, dim=64, dtype=0, scale=0.1, out=heads(),
             lse=P, ws=P, ws_bytes=1 << 27, status=P)
    a.update(over)
    return awq.lib().awq_prompt_attention(*a.values(), None)


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("over,code", [
    (dict(batch=0), OK), (dict(tokens=0), OK), (dict(tokens=0, q=None, cu=None), OK), (dict(batch=-1), INVALID), (dict(tokens=-1), INVALID),
    (dict(q_heads=0), INVALID), (dict(kv_heads=0), INVALID), (dict(q_heads=5), SHAPE), (dict(dim=0), SHAPE), (dict(dim=60), SHAPE),
    (dict(dim=264), SHAPE), (dict(dtype=2), INVALID), (dict(dtype=-1), INVALID), (dict(scale=NAN), INVALID), (dict(scale=INF), INVALID),
    (dict(scale=-INF), INVALID), (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=heads(data=None)), INVALID),
    (dict(out=heads(tok=-1)), INVALID), (dict(cu=None), INVALID), (dict(ws=None), INVALID), (dict(status=None), INVALID),
    (dict(q=heads(data=P + 8)), ALIGN), (dict(k=heads(tok=516)), ALIGN), (dict(v=heads(head=68)), ALIGN), (dict(out=heads(data=P + 1)), ALIGN),
    (dict(cu=P + 2), ALIGN), (dict(lse=P + 2), ALIGN), (dict(ws=P + 128), ALIGN), (dict(status=P + 2), ALIGN), (dict(ws_bytes=1000), SMALL),
    (dict(ws_bytes=awq.prompt_attention_workspace_bytes(64) - 1), SMALL),
    (dict(tokens=(1 << 31) - 1), SHAPE), (dict(tokens=1 << 30, batch=1 << 30), SHAPE),
    (dict(k=heads(tok=0)), SHAPE), (dict(v=heads(tok=0)), SHAPE), (dict(k=heads(tok=1 << 39)), SHAPE), (dict(v=heads(head=1 << 39)), SHAPE)])
def test_prompt_refusals(over, code):
    assert prompt(**over) == code


CACHE_REFUSALS = [
    (dict(cache=None), INVALID), (dict(cache=cache(dtype=1)), INVALID), (dict(cache=cache(dtype=3)), INVALID),
    (dict(cache=cache(pages=0)), INVALID), (dict(cache=cache(page=0)), INVALID), (dict(cache=cache(heads=0)), INVALID),
    (dict(cache=cache(dim=0)), SHAPE), (dict(cache=cache(k=plane(data=None))), INVALID),
    (dict(cache=cache(v=plane(data=None))), INVALID), (dict(cache=cache(k=plane(scale=0.5))), INVALID),
    (dict(cache=cache(dtype=2, v=plane(scale=0.0))), INVALID), (dict(cache=cache(dtype=2, k=plane(scale=NAN))), INVALID),
    (dict(cache=cache(k=plane(page=-1))), INVALID), (dict(cache=cache(k=plane(data=P + 1))), ALIGN), (dict(dtype=2), INVALID)]


def chunk(**over):
    a = dict(q=heads(), cache=cache(), table=P, stride=10, pages=10, cu=P, lens=P, batch=3, tokens=50, q_heads=4, dtype=0, scale=0.1,
             out=heads(), lse=P, ws=P, ws_bytes=1 << 27, status=P)
    a.update(over)
    return awq.lib().awq_chunk_attention(*a.values(), None)


@pytest.mark.parametrize("over,code", CACHE_REFUSALS + [
    (dict(batch=0), OK), (dict(tokens=0), OK), (dict(batch=0, q=None, table=None), OK), (dict(batch=-1), INVALID), (dict(tokens=-1), INVALID),
    (dict(q_heads=0), INVALID), (dict(pages=0), INVALID), (dict(q_heads=5), SHAPE), (dict(cache=cache(dim=264)), SHAPE),
    (dict(cache=cache(dim=60)), SHAPE), (dict(cache=cache(dtype=2, dim=72)), SHAPE), (dict(scale=NAN), INVALID), (dict(q=None), INVALID),
    (dict(out=heads(data=None)), INVALID), (dict(table=None), INVALID), (dict(cu=None), INVALID), (dict(lens=None), INVALID),
    (dict(ws=None), INVALID), (dict(status=None), INVALID), (dict(stride=9), INVALID), (dict(q=heads(data=P + 8)), ALIGN),
    (dict(q=heads(tok=516)), ALIGN), (dict(out=heads(head=68)), ALIGN), (dict(cache=cache(k=plane(data=P + 2))), ALIGN),
    (dict(cache=cache(v=plane(page=2052))), ALIGN), (dict(cache=cache(dtype=2, k=plane(token=136))), ALIGN), (dict(table=P + 2), ALIGN),
    (dict(cu=P + 2), ALIGN), (dict(lens=P + 2), ALIGN), (dict(lse=P + 2), ALIGN), (dict(ws=P + 128), ALIGN), (dict(status=P + 2), ALIGN),
    (dict(ws_bytes=1000), SMALL), (dict(tokens=(1 << 31) - 1), SHAPE), (dict(batch=1 << 30, tokens=1 << 20, pages=1 << 26, stride=1 << 26), SHAPE),
    (dict(cache=cache(k=plane(token=0))), SHAPE), (dict(cache=cache(v=plane(page=1 << 39))), SHAPE)])
def test_chunk_refusals(over, code):
    assert chunk(**over) == code


def norm(**over):
    a = dict(q=heads(), q_out=heads(), k=heads(), v=heads(), qw=P, kw=P, eps=1e-6, positions=P, cos_sin=P, top=100, rotary=64, inter=0,
             slots=P, cache=cache(), tokens=4, q_heads=4, dtype=0, status=P)
    a.update(over)
    return awq.lib().awq_qk_norm_rope_append(*a.values(), None)


@pytest.mark.parametrize("over,code", CACHE_REFUSALS + [
    (dict(tokens=0), OK), (dict(tokens=0, q=None, qw=None), OK), (dict(tokens=-1), INVALID), (dict(q_heads=0), INVALID),
    (dict(top=0), INVALID), (dict(rotary=63), SHAPE), (dict(rotary=66), SHAPE), (dict(cache=cache(dim=1025)), SHAPE), (dict(q=None), INVALID),
    (dict(q_out=heads(data=None)), INVALID), (dict(k=heads(tok=-1)), INVALID), (dict(v=heads(head=-1)), INVALID), (dict(positions=None), INVALID),
    (dict(slots=None), INVALID), (dict(cos_sin=None), INVALID), (dict(status=None), INVALID), (dict(qw=None), INVALID), (dict(kw=None), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=NAN), INVALID), (dict(eps=INF), INVALID), (dict(qw=P + 1), ALIGN), (dict(kw=P + 1), ALIGN),
    (dict(q=heads(data=P + 1)), ALIGN), (dict(positions=P + 2), ALIGN), (dict(slots=P + 4), ALIGN), (dict(cos_sin=P + 4), ALIGN),
    (dict(status=P + 1), ALIGN)])
def test_append_refusals(over, code):
    assert norm(**over) == code


def test_workspace():
    assert awq.prompt_attention_workspace_bytes(0) == awq.prompt_attention_workspace_bytes(264) == awq.prompt_attention_workspace_bytes(12) == 0
    assert all(awq.prompt_attention_workspace_bytes(n) > 0 for n in range(8, 257, 8))
    for dim in ((1 << 32) + 64, -(1 << 32) + 64, 1 << 31):
        assert awq.prompt_attention_workspace_bytes(dim) == 0


def test_binding_checks_types_shapes_and_devices():
    import torch
    q, c = torch.zeros(3, 2, 64, dtype=torch.float16), torch.zeros(1, 1, 1, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="q: must be a CUDA device tensor, got one on cpu"):
        awq.prompt_attention(q, q, q, None, q, None, None)
    with pytest.raises(TypeError, match="q: expected float16 or bfloat16, got float32"):
        awq.prompt_attention(q.float(), q, q, None, q, None, None)
    with pytest.raises(TypeError, match="q: expected a tensor, got NoneType"):
        awq.prompt_attention(None, q, q, None, q, None, None)
    with pytest.raises(ValueError, match="q: expected 3 dimensions"):
        awq.chunk_attention(q[0], c, c, None, None, None, None, None, None)
    with pytest.raises(ValueError, match="CUDA"):
        awq.chunk_attention(q, c, c, None, None, None, None, None, None)
    with pytest.raises(TypeError, match="q: expected float16 or bfloat16, got float32"):
        awq.qk_norm_rope_append(q.float(), None, None, None, None, 1e-6, None, None, None, c, c, None)
    with pytest.raises(ValueError, match="CUDA"):
        awq.qk_norm_rope_append(q, q, q, q, q, 1e-6, None, None, None, c, c, None)
