"""The decoder operators' binding: what it refuses of CUDA tensors, before any
launch."""
import pytest

import gpu_common as gc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    gc.require_gpu()
    gc.build_all()


def zeros(*shape, dtype="float16"):
    import torch
    t = torch.zeros(shape, device="cuda", dtype=torch.float32)
    return t.to(getattr(torch, dtype))


def refused(kind, text, f, *args, **kw):
    with pytest.raises(kind, match=text):
        f(*args, **kw)


def test_norm():
    import awq_int4_moe_gb300 as awq
    x, w = zeros(4, 256), zeros(256)
    q, s = zeros(4, 256, dtype="float8_e4m3fn"), zeros(4, 2, dtype="float32")
    f = awq.add_rmsnorm
    refused(TypeError, "x: expected float16 or bfloat16, got float32", f, x.float(), w, 1e-6, out=x)
    refused(ValueError, "x: expected 2 dimensions", f, x[0], w, 1e-6, out=x)
    refused(TypeError, "weight: expected float16, got float32", f, x, w.float(), 1e-6, out=x)
    refused(ValueError, "weight: expected shape", f, x, w[:255], 1e-6, out=x)
    refused(TypeError, "residual: expected float16, got bfloat16", f, x, w, 1e-6, residual=x.bfloat16(), out=x)
    refused(ValueError, "residual: expected shape", f, x, w, 1e-6, residual=x[:3], out=x)
    refused(ValueError, "residual_out: expected shape", f, x, w, 1e-6, residual_out=x[:3], out=x)
    refused(ValueError, "out: expected shape", f, x, w, 1e-6, out=x[:, :128])
    refused(ValueError, "out: needs dense rows", f, x, w, 1e-6, out=zeros(256, 4).t())
    refused(ValueError, "out: must be a CUDA device tensor, got one on cpu", f, x, w, 1e-6, out=x.cpu())
    refused(TypeError, "out_q: expected float8_e4m3fn", f, x, w, 1e-6, out_q=x, out_scales=s)
    refused(ValueError, "out_scales: expected shape", f, x, w, 1e-6, out_q=q, out_scales=s[:, :1])
    refused(ValueError, "out_scales: needs dense rows", f, x, w, 1e-6, out_q=q, out_scales=zeros(2, 4, dtype="float32").t())
    refused(TypeError, "must be real number", f, x, w, "eps", out=x)
    refused(awq.AwqError, "invalid argument", f, x, w, 1e-6)                      # no output
    refused(awq.AwqError, "invalid argument", f, x, w, 1e-6, out_q=q)            # no scales
    refused(awq.AwqError, "invalid argument", f, x, w, -1.0, out=x)
    refused(awq.AwqError, "unsupported shape", f, zeros(1, 40000), zeros(40000), 1e-6, out=zeros(1, 40000))
    f(zeros(0, 256), w, 1e-6, out=zeros(0, 256))                                  # nothing to do


def test_quantize():
    import awq_int4_moe_gb300 as awq
    x, q, s = zeros(4, 256), zeros(4, 256, dtype="float8_e4m3fn"), zeros(4, 2, dtype="float32")
    f = awq.quantize_fp8
    refused(TypeError, "out_q: expected a tensor, got NoneType", f, x, None, s)
    refused(ValueError, "out_q: expected shape", f, x, q[:2], s)
    refused(ValueError, "out_scales: expected shape", f, x, q, s[:2])
    refused(TypeError, "out_scales: expected a tensor", f, x, q, None)
    f(zeros(0, 256), zeros(0, 256, dtype="float8_e4m3fn"), zeros(0, 2, dtype="float32"))


def cache(pages=2, page=4, heads=1, dim=64, dtype="float16"):
    return zeros(pages, page, heads, dim, dtype=dtype)


def test_rope():
    import awq_int4_moe_gb300 as awq
    q, k = zeros(3, 2, 64), zeros(3, 1, 64)
    pos, slots, table, st = zeros(3, dtype="int32"), zeros(3, dtype="int64"), zeros(8, 64, dtype="float32"), zeros(1, dtype="int32")
    base = dict(q=q, k=k, v=k, positions=pos, cos_sin=table, slots=slots, k_cache=cache(), v_cache=cache(), dev_status=st)

    def bad(kind, text, **over):
        refused(kind, text, awq.rope_append, **{**base, **over})

    bad(ValueError, "k: expected shape", k=zeros(3, 2, 64))
    bad(TypeError, "v: expected float16", v=k.bfloat16())
    bad(ValueError, "positions: expected shape", positions=pos[:2])
    bad(TypeError, "positions: expected int32, got int64", positions=slots)
    bad(TypeError, "slots: expected int64, got int32", slots=pos)
    bad(TypeError, "cos_sin: expected float32", cos_sin=table.half())
    bad(ValueError, "cos_sin: expected 2 dimensions", cos_sin=table[0])
    bad(TypeError, "v_cache: expected float16, got bfloat16", v_cache=cache(dtype="bfloat16"))
    bad(TypeError, "k_cache: expected float16 or float8_e4m3fn", k_cache=cache(dtype="bfloat16"), v_cache=cache(dtype="bfloat16"))
    bad(ValueError, "one shape", v_cache=cache(pages=3))
    bad(ValueError, "head size 64, the cache's is 128", k_cache=cache(dim=128), v_cache=cache(dim=128))
    bad(ValueError, "k_cache: needs dense rows", k_cache=zeros(2, 4, 1, 128)[..., ::2])
    bad(ValueError, "q_out: expected shape", q_out=zeros(3, 2, 32))
    bad(TypeError, "dev_status: expected int32", dev_status=slots)
    bad(TypeError, "q: expected a tensor, got NoneType", q=None)
    bad(awq.AwqError, "invalid argument", k_scale=0.5)                             # a 16-bit cache has no scale
    bad(awq.AwqError, "unsupported shape", cos_sin=zeros(8, 66, dtype="float32"))
    bad(awq.AwqError, "unsupported shape", cos_sin=zeros(8, 63, dtype="float32"))


def test_attention():
    import awq_int4_moe_gb300 as awq
    q, st = zeros(3, 2, 64), zeros(1, dtype="int32")
    ws = zeros(awq.paged_attention_workspace_bytes(64), dtype="uint8")
    base = dict(q=q, k_cache=cache(), v_cache=cache(), page_table=zeros(3, 2, dtype="int32"), seq_lens=zeros(3, dtype="int32"),
                out=zeros(3, 2, 64), workspace=ws, dev_status=st)

    def bad(kind, text, **over):
        refused(kind, text, awq.paged_attention, **{**base, **over})

    bad(TypeError, "out: expected float16", out=zeros(3, 2, 64, dtype="bfloat16"))
    bad(ValueError, "out: expected shape", out=zeros(2, 2, 64))
    bad(ValueError, "page_table: expected shape", page_table=zeros(2, 2, dtype="int32"))
    bad(ValueError, "page_table: expected 2 dimensions", page_table=zeros(3, dtype="int32"))
    bad(TypeError, "seq_lens: expected int32", seq_lens=zeros(3, dtype="int64"))
    bad(ValueError, "lse: expected shape", lse=zeros(3, 3, dtype="float32"))
    bad(ValueError, "workspace: must be a CUDA", workspace=ws.cpu())
    bad(awq.AwqError, "workspace smaller", workspace=ws[:1024])
    bad(awq.AwqError, "misaligned", workspace=zeros(awq.paged_attention_workspace_bytes(64) + 16, dtype="uint8")[16:])
    bad(awq.AwqError, "unsupported shape", q=zeros(3, 3, 64), out=zeros(3, 3, 64), k_cache=cache(heads=2), v_cache=cache(heads=2))
    bad(awq.AwqError, "unsupported shape", q=zeros(3, 2, 60), out=zeros(3, 2, 60), k_cache=cache(dim=60), v_cache=cache(dim=60))
    bad(awq.AwqError, "misaligned", q=zeros(3, 2, 66)[:, :, :64])
    awq.paged_attention(**base)


def test_gemm():
    import awq_int4_moe_gb300 as awq
    f8 = "float8_e4m3fn"
    base = dict(a=zeros(4, 256, dtype=f8), a_scales=zeros(4, 2, dtype="float32"), b=zeros(8, 256, dtype=f8),
                b_scales=zeros(1, 2, dtype="float32"), out=zeros(4, 8), dev_status=zeros(1, dtype="int32"))

    def bad(kind, text, **over):
        refused(kind, text, awq.fp8_gemm, **{**base, **over})

    bad(TypeError, "a: expected float8_e4m3fn, got float16", a=zeros(4, 256))
    bad(ValueError, "b: expected shape", b=zeros(9, 256, dtype=f8))
    bad(ValueError, "b: expected shape", b=zeros(8, 128, dtype=f8))
    bad(ValueError, "a_scales: expected shape", a_scales=zeros(4, 3, dtype="float32"))
    bad(ValueError, "b_scales: expected shape", b_scales=zeros(2, 2, dtype="float32"))
    bad(TypeError, "out: expected float16 or bfloat16", out=zeros(4, 8, dtype="float32"))
    bad(TypeError, "a: expected a tensor", a=None)
    bad(TypeError, "b: expected a tensor, got NoneType", b=None)
    bad(awq.AwqError, "misaligned", a=zeros(4, 264, dtype=f8)[:, :256])
    awq.fp8_gemm(**base)
    awq.fp8_gemm(**{**base, "a": zeros(0, 256, dtype=f8), "a_scales": zeros(0, 2, dtype="float32"), "out": zeros(0, 8)})


def test_a_given_stream_is_used():
    import torch
    import awq_int4_moe_gb300 as awq
    x, w, out = zeros(4, 256) + 1, zeros(256) + 1, zeros(4, 256)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        out.zero_()
        torch.cuda.synchronize()
        awq.add_rmsnorm(x, w, 0.0, out=out, stream=stream)
        side.synchronize()
        assert bool((out == 1).all())
    with torch.cuda.stream(side):
        out.zero_()
        awq.add_rmsnorm(x, w, 0.0, out=out)
    side.synchronize()
    assert bool((out == 1).all())
