"""The prompt's operators' binding: what it refuses of CUDA tensors, before any
launch, and the stream it works on."""
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


def ints(*values, dtype="int32"):
    import torch
    return torch.tensor(values, dtype=getattr(torch, dtype), device="cuda")


def cache(pages=2, page=4, heads=1, dim=64, dtype="float16"):
    return zeros(pages, page, heads, dim, dtype=dtype)


def refused(f, base):
    def bad(kind, text, **over):
        with pytest.raises(kind, match=text):
            f(**{**base, **over})
    return bad


def scratch(dim=64):
    import awq_int4_moe_gb300 as awq
    return zeros(awq.prompt_attention_workspace_bytes(dim), dtype="uint8")


def test_prompt_attention():
    import awq_int4_moe_gb300 as awq
    q, k, ws = zeros(5, 4, 64), zeros(5, 2, 64), scratch()
    base = dict(q=q, k=k, v=k, cu_seqlens=ints(0, 2, 5), out=zeros(5, 4, 64), workspace=ws, dev_status=ints(0))
    bad = refused(awq.prompt_attention, base)
    bad(TypeError, "q: expected float16 or bfloat16, got float32", q=q.float())
    bad(TypeError, "q: expected a tensor, got NoneType", q=None)
    bad(ValueError, "q: expected 3 dimensions", q=q[0])
    bad(TypeError, "k: expected float16, got bfloat16", k=k.bfloat16())
    bad(ValueError, "k: expected 3 dimensions", k=k[0])
    bad(ValueError, "k: expected shape", k=k[:4])
    bad(ValueError, "v: expected shape", v=zeros(5, 1, 64))
    bad(ValueError, "v: expected shape", v=zeros(5, 2, 72))
    bad(ValueError, "out: expected shape", out=zeros(5, 2, 64))
    bad(TypeError, "out: expected float16", out=zeros(5, 4, 64, dtype="bfloat16"))
    bad(ValueError, "out: must be a CUDA device tensor, got one on cpu", out=zeros(5, 4, 64).cpu())
    bad(TypeError, "cu_seqlens: expected int32, got int64", cu_seqlens=ints(0, 2, 5, dtype="int64"))
    bad(ValueError, "cu_seqlens: expected shape", cu_seqlens=zeros(2, 2, dtype="int32"))
    bad(ValueError, "cu_seqlens: expected shape", cu_seqlens=zeros(0, dtype="int32"))
    bad(ValueError, "lse: expected shape", lse=zeros(4, 5, dtype="float32"))
    bad(TypeError, "lse: expected float32", lse=q[..., 0].contiguous())
    bad(TypeError, "dev_status: expected int32", dev_status=ints(0, dtype="int64"))
    bad(TypeError, "must be real number", scale="half")
    bad(ValueError, "workspace: must be a CUDA", workspace=ws.cpu())
    bad(awq.AwqError, "workspace smaller", workspace=ws[:-1])
    bad(awq.AwqError, "misaligned", workspace=zeros(ws.numel() + 16, dtype="uint8")[16:])
    bad(awq.AwqError, "misaligned", q=zeros(5, 4, 66)[:, :, :64])
    bad(awq.AwqError, "misaligned", k=zeros(5, 2, 68)[:, :, 1:65])
    bad(awq.AwqError, "invalid argument", scale=float("inf"))
    bad(awq.AwqError, "unsupported shape", k=zeros(5, 3, 64), v=zeros(5, 3, 64))
    bad(awq.AwqError, "unsupported shape", q=zeros(5, 4, 60), k=zeros(5, 2, 60), v=zeros(5, 2, 60), out=zeros(5, 4, 60))
    bad(awq.AwqError, "unsupported shape", q=zeros(5, 4, 264), k=zeros(5, 2, 264), v=zeros(5, 2, 264), out=zeros(5, 4, 264))
    bad(awq.AwqError, "unsupported shape", k=zeros(1, 2, 64).expand(5, 2, 64))           # one key for all tokens
    bad(awq.AwqError, "unsupported shape", v=zeros(1, 2, 64).expand(5, 2, 64))
    awq.prompt_attention(**base)
    empty = zeros(0, 4, 64)
    awq.prompt_attention(empty, zeros(0, 2, 64), zeros(0, 2, 64), ints(0, 0), empty, ws, ints(0))
    awq.prompt_attention(**{**base, "cu_seqlens": ints(0)})                                 # no sequences


def test_chunk_attention():
    import awq_int4_moe_gb300 as awq
    q, ws, f8 = zeros(3, 2, 64), scratch(), "float8_e4m3fn"
    base = dict(q=q, k_cache=cache(), v_cache=cache(), page_table=zeros(2, 2, dtype="int32"), cu_seqlens=ints(0, 1, 3),
                seq_lens=ints(4, 2), out=zeros(3, 2, 64), workspace=ws, dev_status=ints(0))
    bad = refused(awq.chunk_attention, base)
    bad(ValueError, "q: expected 3 dimensions", q=q[0])
    bad(ValueError, "head size 64, the cache's is 128", k_cache=cache(dim=128), v_cache=cache(dim=128))
    bad(TypeError, "k_cache: expected float16 or float8_e4m3fn", k_cache=cache(dtype="bfloat16"), v_cache=cache(dtype="bfloat16"))
    bad(ValueError, "one shape", v_cache=cache(pages=3))
    bad(ValueError, "k_cache: needs dense rows", k_cache=zeros(2, 4, 1, 128)[..., ::2])
    bad(ValueError, "page_table: expected 2 dimensions", page_table=zeros(2, dtype="int32"))
    bad(ValueError, "page_table: expected shape", page_table=zeros(3, 2, dtype="int32"))
    bad(ValueError, "seq_lens: expected shape", seq_lens=ints(4, 2, 1))
    bad(TypeError, "seq_lens: expected int32", seq_lens=ints(4, 2, dtype="int64"))
    bad(TypeError, "cu_seqlens: expected a tensor, got NoneType", cu_seqlens=None)
    bad(ValueError, "out: expected shape", out=zeros(2, 2, 64))
    bad(ValueError, "lse: expected shape", lse=zeros(3, 3, dtype="float32"))
    bad(ValueError, "workspace: must be a CUDA", workspace=ws.cpu())
    bad(awq.AwqError, "workspace smaller", workspace=ws[:1024])
    bad(awq.AwqError, "invalid argument", k_scale=0.5)                                      # a 16-bit cache has no scale
    bad(awq.AwqError, "invalid argument", page_table=zeros(2, 0, dtype="int32"))
    bad(awq.AwqError, "unsupported shape", q=zeros(3, 3, 64), out=zeros(3, 3, 64), k_cache=cache(heads=2), v_cache=cache(heads=2))
    bad(awq.AwqError, "unsupported shape", q=zeros(3, 2, 72), out=zeros(3, 2, 72), k_cache=cache(dim=72, dtype=f8),
        v_cache=cache(dim=72, dtype=f8))
    bad(awq.AwqError, "unsupported shape", k_cache=zeros(2, 1, 1, 64).expand(2, 4, 1, 64))
    bad(awq.AwqError, "misaligned", out=zeros(3, 2, 66)[:, :, :64])
    awq.chunk_attention(**base)
    awq.chunk_attention(**{**base, "q": zeros(0, 2, 64), "out": zeros(0, 2, 64), "cu_seqlens": ints(0, 0, 0)})


def test_append():
    import awq_int4_moe_gb300 as awq
    q, k, w = zeros(3, 2, 64), zeros(3, 1, 64), zeros(64)
    base = dict(q=q, k=k, v=k, q_weight=w, k_weight=w, eps=1e-6, positions=ints(0, 1, 2), cos_sin=zeros(8, 64, dtype="float32"),
                slots=ints(0, 1, 2, dtype="int64"), k_cache=cache(), v_cache=cache(), dev_status=ints(0))
    bad = refused(awq.qk_norm_rope_append, base)
    bad(ValueError, "k: expected shape", k=zeros(3, 2, 64))
    bad(TypeError, "v: expected float16", v=k.bfloat16())
    bad(ValueError, "q_weight: expected shape", q_weight=zeros(2, 64))
    bad(ValueError, "k_weight: expected shape", k_weight=zeros(32))
    bad(TypeError, "k_weight: expected float16, got float32", k_weight=w.float())
    bad(TypeError, "q_weight: expected a tensor, got NoneType", q_weight=None)
    bad(TypeError, "must be real number", eps="small")
    bad(ValueError, "positions: expected shape", positions=ints(0, 1))
    bad(TypeError, "slots: expected int64, got int32", slots=ints(0, 1, 2))
    bad(TypeError, "cos_sin: expected float32", cos_sin=zeros(8, 64))
    bad(ValueError, "q_out: expected shape", q_out=zeros(3, 2, 32))
    bad(ValueError, "one shape", v_cache=cache(pages=3))
    bad(awq.AwqError, "invalid argument", eps=-1.0)
    bad(awq.AwqError, "invalid argument", v_scale=0.5)
    bad(awq.AwqError, "unsupported shape", cos_sin=zeros(8, 66, dtype="float32"))
    awq.qk_norm_rope_append(**base)


def test_a_given_stream_is_used():
    import torch
    import awq_int4_moe_gb300 as awq
    q, k = zeros(4, 2, 64), zeros(4, 1, 64) + 1
    out, cu, st, ws, w = zeros(4, 2, 64), ints(0, 4), ints(0), scratch(), zeros(64) + 1
    kc, vc = cache(), cache()
    table, lens, slots = ints(0, 1).view(1, 2), ints(4), ints(0, 1, 2, 3, dtype="int64")
    positions, cos_sin = ints(0, 1, 2, 3), torch.cat([torch.ones(8, 32, device="cuda"), torch.zeros(8, 32, device="cuda")], 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def all_three(**stream):
        awq.qk_norm_rope_append(q, k, k, w, w, 0.0, positions, cos_sin, slots, kc, vc, st, **stream)
        awq.prompt_attention(q, k, k, cu, out, ws, st, **stream)
        first = out.clone() if not stream else None
        awq.chunk_attention(q, kc, vc, table, cu, lens, out, ws, st, **stream)
        return first

    for stream in (side, side.cuda_stream):
        out.zero_(), kc.zero_(), vc.zero_(), q.fill_(2)
        torch.cuda.synchronize()
        all_three(stream=stream)
        side.synchronize()
        assert bool((out == 1).all()) and bool((kc[0] == 1).all()) and bool((q == 1).all())
    with torch.cuda.stream(side):
        out.zero_(), kc.zero_(), vc.zero_(), q.fill_(2)
        first = all_three()
    side.synchronize()
    assert bool((out == 1).all()) and bool((first == 1).all()) and int(st) == 0
