"""Python binding of ``include/awq_decoder.h``: the decoder layer's operators
around the expert stage.

Each function has its C entry point's name without the ``awq_`` prefix, takes
CUDA tensors (any strides whose last one is 1, unless stated otherwise), takes
sizes and strides from them, checks what the C call cannot see (types, shapes,
devices) and raises :class:`AwqError` on a non-zero status. Outputs, the
workspace and the status word are the caller's tensors; work goes to the
current CUDA stream unless ``stream`` is given.
"""
from __future__ import annotations

import ctypes as C

DTYPE_F16, DTYPE_BF16, DTYPE_E4M3 = 0, 1, 2     # awq_dtype
FP8_BLOCK = 128                                 # AWQ_FP8_BLOCK


class Heads(C.Structure):
    _fields_ = [("data", C.c_void_p), ("token_stride", C.c_int64), ("head_stride", C.c_int64)]


class KvPlane(C.Structure):
    _fields_ = [("data", C.c_void_p), ("page_stride", C.c_int64), ("token_stride", C.c_int64),
                ("head_stride", C.c_int64), ("scale", C.c_float)]


class KvCache(C.Structure):
    _fields_ = [("k", KvPlane), ("v", KvPlane), ("dtype", C.c_int32), ("num_pages", C.c_int32),
                ("page_size", C.c_int32), ("num_heads", C.c_int32), ("head_dim", C.c_int32)]


def declare(L) -> None:
    """Argument types of the entry points."""
    P, i32, i64, f32, st = C.c_void_p, C.c_int32, C.c_int64, C.c_float, C.c_int
    HP, CP = C.POINTER(Heads), C.POINTER(KvCache)
    for name, res, args in (
            ("awq_add_rmsnorm", st, [P, i64, P, i64, P, i64, P, f32, P, i64, P, i64, P, i32, i32, i32, P]),
            ("awq_quantize_fp8", st, [P, i64, P, i64, P, i32, i32, i32, P]),
            ("awq_rope_append", st, [HP, HP, HP, HP, P, P, i32, i32, i32, P, CP, i32, i32, i32, P, P]),
            ("awq_paged_attention_workspace_bytes", C.c_size_t, [i32]),
            ("awq_paged_attention", st, [HP, CP, P, i64, i32, P, i32, i32, i32, f32, HP, P, P, C.c_size_t, P, P]),
            ("awq_fp8_gemm", st, [P, i64, P, P, i64, P, P, i64, i32, i32, i32, i32, P, P])):
        f = getattr(L, name)
        f.restype, f.argtypes = res, args


_T = None


def _types():
    """torch dtypes by role (torch is imported on first use)."""
    global _T
    if _T is None:
        import torch
        _T = ({torch.float16: DTYPE_F16, torch.bfloat16: DTYPE_BF16}, torch.float8_e4m3fn, torch.float32,
              torch.int32, torch.int64)
    return _T


def _bad(name, t, dtype, shape):
    """The error of a tensor that is not what the call needs."""
    if t.dtype != dtype:
        return TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        return ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_cuda:
        return ValueError(f"{name}: must be a CUDA device tensor, got one on {t.device}")
    return ValueError(f"{name}: needs dense rows (last stride 1{', contiguous' if t.dim() == 1 else ''}), "
                      f"got strides {tuple(t.stride())}")


def _rows(name, t, dtype, shape):
    """Address and row stride of a 2D tensor with dense rows."""
    if t is None:
        return None, 0
    if t.dtype != dtype or t.shape != shape or not t.is_cuda:
        raise _bad(name, t, dtype, shape)
    ld, one = t.stride()
    if one != 1 and shape[1] > 1:
        raise _bad(name, t, dtype, shape)
    # a single row's stride carries no information and may be anything
    return t.data_ptr(), ld if shape[0] > 1 else max(ld, shape[1])


def _dense(name, t, dtype, shape):
    """Address of a contiguous tensor."""
    if t.dtype != dtype or t.shape != shape or not t.is_cuda or not t.is_contiguous():
        raise _bad(name, t, dtype, shape)
    return t.data_ptr()


_raw_stream = None


def _queue(t, stream):
    """The CUDA stream of a call: the current one of the tensor's device, unless given."""
    if stream is not None:
        return _stream(stream)
    global _raw_stream
    if _raw_stream is None:
        import torch
        # the current stream's handle without building a Stream object (2.8 of the 9 us a call took here)
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
            (lambda device: torch.cuda.current_stream(device).cuda_stream)
    return _raw_stream(t.get_device())


def _status(t):
    if t.dtype != _types()[3] or t.numel() < 1 or not t.is_cuda:
        raise _bad("dev_status", t, _types()[3], (1,))
    return t.data_ptr()


def _activation(name, t, dims):
    code = _types()[0].get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: expected float16 or bfloat16, got {t.dtype}")
    if t.dim() != dims:
        raise ValueError(f"{name}: expected {dims} dimensions, got shape {tuple(t.shape)}")
    return code


def _heads(name, t, dtype, shape):
    if t.dtype != dtype or t.shape != shape or not t.is_cuda:
        raise _bad(name, t, dtype, shape)
    tok, head, one = t.stride()
    if one != 1 and shape[2] > 1:
        raise _bad(name, t, dtype, shape)
    return Heads(t.data_ptr(), tok, head)


def _cache(k_cache, v_cache, k_scale, v_scale, act_dtype):
    """The descriptor of a cache [pages][page size][KV heads][head dim] (any strides but the last)."""
    if k_cache.dtype != v_cache.dtype:
        raise TypeError(f"v_cache: expected {k_cache.dtype}, got {v_cache.dtype}")
    if k_cache.dtype == _types()[1]:
        code = DTYPE_E4M3
    elif k_cache.dtype == act_dtype:
        code = _types()[0][act_dtype]
    else:
        raise TypeError(f"k_cache: expected {act_dtype} or float8_e4m3fn, got {k_cache.dtype}")
    shape = k_cache.shape
    if len(shape) != 4 or v_cache.shape != shape:
        raise ValueError(f"k_cache, v_cache: expected one shape [pages][page size][heads][dim], got {tuple(shape)} "
                         f"and {tuple(v_cache.shape)}")
    if not (k_cache.is_cuda and v_cache.is_cuda):
        raise ValueError(f"k_cache, v_cache: must be CUDA device tensors, got {k_cache.device} and {v_cache.device}")
    pages, page, heads, dim = shape
    ks, vs = k_cache.stride(), v_cache.stride()
    if (ks[3] != 1 or vs[3] != 1) and dim > 1:
        raise ValueError(f"k_cache, v_cache: the last stride must be 1, got {ks} and {vs}")
    return KvCache(KvPlane(k_cache.data_ptr(), ks[0], ks[1], ks[2], k_scale),
                   KvPlane(v_cache.data_ptr(), vs[0], vs[1], vs[2], v_scale), code, pages, page, heads, dim)


def add_rmsnorm(x, weight, eps: float, residual=None, residual_out=None, out=None, out_q=None, out_scales=None,
                stream=None):
    """r = x + residual; out = r / rms(r) * weight, and / or as e4m3 with a
    scale per 128 columns (out_q, out_scales f32[rows][ceil(hidden / 128)]);
    residual_out = r. x, residual, residual_out, out: [rows][hidden]."""
    code = _activation("x", x, 2)
    dt, shape = x.dtype, x.shape
    rows, hidden = shape
    px, ldx = _rows("x", x, dt, shape)
    pr, ldr = _rows("residual", residual, dt, shape)
    pro, ldro = _rows("residual_out", residual_out, dt, shape)
    po, ldo = _rows("out", out, dt, shape)
    pq, ldq = _rows("out_q", out_q, _types()[1], shape)
    ps = None if out_scales is None else _dense("out_scales", out_scales, _types()[2],
                                                (rows, (hidden + FP8_BLOCK - 1) // FP8_BLOCK))
    pw = _dense("weight", weight, dt, (hidden,))
    _check(lib().awq_add_rmsnorm(px, ldx, pr, ldr, pro, ldro, pw, eps, po, ldo, pq, ldq, ps, rows, hidden, code,
                                 _queue(x, stream)), "awq_add_rmsnorm")


def quantize_fp8(x, out_q, out_scales, stream=None):
    """[rows][cols] activations to e4m3 with a scale per row and 128 columns."""
    code = _activation("x", x, 2)
    rows, cols = x.shape
    px, ldx = _rows("x", x, x.dtype, x.shape)
    pq, ldq = _rows("out_q", out_q, _types()[1], x.shape)
    ps = _dense("out_scales", out_scales, _types()[2], (rows, (cols + FP8_BLOCK - 1) // FP8_BLOCK))
    _check(lib().awq_quantize_fp8(px, ldx, pq, ldq, ps, rows, cols, code, _queue(x, stream)), "awq_quantize_fp8")


def rope_append(q, k, v, positions, cos_sin, slots, k_cache, v_cache, dev_status, q_out=None,
                interleaved: bool = False, k_scale: float = 1.0, v_scale: float = 1.0, stream=None):
    """Rotate q (into q_out; in place where that is None) and k by position and
    append k and v to the cache [pages][page size][KV heads][dim]. q: [tokens]
    [q heads][dim]; k, v: [tokens][KV heads][dim]; positions i32, slots i64
    [tokens]; cos_sin f32[positions][rotary dim], cosines then sines."""
    code = _activation("q", q, 3)
    dt, shape = q.dtype, q.shape
    cache = _cache(k_cache, v_cache, k_scale, v_scale, dt)
    tokens, q_heads, dim = shape
    if dim != cache.head_dim:
        raise ValueError(f"q: head size {dim}, the cache's is {cache.head_dim}")
    kv_shape = (tokens, cache.num_heads, dim)
    hq = _heads("q", q, dt, shape)
    ho = hq if q_out is None else _heads("q_out", q_out, dt, shape)
    hk, hv = _heads("k", k, dt, kv_shape), _heads("v", v, dt, kv_shape)
    if cos_sin.dim() != 2:
        raise ValueError(f"cos_sin: expected 2 dimensions, got shape {tuple(cos_sin.shape)}")
    top, rotary = cos_sin.shape
    _, _, f32, i32, i64 = _types()
    pc = _dense("cos_sin", cos_sin, f32, (top, rotary))
    pp, ps = _dense("positions", positions, i32, (tokens,)), _dense("slots", slots, i64, (tokens,))
    _check(lib().awq_rope_append(hq, ho, hk, hv, pp, pc, top, rotary, int(interleaved), ps, cache, tokens, q_heads,
                                 code, _status(dev_status), _queue(q, stream)), "awq_rope_append")


def paged_attention_workspace_bytes(head_dim: int) -> int:
    """Workspace bytes of paged_attention at a head size, for any batch."""
    return int(lib().awq_paged_attention_workspace_bytes(int(head_dim)))


def paged_attention(q, k_cache, v_cache, page_table, seq_lens, out, workspace, dev_status, scale=None, lse=None,
                    k_scale: float = 1.0, v_scale: float = 1.0, stream=None):
    """Attention of one new token per sequence over the paged cache. q, out:
    [batch][q heads][dim]; page_table i32[batch][max pages]; seq_lens
    i32[batch]; lse f32[batch][q heads] or None; scale: 1 / sqrt(dim) where
    None. workspace: zero-filled once, then reused."""
    code = _activation("q", q, 3)
    dt, shape = q.dtype, q.shape
    batch, q_heads, dim = shape
    cache = _cache(k_cache, v_cache, k_scale, v_scale, dt)
    if dim != cache.head_dim:
        raise ValueError(f"q: head size {dim}, the cache's is {cache.head_dim}")
    hq, ho = _heads("q", q, dt, shape), _heads("out", out, dt, shape)
    _, _, f32, i32, _ = _types()
    if page_table.dim() != 2:
        raise ValueError(f"page_table: expected 2 dimensions, got shape {tuple(page_table.shape)}")
    pages = page_table.shape[1]
    pt, ldt = _rows("page_table", page_table, i32, (batch, pages))
    pl = _dense("seq_lens", seq_lens, i32, (batch,))
    ps = None if lse is None else _dense("lse", lse, f32, (batch, q_heads))
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace: must be a contiguous CUDA device tensor")
    _check(lib().awq_paged_attention(hq, cache, pt, ldt, pages, pl, batch, q_heads, code,
                                     dim ** -0.5 if scale is None else scale, ho, ps, workspace.data_ptr(),
                                     workspace.numel() * workspace.element_size(), _status(dev_status),
                                     _queue(q, stream)), "awq_paged_attention")


def fp8_gemm(a, a_scales, b, b_scales, out, dev_status, stream=None):
    """out[M][N] = a[M][K] b[N][K]^T, e4m3 operands with a scale per 128 columns
    of K (a_scales f32[M][ceil(K / 128)]) and per 128 x 128 block (b_scales
    f32[ceil(N / 128)][ceil(K / 128)])."""
    code = _activation("out", out, 2)
    m, n = out.shape
    if a.dim() != 2:
        raise ValueError(f"a: expected 2 dimensions, got shape {tuple(a.shape)}")
    k = a.shape[1]
    _, f8, f32, _, _ = _types()
    kb = (k + FP8_BLOCK - 1) // FP8_BLOCK
    pa, lda = _rows("a", a, f8, (m, k))
    pb, ldb = _rows("b", b, f8, (n, k))
    po, ldo = _rows("out", out, out.dtype, (m, n))
    pas = _dense("a_scales", a_scales, f32, (m, kb))
    pbs = _dense("b_scales", b_scales, f32, ((n + FP8_BLOCK - 1) // FP8_BLOCK, kb))
    _check(lib().awq_fp8_gemm(pa, lda, pas, pb, ldb, pbs, po, ldo, m, n, k, code, _status(dev_status),
                              _queue(out, stream)), "awq_fp8_gemm")


from . import _check, _stream, lib  # noqa: E402
