"""Python binding of ``include/awq_decoder.h``: the decoder layer's operators
around the expert stage.

Each function has its C entry point's name without the ``awq_`` prefix, takes
CUDA tensors (any strides whose last one is 1, unless stated otherwise), takes
sizes and strides from them and raises :class:`AwqError` on a non-zero status.
Outputs, the workspace and the status word are the caller's tensors; work goes
to the current CUDA stream of the tensors' device unless ``stream`` is given.
The checks that the C call cannot make (types, shapes, devices) are in
``csrc/awq_bind.cpp``.
"""
from __future__ import annotations

import ctypes as C
import os

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


_bind = None


def _load():
    """The binding module, built beside the library; there is no other."""
    global _bind
    import importlib.machinery
    import importlib.util

    import torch  # noqa: F401  (its libraries are what the module links to)
    path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_bind.so")
    if not os.path.exists(path):
        raise RuntimeError(f"binding module {path} is missing; build it with awq_int4_moe_gb300.build.build()")
    lib()
    loader = importlib.machinery.ExtensionFileLoader("awq_int4_moe_gb300._bind", path)
    _bind = importlib.util.module_from_spec(importlib.util.spec_from_loader(loader.name, loader))
    loader.exec_module(_bind)
    return _bind


def _handle(stream):
    return stream if stream is None or isinstance(stream, int) else stream.cuda_stream


def add_rmsnorm(x, weight, eps: float, residual=None, residual_out=None, out=None, out_q=None, out_scales=None,
                stream=None):
    """r = x + residual; out = r / rms(r) * weight, and / or as e4m3 with a
    scale per 128 columns (out_q, out_scales f32[rows][ceil(hidden / 128)]);
    residual_out = r. x, residual, residual_out, out: [rows][hidden]."""
    code = (_bind or _load()).add_rmsnorm(x, weight, eps, residual, residual_out, out, out_q, out_scales, _handle(stream))
    if code:
        raise AwqError(code, "awq_add_rmsnorm")


def quantize_fp8(x, out_q, out_scales, stream=None):
    """[rows][cols] activations to e4m3 with a scale per row and 128 columns."""
    code = (_bind or _load()).quantize_fp8(x, out_q, out_scales, _handle(stream))
    if code:
        raise AwqError(code, "awq_quantize_fp8")


def rope_append(q, k, v, positions, cos_sin, slots, k_cache, v_cache, dev_status, q_out=None,
                interleaved: bool = False, k_scale: float = 1.0, v_scale: float = 1.0, stream=None):
    """Rotate q (into q_out; in place where that is None) and k by position and
    append k and v to the cache [pages][page size][KV heads][dim]. q: [tokens]
    [q heads][dim]; k, v: [tokens][KV heads][dim]; positions i32, slots i64
    [tokens]; cos_sin f32[positions][rotary dim], cosines then sines."""
    code = (_bind or _load()).rope_append(q, k, v, positions, cos_sin, slots, k_cache, v_cache, dev_status, q_out, interleaved,
                                          k_scale, v_scale, _handle(stream))
    if code:
        raise AwqError(code, "awq_rope_append")


def paged_attention_workspace_bytes(head_dim: int) -> int:
    """Workspace bytes of paged_attention at a head size, for any batch."""
    head_dim = int(head_dim)
    if head_dim != C.c_int32(head_dim).value:            # no head size that the C call could be asked about
        return 0
    return int(lib().awq_paged_attention_workspace_bytes(head_dim))


def paged_attention(q, k_cache, v_cache, page_table, seq_lens, out, workspace, dev_status, scale=None, lse=None,
                    k_scale: float = 1.0, v_scale: float = 1.0, stream=None):
    """Attention of one new token per sequence over the paged cache. q, out:
    [batch][q heads][dim]; page_table i32[batch][max pages]; seq_lens
    i32[batch]; lse f32[batch][q heads] or None; scale: 1 / sqrt(dim) where
    None. workspace: zero-filled once, then reused."""
    code = (_bind or _load()).paged_attention(q, k_cache, v_cache, page_table, seq_lens, out, workspace, dev_status, scale, lse,
                                              k_scale, v_scale, _handle(stream))
    if code:
        raise AwqError(code, "awq_paged_attention")


def fp8_gemm(a, a_scales, b, b_scales, out, dev_status, stream=None):
    """out[M][N] = a[M][K] b[N][K]^T, e4m3 operands with a scale per 128 columns
    of K (a_scales f32[M][ceil(K / 128)]) and per 128 x 128 block (b_scales
    f32[ceil(N / 128)][ceil(K / 128)])."""
    code = (_bind or _load()).fp8_gemm(a, a_scales, b, b_scales, out, dev_status, _handle(stream))
    if code:
        raise AwqError(code, "awq_fp8_gemm")


from . import AwqError, lib  # noqa: E402
