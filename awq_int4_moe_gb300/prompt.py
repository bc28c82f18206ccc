"""Python binding of ``include/awq_prompt.h``: the operators that take a prompt
through the attention half of a decoder layer.

The manner is that of the decoder operators' binding: each function has its C
entry point's name without the ``awq_`` prefix, takes CUDA tensors (any strides
whose last one is 1) and the caller's outputs, workspace and status word, works
on the current CUDA stream of the tensors' device unless ``stream`` is given and
raises :class:`AwqError` on a non-zero status.
"""
from __future__ import annotations

import ctypes as C

from . import decoder
from .decoder import Heads, KvCache, _handle


def declare(L) -> None:
    """Argument types of the entry points."""
    P, i32, i64, f32, st, size = C.c_void_p, C.c_int32, C.c_int64, C.c_float, C.c_int, C.c_size_t
    HP, CP = C.POINTER(Heads), C.POINTER(KvCache)
    for name, res, args in (
            ("awq_prompt_attention", st, [HP, HP, HP, P, i32, i32, i32, i32, i32, i32, f32, HP, P, P, size, P, P]),
            ("awq_prompt_attention_workspace_bytes", size, [i32]),
            ("awq_chunk_attention", st, [HP, CP, P, i64, i32, P, P, i32, i32, i32, i32, f32, HP, P, P, size, P, P]),
            ("awq_qk_norm_rope_append", st, [HP, HP, HP, HP, P, P, f32, P, P, i32, i32, i32, P, CP, i32, i32, i32, P, P])):
        f = getattr(L, name)
        f.restype, f.argtypes = res, args


def _bind():
    return decoder._bind or decoder._load()


def prompt_attention_workspace_bytes(head_dim: int) -> int:
    """Workspace bytes of prompt_attention and chunk_attention at a head size,
    for any batch."""
    head_dim = int(head_dim)
    if head_dim != C.c_int32(head_dim).value:            # no head size that the C call could be asked about
        return 0
    return int(lib().awq_prompt_attention_workspace_bytes(head_dim))


def prompt_attention(q, k, v, cu_seqlens, out, workspace, dev_status, scale=None, lse=None, stream=None):
    """Causal attention over whole prompts packed one behind the other: sequence
    b has the rows cu_seqlens[b] .. cu_seqlens[b + 1] - 1. q, out: [tokens]
    [q heads][dim]; k, v: [tokens][KV heads][dim]; cu_seqlens i32[batch + 1]; lse
    f32[tokens][q heads] or None; scale: 1 / sqrt(dim) where None. workspace:
    zero-filled once, then reused."""
    code = _bind().prompt_attention(q, k, v, cu_seqlens, out, workspace, dev_status, scale, lse, _handle(stream))
    if code:
        raise AwqError(code, "awq_prompt_attention")


def chunk_attention(q, k_cache, v_cache, page_table, cu_seqlens, seq_lens, out, workspace, dev_status, scale=None, lse=None,
                    k_scale: float = 1.0, v_scale: float = 1.0, stream=None):
    """Causal attention of the newest tokens of each sequence over the paged
    cache, which has them already: sequence b's are the rows cu_seqlens[b] ..
    cu_seqlens[b + 1] - 1 of q and out, the last of its seq_lens[b] tokens.
    q, out: [tokens][q heads][dim]; caches [pages][page size][KV heads][dim];
    page_table i32[batch][max pages]; seq_lens i32[batch]; the rest as in
    prompt_attention, whose workspace serves both."""
    code = _bind().chunk_attention(q, k_cache, v_cache, page_table, cu_seqlens, seq_lens, out, workspace, dev_status, scale, lse,
                                   k_scale, v_scale, _handle(stream))
    if code:
        raise AwqError(code, "awq_chunk_attention")


def qk_norm_rope_append(q, k, v, q_weight, k_weight, eps: float, positions, cos_sin, slots, k_cache, v_cache, dev_status,
                        q_out=None, interleaved: bool = False, k_scale: float = 1.0, v_scale: float = 1.0, stream=None):
    """rope_append with an RMS norm of each head of q and k (weights [dim]) in
    front of the rotation, in the same pass."""
    code = _bind().qk_norm_rope_append(q, k, v, q_weight, k_weight, eps, positions, cos_sin, slots, k_cache, v_cache, dev_status,
                                       q_out, interleaved, k_scale, v_scale, _handle(stream))
    if code:
        raise AwqError(code, "awq_qk_norm_rope_append")


from . import AwqError, lib  # noqa: E402
