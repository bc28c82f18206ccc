// Argument checks that the host sides of awq_decoder.h and awq_prompt.h share.
#pragma once

#include <cmath>

#include "awq_decoder_kernels.cuh"

namespace awq {

inline bool aligned(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// A multiple of `a` bytes in both (a NULL pointer is).
inline bool aligned_rows(const void *p, int64_t ld, int64_t elem, int64_t a) { return !p || (aligned(p, a) && ld * elem % a == 0); }

inline awq_status check_dtype(int32_t dtype)
{
    return dtype == AWQ_DTYPE_F16 || dtype == AWQ_DTYPE_BF16 ? AWQ_OK : AWQ_ERR_INVALID_ARG;
}

inline awq_status check_heads(const awq_heads *h)
{
    if (!h || !h->data || h->token_stride < 0 || h->head_stride < 0) return AWQ_ERR_INVALID_ARG;
    return aligned(h->data, 2) ? AWQ_OK : AWQ_ERR_MISALIGNED;
}

inline awq_status check_plane(const awq_kv_plane &p, bool fp8)
{
    if (!p.data || p.page_stride < 0 || p.token_stride < 0 || p.head_stride < 0) return AWQ_ERR_INVALID_ARG;
    if (fp8 ? !(p.scale > 0.f && std::isfinite(p.scale)) : p.scale != 1.f) return AWQ_ERR_INVALID_ARG;
    return fp8 || aligned(p.data, 2) ? AWQ_OK : AWQ_ERR_MISALIGNED;
}

inline awq_status check_cache(const awq_kv_cache *c, int32_t dtype, int max_dim)
{
    if (!c) return AWQ_ERR_INVALID_ARG;
    const bool fp8 = c->dtype == AWQ_DTYPE_E4M3;
    if (!fp8 && c->dtype != dtype) return AWQ_ERR_INVALID_ARG;
    if (c->num_pages < 1 || c->page_size < 1 || c->num_heads < 1) return AWQ_ERR_INVALID_ARG;
    if (c->head_dim < 1 || c->head_dim > max_dim) return AWQ_ERR_UNSUPPORTED_SHAPE;
    awq_status r = check_plane(c->k, fp8);
    return r ? r : check_plane(c->v, fp8);
}

// The stride of a dimension of one is never used: 0, which every alignment
// allows.
inline awq_heads used_strides(const awq_heads &h, int32_t tokens, int32_t heads)
{
    return awq_heads{h.data, tokens > 1 ? h.token_stride : 0, heads > 1 ? h.head_stride : 0};
}
inline awq_kv_plane used_strides(const awq_kv_plane &p, const awq_kv_cache &c)
{
    return awq_kv_plane{p.data, c.num_pages > 1 ? p.page_stride : 0, c.page_size > 1 ? p.token_stride : 0,
                        c.num_heads > 1 ? p.head_stride : 0, p.scale};
}
inline awq_kv_cache used_strides(const awq_kv_cache &c)
{
    awq_kv_cache u = c;
    u.k = used_strides(c.k, c);
    u.v = used_strides(c.v, c);
    return u;
}

// Every address of the plane's rows is a multiple of `a` bytes.
inline bool plane_aligned(const awq_kv_plane &p, int64_t elem, int64_t a)
{
    return aligned(p.data, a) && p.page_stride * elem % a == 0 && p.token_stride * elem % a == 0 &&
           p.head_stride * elem % a == 0;
}
inline bool heads_aligned(const awq_heads &h, int64_t a)
{
    return aligned(h.data, a) && h.token_stride * 2 % a == 0 && h.head_stride * 2 % a == 0;
}

// The checks of awq_rope_append's arguments; its block of them (none where
// there are no tokens), and in `vec` the elements of an access.
inline awq_status rope_args(RopeArgs &a, int &vec, const awq_heads *q, const awq_heads *q_out, const awq_heads *k,
                            const awq_heads *v, const int32_t *positions, const float *cos_sin, int32_t max_positions,
                            int32_t rotary_dim, int32_t interleaved, const int64_t *slots, const awq_kv_cache *cache,
                            int32_t tokens, int32_t q_heads, int32_t dtype, int32_t *dev_status)
{
    awq_status r = check_dtype(dtype);
    if (r) return r;
    if (tokens < 0 || q_heads < 1 || max_positions < 1) return AWQ_ERR_INVALID_ARG;
    r = check_cache(cache, dtype, 1024);
    if (r) return r;
    if (rotary_dim < 0 || rotary_dim > cache->head_dim || rotary_dim % 2) return AWQ_ERR_UNSUPPORTED_SHAPE;
    // (a token's rows, and the turns of threads past them, are counted in 32 bits)
    if (static_cast<int64_t>(q_heads) + 2 * static_cast<int64_t>(cache->num_heads) > 0x7fffffff - 2047) return AWQ_ERR_UNSUPPORTED_SHAPE;
    if (tokens == 0) return AWQ_OK;
    for (const awq_heads *h : {q, q_out, k, v}) {
        r = check_heads(h);
        if (r) return r;
    }
    if (!positions || !slots || !dev_status || (rotary_dim && !cos_sin)) return AWQ_ERR_INVALID_ARG;
    if (!aligned(positions, 4) || !aligned(slots, 8) || !aligned(dev_status, 4) || !aligned(cos_sin, 16))
        return AWQ_ERR_MISALIGNED;
    const int64_t elem = cache->dtype == AWQ_DTYPE_E4M3 ? 1 : 2;
    const awq_kv_cache uc = used_strides(*cache);
    const awq_heads uq = used_strides(*q, tokens, q_heads), uo = used_strides(*q_out, tokens, q_heads),
                    uk = used_strides(*k, tokens, cache->num_heads), uv = used_strides(*v, tokens, cache->num_heads);
    // the widest access that every row, the head and the rotated part allow
    vec = 1;
    for (int n : {8, 4}) {
        const bool rows = heads_aligned(uq, 2 * n) && heads_aligned(uo, 2 * n) && heads_aligned(uk, 2 * n) &&
                          heads_aligned(uv, 2 * n) && plane_aligned(uc.k, elem, elem * n) &&
                          plane_aligned(uc.v, elem, elem * n);
        if (rows && cache->head_dim % n == 0 && (interleaved ? rotary_dim : rotary_dim / 2) % n == 0) {
            vec = n;
            break;
        }
    }
    a = RopeArgs{uq, uo, uk, uv, positions, cos_sin, slots, uc, dev_status, max_positions,
                 rotary_dim, interleaved != 0, tokens, q_heads};
    return AWQ_OK;
}

}  // namespace awq
