// Host side of the C ABI declared in include/awq_prompt.h: argument checks
// (nothing is launched on a host-visible error) and the choice of the kernel.
#include <algorithm>
#include <cfloat>
#include <climits>
#include <cmath>

#include "awq_decoder_checks.cuh"
#include "awq_prompt_kernels.cuh"

namespace awq {

namespace {

constexpr uint64_t kChunkTimeoutNs = 1000000000ull;    // 1 s and a block's own time per wait for another block

// What both attention calls have in common, behind their own checks: `a` has
// q, out, the planes, their index arrays, sizes and max_len.
awq_status chunk_call(ChunkArgs &a, int32_t dtype, float scale, void *workspace, size_t ws_bytes, void *stream)
{
    const int dim = a.cache.head_dim;
    const bool fp8 = a.cache.dtype == AWQ_DTYPE_E4M3;
    const int64_t elem = fp8 ? 1 : 2;
    if (!heads_aligned(a.q, 16) || !heads_aligned(a.out, 16) || !plane_aligned(a.cache.k, elem, 16) ||
        !plane_aligned(a.cache.v, elem, 16) || !aligned(a.cu_seqlens, 4) || !aligned(a.seq_lens, 4) ||
        !aligned(a.page_table, 4) || !aligned(a.lse, 4) || !aligned(workspace, 256) || !aligned(a.status, 4))
        return AWQ_ERR_MISALIGNED;
    // Units are of whole tokens where they can be, so that Q comes in boxes of a
    // tensor map: of the numbers of tokens that nearly fill one, that with the
    // fewest boxes of up to 64 rows.
    const int most_rows = chunk_rows(attn_padded_dim(dim));
    a.unit_rows = most_rows;
    const int64_t far = 1ll << 39;               // elements: a tensor map's strides end at 2^40 bytes
    if (a.group <= most_rows && (a.q_heads == 1 || (a.q.head_stride > 0 && a.q.head_stride < far)) &&
        (a.tokens == 1 || (a.q.token_stride > 0 && a.q.token_stride < far))) {
        int best = INT_MAX;
        for (int n = most_rows / a.group, least = n - n / 32; n >= least; --n) {
            int d = std::max(1, 64 / a.group);
            while (n % d) --d;
            if (n / d < best) {
                best = n / d;
                a.unit_rows = n * a.group;
                a.q_box = d;
            }
        }
    }
    a.narrow_cost = fp8 ? kChunkNarrowCost : 0;
    // rows of a KV head are counted in 32 bits, costs (and products of them) in 64
    const double G = a.group, rows = static_cast<double>(a.tokens) * G, R = a.unit_rows;
    if (rows > 0x7fffff00) return AWQ_ERR_UNSUPPORTED_SHAPE;
    const double unit = G * (static_cast<double>(a.max_len) + kChunkUnitCost + kChunkNarrowCost + a.tokens) + 2 * R;
    // (a cost times tiles; the sum of all costs, units of as few as 65 rows, and a block's share more)
    if (unit * (a.max_len / 128 + 1) > 4.6e18 || unit * (rows / R + 1) * a.cache.num_heads * a.batch > 8.5e18)
        return AWQ_ERR_UNSUPPORTED_SHAPE;
    if (ws_bytes < chunk_workspace_bytes(dim)) return AWQ_ERR_WORKSPACE_TOO_SMALL;
    // copies are boxes of keys that lie in one page wherever they begin
    a.box = kChunkKeys;
    while (a.page_table && a.cache.page_size % a.box) a.box /= 2;
    const int64_t place = a.page_table ? a.cache.page_size : a.tokens;
    for (int i = 0; i < 2; ++i) {
        const awq_kv_plane &p = i ? a.cache.v : a.cache.k;
        if ((place > 1 && p.token_stride == 0) || p.token_stride >= far || p.head_stride >= far || p.page_stride >= far)
            return AWQ_ERR_UNSUPPORTED_SHAPE;
        a.head_step[i] = p.head_stride ? 1 : 0;
        a.page_step[i] = p.page_stride ? 1 : 0;
    }
    a.counters = static_cast<int32_t *>(workspace);
    a.parts = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + kChunkCounterBytes);
    a.negative = scale < 0.f;
    a.factor = static_cast<float>(std::min(std::fabs(static_cast<double>(scale)) * 1.4426950408889634 * a.cache.k.scale,
                                           static_cast<double>(FLT_MAX)));
    a.timeout_ns = kChunkTimeoutNs;
    const int sms = current_sm_count();
    if (sms <= 0) return AWQ_ERR_CUDA;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dtype == AWQ_DTYPE_F16) return fp8 ? launch_chunk_f16_e4m3(a, sms, st) : launch_chunk_f16(a, sms, st);
    return fp8 ? launch_chunk_bf16_e4m3(a, sms, st) : launch_chunk_bf16(a, sms, st);
}

}  // namespace

}  // namespace awq

using namespace awq;

extern "C" {

size_t awq_prompt_attention_workspace_bytes(int32_t head_dim)
{
    if (head_dim < 8 || head_dim > AWQ_ATTN_MAX_HEAD_DIM || head_dim % 8) return 0;
    return chunk_workspace_bytes(head_dim);
}

awq_status awq_prompt_attention(const awq_heads *q, const awq_heads *k, const awq_heads *v, const int32_t *cu_seqlens,
                                int32_t batch, int32_t tokens, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                                int32_t dtype, float scale, const awq_heads *out, float *lse, void *workspace,
                                size_t ws_bytes, int32_t *dev_status, void *stream)
{
    awq_status r = check_dtype(dtype);
    if (r) return r;
    if (batch < 0 || tokens < 0 || q_heads < 1 || kv_heads < 1 || !std::isfinite(scale)) return AWQ_ERR_INVALID_ARG;
    if (head_dim < 8 || head_dim > AWQ_ATTN_MAX_HEAD_DIM || head_dim % 8 || q_heads % kv_heads) return AWQ_ERR_UNSUPPORTED_SHAPE;
    if (batch == 0 || tokens == 0) return AWQ_OK;
    for (const awq_heads *h : {q, k, v, out}) {
        r = check_heads(h);
        if (r) return r;
    }
    if (!cu_seqlens || !workspace || !dev_status) return AWQ_ERR_INVALID_ARG;
    ChunkArgs a{};
    a.q = used_strides(*q, tokens, q_heads);
    a.out = used_strides(*out, tokens, q_heads);
    const awq_heads uk = used_strides(*k, tokens, kv_heads), uv = used_strides(*v, tokens, kv_heads);
    a.cache.k = awq_kv_plane{uk.data, 0, uk.token_stride, uk.head_stride, 1.f};
    a.cache.v = awq_kv_plane{uv.data, 0, uv.token_stride, uv.head_stride, 1.f};
    a.cache.dtype = dtype;
    a.cache.num_heads = kv_heads;
    a.cache.head_dim = head_dim;
    a.cu_seqlens = cu_seqlens;
    a.lse = lse;
    a.status = dev_status;
    a.max_len = tokens;
    a.batch = batch;
    a.tokens = tokens;
    a.q_heads = q_heads;
    a.group = q_heads / kv_heads;
    return chunk_call(a, dtype, scale, workspace, ws_bytes, stream);
}

awq_status awq_chunk_attention(const awq_heads *q, const awq_kv_cache *cache, const int32_t *page_table,
                               int64_t table_stride, int32_t max_pages, const int32_t *cu_seqlens,
                               const int32_t *seq_lens, int32_t batch, int32_t tokens, int32_t q_heads, int32_t dtype,
                               float scale, const awq_heads *out, float *lse, void *workspace, size_t ws_bytes,
                               int32_t *dev_status, void *stream)
{
    awq_status r = check_dtype(dtype);
    if (r) return r;
    if (batch < 0 || tokens < 0 || q_heads < 1 || max_pages < 1 || !std::isfinite(scale)) return AWQ_ERR_INVALID_ARG;
    r = check_cache(cache, dtype, AWQ_ATTN_MAX_HEAD_DIM);
    if (r) return r;
    const int64_t elem = cache->dtype == AWQ_DTYPE_E4M3 ? 1 : 2;
    if (q_heads % cache->num_heads || cache->head_dim * elem % 16) return AWQ_ERR_UNSUPPORTED_SHAPE;
    if (batch == 0 || tokens == 0) return AWQ_OK;
    for (const awq_heads *h : {q, out}) {
        r = check_heads(h);
        if (r) return r;
    }
    if (!page_table || !cu_seqlens || !seq_lens || !workspace || !dev_status || table_stride < max_pages) return AWQ_ERR_INVALID_ARG;
    ChunkArgs a{};
    a.q = used_strides(*q, tokens, q_heads);
    a.out = used_strides(*out, tokens, q_heads);
    a.cache = used_strides(*cache);
    a.page_table = page_table;
    a.table_stride = table_stride;
    a.cu_seqlens = cu_seqlens;
    a.seq_lens = seq_lens;
    a.lse = lse;
    a.status = dev_status;
    // exact for every token below 2^31: with 2^shift >= page_size, magic =
    // floor(2^(31 + shift) / page_size) + 1 exceeds the quotient by at most 1
    while ((1ll << a.page_shift) < cache->page_size) ++a.page_shift;
    a.page_magic = static_cast<uint32_t>((1ull << (31 + a.page_shift)) / cache->page_size + 1);
    a.max_len = static_cast<int32_t>(std::min<int64_t>(static_cast<int64_t>(max_pages) * cache->page_size, 0x7fffff00));
    a.batch = batch;
    a.tokens = tokens;
    a.q_heads = q_heads;
    a.group = q_heads / cache->num_heads;
    return chunk_call(a, dtype, scale, workspace, ws_bytes, stream);
}

awq_status awq_qk_norm_rope_append(const awq_heads *q, const awq_heads *q_out, const awq_heads *k, const awq_heads *v,
                                   const void *q_weight, const void *k_weight, float eps, const int32_t *positions,
                                   const float *cos_sin, int32_t max_positions, int32_t rotary_dim, int32_t interleaved,
                                   const int64_t *slots, const awq_kv_cache *cache, int32_t tokens, int32_t q_heads,
                                   int32_t dtype, int32_t *dev_status, void *stream)
{
    if (!(eps >= 0.f) || !std::isfinite(eps)) return AWQ_ERR_INVALID_ARG;
    HeadNormArgs a{};
    int vec = 1;
    awq_status r = rope_args(a.rope, vec, q, q_out, k, v, positions, cos_sin, max_positions, rotary_dim, interleaved, slots,
                             cache, tokens, q_heads, dtype, dev_status);
    if (r || tokens == 0) return r;
    if (!q_weight || !k_weight) return AWQ_ERR_INVALID_ARG;
    if (!aligned(q_weight, 2) || !aligned(k_weight, 2)) return AWQ_ERR_MISALIGNED;
    while (vec > 1 && (!aligned(q_weight, 2 * vec) || !aligned(k_weight, 2 * vec))) vec = vec == 8 ? 4 : 1;
    a.q_weight = q_weight;
    a.k_weight = k_weight;
    a.eps = eps;
    const int sms = current_sm_count();
    if (sms <= 0) return AWQ_ERR_CUDA;
    return launch_head_norm(a, dtype, vec, sms, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
