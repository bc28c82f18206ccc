// Host side of the C ABI declared in include/awq_decoder.h: argument checks
// (nothing is launched on a host-visible error) and the choice of the access
// width.
#include <algorithm>
#include <cmath>

#include "awq_decoder_checks.cuh"

namespace awq {

namespace {

constexpr uint64_t kGemmTimeoutNs = 1000000000ull;     // 1 s per device wait

}  // namespace

}  // namespace awq

using namespace awq;

extern "C" {

awq_status awq_add_rmsnorm(const void *x, int64_t ldx, const void *residual, int64_t ldr, void *residual_out,
                           int64_t ldro, const void *weight, float eps, void *out, int64_t ldo, uint8_t *out_q,
                           int64_t ldq, float *out_scales, int32_t rows, int32_t hidden, int32_t dtype, void *stream)
{
    awq_status r = check_dtype(dtype);
    if (r) return r;
    if (rows < 0 || !(eps >= 0.f) || !std::isfinite(eps)) return AWQ_ERR_INVALID_ARG;
    if (hidden < 1 || hidden > AWQ_NORM_MAX_HIDDEN) return AWQ_ERR_UNSUPPORTED_SHAPE;
    if (rows == 0) return AWQ_OK;
    if (!x || !weight || (!out && !out_q) || !out_q != !out_scales) return AWQ_ERR_INVALID_ARG;
    if (ldx < hidden || (residual && ldr < hidden) || (residual_out && ldro < hidden) || (out && ldo < hidden) ||
        (out_q && ldq < hidden))
        return AWQ_ERR_INVALID_ARG;
    if (!aligned(x, 2) || !aligned(residual, 2) || !aligned(residual_out, 2) || !aligned(weight, 2) ||
        !aligned(out, 2) || !aligned(out_scales, 4))
        return AWQ_ERR_MISALIGNED;
    if (rows == 1) ldx = ldr = ldro = ldo = ldq = 0;    // the stride of a single row is not used
    const bool wide = hidden % 8 == 0 && aligned(weight, 16) && aligned_rows(x, ldx, 2, 16) &&
                      aligned_rows(residual, ldr, 2, 16) && aligned_rows(residual_out, ldro, 2, 16) &&
                      aligned_rows(out, ldo, 2, 16) && aligned_rows(out_q, ldq, 1, 8);
    const int sms = current_sm_count();
    if (sms <= 0) return AWQ_ERR_CUDA;
    const NormArgs a{x, residual, weight, residual_out, out, out_q, out_scales, ldx, ldr, ldro, ldo, ldq, eps, rows, hidden};
    return launch_norm(a, dtype, wide, sms, static_cast<cudaStream_t>(stream));
}

awq_status awq_quantize_fp8(const void *x, int64_t ldx, uint8_t *q, int64_t ldq, float *scales, int32_t rows,
                            int32_t cols, int32_t dtype, void *stream)
{
    awq_status r = check_dtype(dtype);
    if (r) return r;
    if (rows < 0 || cols < 1) return AWQ_ERR_INVALID_ARG;
    if (cols > 1 << 30) return AWQ_ERR_UNSUPPORTED_SHAPE;    // columns are counted in 32 bits
    if (rows == 0) return AWQ_OK;
    if (!x || !q || !scales || ldx < cols || ldq < cols) return AWQ_ERR_INVALID_ARG;
    if (!aligned(x, 2) || !aligned(scales, 4)) return AWQ_ERR_MISALIGNED;
    if (rows == 1) ldx = ldq = 0;                       // the stride of a single row is not used
    const bool wide = cols % 8 == 0 && aligned_rows(x, ldx, 2, 16) && aligned_rows(q, ldq, 1, 8);
    const int sms = current_sm_count();
    if (sms <= 0) return AWQ_ERR_CUDA;
    return launch_quantize(QuantArgs{x, q, scales, ldx, ldq, rows, cols}, dtype, wide, sms,
                           static_cast<cudaStream_t>(stream));
}

awq_status awq_rope_append(const awq_heads *q, const awq_heads *q_out, const awq_heads *k, const awq_heads *v,
                           const int32_t *positions, const float *cos_sin, int32_t max_positions, int32_t rotary_dim,
                           int32_t interleaved, const int64_t *slots, const awq_kv_cache *cache, int32_t tokens,
                           int32_t q_heads, int32_t dtype, int32_t *dev_status, void *stream)
{
    RopeArgs a{};
    int vec = 1;
    const awq_status r = rope_args(a, vec, q, q_out, k, v, positions, cos_sin, max_positions, rotary_dim, interleaved, slots,
                                   cache, tokens, q_heads, dtype, dev_status);
    if (r || tokens == 0) return r;
    const int sms = current_sm_count();
    if (sms <= 0) return AWQ_ERR_CUDA;
    return launch_rope(a, dtype, vec, sms, static_cast<cudaStream_t>(stream));
}

size_t awq_paged_attention_workspace_bytes(int32_t head_dim)
{
    if (head_dim < 8 || head_dim > AWQ_ATTN_MAX_HEAD_DIM || head_dim % 8) return 0;
    return attn_workspace_bytes(head_dim);
}

awq_status awq_paged_attention(const awq_heads *q, const awq_kv_cache *cache, const int32_t *page_table,
                               int64_t table_stride, int32_t max_pages, const int32_t *seq_lens, int32_t batch,
                               int32_t q_heads, int32_t dtype, float scale, const awq_heads *out, float *lse,
                               void *workspace, size_t ws_bytes, int32_t *dev_status, void *stream)
{
    awq_status r = check_dtype(dtype);
    if (r) return r;
    if (batch < 0 || q_heads < 1 || max_pages < 1 || !std::isfinite(scale)) return AWQ_ERR_INVALID_ARG;
    r = check_cache(cache, dtype, AWQ_ATTN_MAX_HEAD_DIM);
    if (r) return r;
    const int64_t elem = cache->dtype == AWQ_DTYPE_E4M3 ? 1 : 2;
    if (q_heads % cache->num_heads || cache->head_dim * elem % 16) return AWQ_ERR_UNSUPPORTED_SHAPE;
    if (batch == 0) return AWQ_OK;
    for (const awq_heads *h : {q, out}) {
        r = check_heads(h);
        if (r) return r;
    }
    if (!page_table || !seq_lens || !workspace || !dev_status || table_stride < max_pages) return AWQ_ERR_INVALID_ARG;
    const awq_kv_cache uc = used_strides(*cache);
    const awq_heads uq = used_strides(*q, batch, q_heads), uo = used_strides(*out, batch, q_heads);
    if (!heads_aligned(uq, 16) || !heads_aligned(uo, 16) || !plane_aligned(uc.k, elem, 16) || !plane_aligned(uc.v, elem, 16) || !aligned(page_table, 4) || !aligned(seq_lens, 4) || !aligned(lse, 4) ||
        !aligned(workspace, 256) || !aligned(dev_status, 4))
        return AWQ_ERR_MISALIGNED;
    if (ws_bytes < attn_workspace_bytes(cache->head_dim)) return AWQ_ERR_WORKSPACE_TOO_SMALL;
    AttnArgs a{};
    a.q = uq;
    a.out = uo;
    a.cache = uc;
    a.page_table = page_table;
    a.seq_lens = seq_lens;
    a.lse = lse;
    a.counters = static_cast<int32_t *>(workspace);
    a.parts = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + kAttnCounterBytes);
    a.status = dev_status;
    a.table_stride = table_stride;
    a.max_pages = max_pages;
    a.batch = batch;
    a.q_heads = q_heads;
    a.group = q_heads / cache->num_heads;
    a.row_tiles = (a.group + kAttnRows - 1) / kAttnRows;
    // exact for every token below 2^31: with 2^shift >= page_size, magic =
    // floor(2^(31 + shift) / page_size) + 1 exceeds the quotient by at most 1
    while ((1ll << a.page_shift) < cache->page_size) ++a.page_shift;
    a.page_magic = static_cast<uint32_t>((1ull << (31 + a.page_shift)) / cache->page_size + 1);
    a.same_strides = uc.k.page_stride == uc.v.page_stride && uc.k.token_stride == uc.v.token_stride &&
                     uc.k.head_stride == uc.v.head_stride;
    a.scale = scale;
    // units (of at least 16 tokens) are numbered in 32 bits
    const int64_t most = static_cast<int64_t>(max_pages) * cache->page_size, units = std::min<int64_t>(most, 0x7fffffc0) / 16 + 1;
    if (units > 0x7fffffff / batch || units * batch > 0x7fffffff / cache->num_heads / a.row_tiles) return AWQ_ERR_UNSUPPORTED_SHAPE;
    const int sms = current_sm_count();
    if (sms <= 0) return AWQ_ERR_CUDA;
    return launch_attention(a, dtype, sms, static_cast<cudaStream_t>(stream));
}

awq_status awq_fp8_gemm(const uint8_t *a, int64_t lda, const float *a_scales, const uint8_t *b, int64_t ldb,
                        const float *b_scales, void *out, int64_t ldo, int32_t M, int32_t N, int32_t K, int32_t dtype,
                        int32_t *dev_status, void *stream)
{
    awq_status r = check_dtype(dtype);
    if (r) return r;
    if (M < 0 || N < 0 || K < 1) return AWQ_ERR_INVALID_ARG;
    if (M > 1 << 30 || N > 1 << 30 || K > 1 << 30) return AWQ_ERR_UNSUPPORTED_SHAPE;    // counted in 32 bits
    if (M == 0 || N == 0) return AWQ_OK;
    if (!a || !a_scales || !b || !b_scales || !out || !dev_status || lda < K || ldb < K || ldo < N)
        return AWQ_ERR_INVALID_ARG;
    // the stride of a single row is never used
    if (M == 1) lda = (lda + 15) / 16 * 16;
    if (N == 1) ldb = (ldb + 15) / 16 * 16;
    if (!aligned_rows(a, lda, 1, 16) || !aligned_rows(b, ldb, 1, 16) || !aligned(a_scales, 4) || !aligned(b_scales, 4) ||
        !aligned(out, 2) || !aligned(dev_status, 4))
        return AWQ_ERR_MISALIGNED;
    const int sms = current_sm_count();
    if (sms <= 0) return AWQ_ERR_CUDA;
    const GemmArgs g{a_scales, b_scales, out, ldo, dev_status, M, N, K, kGemmTimeoutNs};
    return launch_fp8_gemm(g, a, lda, b, ldb, dtype, sms, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
