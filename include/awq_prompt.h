/*
 * awq_prompt.h -- C ABI of the operators that take a prompt through the
 * attention half of a decoder layer: causal attention over packed prompts, the
 * attention of a chunk of new tokens over the paged cache, and the norm of each
 * head of q and k with the rotation and the append to that cache. Same library
 * (libawqmoe.so), types, conventions and errors as awq_decoder.h, whose calls
 * they stand beside: awq_paged_attention decodes from the cache that they fill.
 */
#ifndef AWQ_PROMPT_H
#define AWQ_PROMPT_H

#include "awq_decoder.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * awq_prompt_attention -- causal attention over whole prompts, packed one
 * behind the other.
 * Sequence b has the rows cu_seqlens[b] .. cu_seqlens[b + 1] - 1 of q, k, v and
 * out. Query head h reads KV head h / (q_heads / kv_heads); row i of a sequence
 * sees its rows 0 .. i:
 *   s[i][j] = scale * (q[i] . k[j]),  j <= i
 *   out[i] = sum_j softmax(s[i])[j] v[j],  lse[i] = log(sum_j exp(s[i][j]))
 * scale is any finite number; scores past fp32's range count as infinite.
 * What a row does not see does not reach it, NaN and
 * infinities among it; a value of v that is not finite leaves its element of out
 * not finite in every row that sees it. A row whose scores are all -infinity has out =
 * 0 and lse = -infinity. Held in fewer than 32 bits: a weight, which enters the
 * product with v in the type of q (fp16: off by at most 2^-11 of it or 2^-32 of
 * the largest one; bf16: 2^-8 of it); the sum that it is divided by takes it in fp32.
 * Rows past cu_seqlens[batch] (of `tokens`) are left as they were. cu_seqlens
 * that fall, or leave [0, tokens], set AWQ_ERR_BAD_INDEX; nothing outside the
 * buffers is touched, and the sequences that they bound are undefined.
 * q, out: 16-bit [tokens][q_heads][head_dim]; k, v: [tokens][kv_heads]
 * [head_dim], all 16-byte aligned with strides that are multiples of 16 bytes
 * (k's and v's below 2^39 elements, and not 0 between tokens if there are more
 * than one); cu_seqlens i32[batch + 1]; lse f32[tokens][q_heads], dense, or
 * NULL; outputs overlap no input.
 * batch, tokens >= 0 (0 launches nothing); q_heads a multiple of kv_heads;
 * head_dim a multiple of 8 up to AWQ_ATTN_MAX_HEAD_DIM. Sizes that the 32-bit
 * rows and 64-bit costs of the split cannot hold are refused: with G = q_heads /
 * kv_heads, tokens * G has to be at most 2^31 - 256, and with the longest
 * context L (here: tokens) and u = G * (L + tokens + 640) + 512, both u * (L /
 * 128 + 1) and u * (tokens * G / 120 + 1) * kv_heads * batch at most 4 * 10^18.
 * Work is split over the rows, and over the keys where that alone does not fill
 * the card, by the lengths on the device; the parts are joined in the same
 * launch, which is cooperative (all blocks at once on the multiprocessors).
 * workspace: at least awq_prompt_attention_workspace_bytes() of device scratch,
 * 256-byte aligned, zero-filled once before its first use; every call leaves it
 * ready for the next one on the same device (but for one that ended in
 * AWQ_ERR_DEVICE_TIMEOUT, which a block sets that has waited for the others a second longer
 * than it worked itself: then zero it again). It must not be used by two calls
 * that can run at the same time, nor by calls other than this one and
 * awq_chunk_attention.
 */
AWQ_API awq_status awq_prompt_attention(const awq_heads *q, const awq_heads *k, const awq_heads *v,
                                        const int32_t *cu_seqlens, int32_t batch, int32_t tokens,
                                        int32_t q_heads, int32_t kv_heads, int32_t head_dim, int32_t dtype,
                                        float scale, const awq_heads *out, float *lse, void *workspace,
                                        size_t ws_bytes, int32_t *dev_status, void *stream);

/* Workspace bytes of awq_prompt_attention and awq_chunk_attention at this head
 * size, for any batch, lengths and heads (0 for a head size that they do not
 * take). Host-only, no CUDA call. */
AWQ_API size_t awq_prompt_attention_workspace_bytes(int32_t head_dim);

/*
 * awq_chunk_attention -- attention of a chunk of new tokens per sequence over
 * the paged cache: the next part of a long prompt, drafted tokens to be
 * verified, single tokens, or a batch that mixes them. (For a batch of single tokens alone
 * awq_paged_attention is faster and rounds a weight less: it multiplies it as two terms.)
 * Sequence b has n = cu_seqlens[b + 1] - cu_seqlens[b] new tokens, the rows
 * from cu_seqlens[b] on of q and out, and L = seq_lens[b] tokens in the cache,
 * the new ones among them (appended before the call). Its new token i is at
 * position p = L - n + i and sees the cached tokens 0 .. p; where p < 0 it sees
 * none: out = 0, lse = -infinity. Page table, cache and the formulas are as in
 * awq_paged_attention and awq_prompt_attention; e4m3 values enter the products
 * as fp16 (exact), a weight over an e4m3 cache as fp16, and a bf16 query over
 * it as fp16 with its row's power of two taken out (off by at most 2^-24 of its
 * row's largest element).
 * Pages past a sequence's last token are not read, and what the places after it hold does
 * not reach the output.
 * A length outside [0, max_pages * page_size] or above 2^31 - 256, a page outside [0, num_pages)
 * that is needed, and cu_seqlens as in awq_prompt_attention set
 * AWQ_ERR_BAD_INDEX; that sequence's output is then undefined.
 * page_table i32[batch][max_pages], row stride table_stride; seq_lens
 * i32[batch]; q, out, cu_seqlens, lse, workspace and limits as in
 * awq_prompt_attention, with L = max_pages * page_size; head_dim a multiple of
 * 16 for an e4m3 cache; both planes 16-byte aligned with strides that are
 * multiples of 16 bytes, below 2^39 elements, and not 0 between tokens if a
 * page holds more than one.
 * The cache is copied in boxes of as many tokens as the largest power of two up
 * to 128 that divides page_size: pages of an odd size are read token by token.
 */
AWQ_API awq_status awq_chunk_attention(const awq_heads *q, const awq_kv_cache *cache,
                                       const int32_t *page_table, int64_t table_stride, int32_t max_pages,
                                       const int32_t *cu_seqlens, const int32_t *seq_lens, int32_t batch,
                                       int32_t tokens, int32_t q_heads, int32_t dtype, float scale,
                                       const awq_heads *out, float *lse, void *workspace, size_t ws_bytes,
                                       int32_t *dev_status, void *stream);

/*
 * awq_qk_norm_rope_append -- awq_rope_append with an RMS norm of each head of
 * q and k in front of the rotation, in the same pass:
 *   y[d] = x[d] / sqrt(mean over the head of x^2 + eps) * weight[d]
 * in fp32; y is rotated (and copied past rotary_dim) without being rounded in
 * between. v is appended as it is. The squares are added in fp32: a head whose
 * sum passes its range (finite bf16 values can) has y = 0, and squares below its
 * range count as 0. A weight of k divided by its e4m3 plane's scale has to stay in that range, too.
 * q_weight, k_weight: 16-bit [head_dim] of the activations' type, 2-byte
 * aligned; eps >= 0 and finite. All else as in awq_rope_append.
 */
AWQ_API awq_status awq_qk_norm_rope_append(const awq_heads *q, const awq_heads *q_out, const awq_heads *k,
                                           const awq_heads *v, const void *q_weight, const void *k_weight,
                                           float eps, const int32_t *positions, const float *cos_sin,
                                           int32_t max_positions, int32_t rotary_dim, int32_t interleaved,
                                           const int64_t *slots, const awq_kv_cache *cache, int32_t tokens,
                                           int32_t q_heads, int32_t dtype, int32_t *dev_status, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* AWQ_PROMPT_H */
