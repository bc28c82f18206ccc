/*
 * awq_decoder.h -- C ABI of the decoder layer's operators around the expert
 * stage of awq_moe.h: the norm before a product, the 8-bit product itself,
 * the rotation of q and k with the append to a paged cache, and the attention
 * of one new token over that cache. Same library (libawqmoe.so).
 *
 * The conventions are those of awq_moe.h: every pointer is a DEVICE pointer
 * unless stated otherwise, structs are read on the host during the call, the
 * caller owns all memory and the library allocates nothing; work is enqueued
 * asynchronously on `stream` (NULL: the legacy default stream) and may be
 * captured in a CUDA graph; what the host can see to be wrong is rejected
 * with a non-zero awq_status before anything is launched; what only the data
 * can show goes to `dev_status` (device int32, zeroed by the caller, the
 * first code raised is kept): an index outside its array gives
 * AWQ_ERR_BAD_INDEX, a device wait that ran out AWQ_ERR_DEVICE_TIMEOUT.
 * Every call is deterministic: the same inputs give the same bits.
 *
 * Types (awq_dtype). Activations are fp16 or bf16 (`dtype`), held as 16-bit
 * words; sums, softmax statistics and norms are held in fp32 and every output
 * element is rounded once. e4m3 is FP8 E4M3 with a largest value of 448 and
 * no infinity (codes 0x7F and 0xFF are NaN); conversions to it round to
 * nearest even and saturate at +-448 (NaN stays NaN).
 */
#ifndef AWQ_DECODER_H
#define AWQ_DECODER_H

#include "awq_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    AWQ_DTYPE_F16 = 0,
    AWQ_DTYPE_BF16 = 1,
    AWQ_DTYPE_E4M3 = 2
} awq_dtype;

/* Columns that share one activation scale; rows x columns of a weight that
 * share one weight scale. */
#define AWQ_FP8_BLOCK 128
/* A group's largest magnitude is taken as at least this when its scale is
 * formed (a group of zeros has the scale 1e-12 / 448 and codes 0). */
#define AWQ_FP8_MIN_AMAX 1e-12f
/* Largest row awq_add_rmsnorm takes (a row lives in one block's registers). */
#define AWQ_NORM_MAX_HIDDEN 32768
/* Largest head size of awq_paged_attention. */
#define AWQ_ATTN_MAX_HEAD_DIM 256

/*
 * awq_add_rmsnorm -- the norm before a product, with the residual's addition
 * and an 8-bit output.
 *   r = x + residual (x alone where residual is NULL), in fp32
 *   y[c] = r[c] / sqrt(mean(r^2) + eps) * weight[c], in fp32
 *   residual_out = r;  out = y;  (out_q, out_scales) = y as e4m3 in groups:
 *   per row and group of 128 columns (the last one may be shorter)
 *     out_scales = max(amax, AWQ_FP8_MIN_AMAX) / 448,
 *     out_q = e4m3(y * (448 / max(amax, AWQ_FP8_MIN_AMAX)))
 * y is taken from r before r is rounded for residual_out, and out_q from y
 * before y is rounded for out. A row whose sum of squares passes fp32's range
 * (finite bf16 values can) has y = 0. A NaN in a group is left out of its amax and
 * stays NaN in out_q; an infinity makes its group's scale infinite.
 * x, residual, residual_out, out: 16-bit [rows][hidden], row strides ldx, ldr,
 * ldro, ldo in elements (each >= hidden; not used for a single row). weight: 16-bit [hidden]. out_q:
 * e4m3 [rows][hidden], row stride ldq. out_scales: f32[rows][ceil(hidden /
 * 128)], dense. residual, residual_out, out and the pair out_q/out_scales may
 * each be NULL, but out or out_q must be given. residual_out may be residual
 * or x, and out may be x, at the same address and stride; other overlaps of
 * inputs and outputs are not allowed.
 * rows >= 0 (0 launches nothing), hidden 1..AWQ_NORM_MAX_HIDDEN, any size;
 * 16-bit pointers 2-byte aligned, out_scales and weight by their type. Rows
 * whose addresses and strides are all multiples of 16 bytes (8 for out_q) and
 * hidden % 8 == 0 take 16-byte accesses.
 */
AWQ_API awq_status awq_add_rmsnorm(const void *x, int64_t ldx, const void *residual, int64_t ldr,
                                   void *residual_out, int64_t ldro, const void *weight, float eps,
                                   void *out, int64_t ldo, uint8_t *out_q, int64_t ldq,
                                   float *out_scales, int32_t rows, int32_t hidden, int32_t dtype,
                                   void *stream);

/*
 * awq_quantize_fp8 -- 16-bit rows to e4m3 with a scale per row and group of
 * 128 columns: the quantisation of awq_add_rmsnorm without the norm (for the
 * operand of a product that no norm precedes). x: 16-bit [rows][cols], row
 * stride ldx; q: e4m3 [rows][cols], row stride ldq; scales: f32[rows][ceil(
 * cols / 128)], dense. rows >= 0 (0 launches nothing), cols 1..2^30.
 */
AWQ_API awq_status awq_quantize_fp8(const void *x, int64_t ldx, uint8_t *q, int64_t ldq, float *scales,
                                    int32_t rows, int32_t cols, int32_t dtype, void *stream);

/* Vectors of one head each, [tokens][heads][head_dim]: element (t, h, d) is
 * data[t * token_stride + h * head_stride + d]. Strides in elements; that of a
 * dimension of one is not used. */
typedef struct {
    void *data;
    int64_t token_stride;
    int64_t head_stride;
} awq_heads;

/* One plane (K or V) of a paged cache: element (page, i, h, d) of the page's
 * i-th token is data[page * page_stride + i * token_stride + h * head_stride
 * + d], so that pages of [page_size][heads][dim] and of [heads][page_size]
 * [dim] are both described. Strides in elements; that of a dimension of one is
 * not used. In an e4m3 cache the stored value stands for value * scale; in a
 * 16-bit cache scale must be 1. */
typedef struct {
    void *data;
    int64_t page_stride;
    int64_t token_stride;
    int64_t head_stride;
    float scale;
} awq_kv_plane;

typedef struct {
    awq_kv_plane k, v;
    int32_t dtype;      /* AWQ_DTYPE_E4M3, or the activations' type */
    int32_t num_pages;
    int32_t page_size;  /* tokens of a page, >= 1 */
    int32_t num_heads;  /* KV heads */
    int32_t head_dim;
} awq_kv_cache;

/*
 * awq_rope_append -- rotation of q and k by position, and the append of k and
 * v to the paged cache.
 * Token t of the call has position p = positions[t] and goes to slot
 * slots[t]: page slots[t] / page_size, place slots[t] % page_size. Each head's
 * first rotary_dim elements are rotated in pairs, the rest is copied:
 *   (a, b) -> (a cos - b sin, b cos + a sin),
 *   cos = cos_sin[p][i], sin = cos_sin[p][rotary_dim / 2 + i];
 * pair i is elements (i, i + rotary_dim / 2), or (2i, 2i + 1) where
 * `interleaved` is not 0. Products in fp32, one rounding. q goes to q_out
 * (which may be q at the same strides), k (rotated) and v to the cache: in
 * its 16-bit type, or as e4m3(value * (1 / scale)).
 * A negative slot leaves the cache as it is (a padded batch's unused token);
 * its q is still rotated. A position outside [0, max_positions) or a slot
 * past the cache sets AWQ_ERR_BAD_INDEX and nothing is written for that
 * token. Two tokens of one call must not have the same slot.
 * positions i32[tokens]; cos_sin f32[max_positions][rotary_dim], dense,
 * 16-byte aligned; slots i64[tokens]; q, q_out [tokens][q_heads][head_dim],
 * k, v [tokens][cache->num_heads][head_dim]. tokens >= 0 (0 launches
 * nothing); q_heads >= 1; head_dim 1..1024; rotary_dim even, 0..head_dim.
 */
AWQ_API awq_status awq_rope_append(const awq_heads *q, const awq_heads *q_out, const awq_heads *k,
                                   const awq_heads *v, const int32_t *positions, const float *cos_sin,
                                   int32_t max_positions, int32_t rotary_dim, int32_t interleaved,
                                   const int64_t *slots, const awq_kv_cache *cache, int32_t tokens,
                                   int32_t q_heads, int32_t dtype, int32_t *dev_status, void *stream);

/*
 * awq_paged_attention -- attention of one new token per sequence over the
 * paged cache.
 * Sequence b has n = seq_lens[b] tokens in the cache (its new one among
 * them); token j is at place j % page_size of page page_table[b][j /
 * page_size]. Query head h reads KV head h / (q_heads / num_heads):
 *   s[j] = scale * (q . k[j]),  out = sum_j softmax(s)[j] v[j],
 *   lse = log(sum_j exp(s[j]))
 * k and v as the values the cache's codes stand for; scale is any finite
 * number. n = 0 gives out = 0 and lse = -infinity. A value of v that is not
 * finite makes its element of out NaN or infinite, which of the two is not
 * defined (a weight is multiplied as two terms, the second of any sign or 0);
 * other elements and lse do not change. Held in fewer than 32 bits: a weight, in
 * two terms of the tensor core's type (fp16: off by at most 2^-23 of it or 2^-32
 * of the largest one; bf16 cache: 2^-17 of it), and a bf16 query over an e4m3
 * cache, as fp16 with its head's power of two taken out (off by at most 2^-24 of
 * its largest element). Pages past a sequence's last token are not read, nor
 * are the places after it. A length outside [0, max_pages * page_size] or a
 * page outside [0, num_pages) that is needed sets AWQ_ERR_BAD_INDEX; that
 * sequence's output is then undefined.
 * q, out: 16-bit [batch][q_heads][head_dim] (token_stride = between
 * sequences); page_table i32[batch][max_pages], row stride table_stride;
 * seq_lens i32[batch]; lse f32[batch][q_heads], dense, or NULL.
 * batch >= 0 (0 launches nothing), q_heads a multiple of the cache's
 * num_heads, head_dim a multiple of 8 (16 for an e4m3 cache) up to
 * AWQ_ATTN_MAX_HEAD_DIM, batch * num_heads * ceil(q_heads / num_heads / 16) *
 * (max_pages * page_size / 16 + 1) below 2^31; q, out and both planes 16-byte aligned with strides
 * that are multiples of 16 bytes.
 * The work is split over the sequences' lengths (read on the device) and
 * joined in the same launch. workspace: at least
 * awq_paged_attention_workspace_bytes() of device scratch, 256-byte aligned,
 * zero-filled once before its first use; every call leaves it ready for the
 * next one on the same device. It must not be used by two calls that can run
 * at the same time, nor by other calls of this library.
 */
AWQ_API awq_status awq_paged_attention(const awq_heads *q, const awq_kv_cache *cache,
                                       const int32_t *page_table, int64_t table_stride,
                                       int32_t max_pages, const int32_t *seq_lens, int32_t batch,
                                       int32_t q_heads, int32_t dtype, float scale,
                                       const awq_heads *out, float *lse, void *workspace,
                                       size_t ws_bytes, int32_t *dev_status, void *stream);

/* Workspace bytes awq_paged_attention needs at this head size, for any batch,
 * lengths and heads (0 for a head size that it does not take). Host-only, no
 * CUDA call. */
AWQ_API size_t awq_paged_attention_workspace_bytes(int32_t head_dim);

/*
 * awq_fp8_gemm -- matrix product of e4m3 operands with a scale per block of
 * 128:
 *   out[m][n] = sum over blocks j of 128 columns of K of
 *     a_scales[m][j] * b_scales[n / 128][j] * (sum over k in j of a[m][k] b[n][k])
 * The products are exact; the tensor core adds a block's 128 to within 2^-17 of
 * the sum of their magnitudes; the scales and the sum over the blocks are fp32,
 * with one rounding at the end.
 * a: e4m3 [M][K], row stride lda (bytes); a_scales f32[M][ceil(K / 128)],
 * dense (as awq_add_rmsnorm and awq_quantize_fp8 write them); b: e4m3 [N][K]
 * (a weight, row n = output n), row stride ldb; b_scales f32[ceil(N / 128)]
 * [ceil(K / 128)], dense; out: 16-bit [M][N], row stride ldo (elements).
 * M, N 0..2^30 (0 launches nothing), K 1..2^30, any size up to 2^30 tiles of
 * 128 x 128. a and b 16-byte aligned with row strides that are multiples of 16
 * bytes (a single row's stride is not used); out of any alignment is taken.
 */
AWQ_API awq_status awq_fp8_gemm(const uint8_t *a, int64_t lda, const float *a_scales, const uint8_t *b,
                                int64_t ldb, const float *b_scales, void *out, int64_t ldo, int32_t M,
                                int32_t N, int32_t K, int32_t dtype, int32_t *dev_status,
                                void *stream);

#ifdef __cplusplus
}
#endif
#endif /* AWQ_DECODER_H */
