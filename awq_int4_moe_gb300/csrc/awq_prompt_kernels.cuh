// Kernel-side declarations of the prompt's operators (awq_prompt.h): argument
// blocks, launchers and the sizes that the host and the kernels share.
#pragma once

#include "../../include/awq_prompt.h"
#include "awq_decoder_kernels.cuh"

namespace awq {

// Attention of several new tokens per sequence; K and V packed like q
// (page_table NULL) or in the paged cache.
struct ChunkArgs {
    awq_heads q, out;
    awq_kv_cache cache;            // packed: its planes' token and head strides alone, and the head size
    const int32_t *page_table;     // NULL: packed
    const int32_t *cu_seqlens;     // [batch + 1]
    const int32_t *seq_lens;       // [batch]; NULL: as many as are new
    float *lse;
    int32_t *counters;             // [2 * kChunkMaxCtas], zero between calls
    float *parts;                  // pieces of cut units, see awq_prompt_attn.cuh
    int32_t *status;
    int64_t table_stride;
    int32_t max_len, batch, tokens, q_heads, group;
    uint32_t page_magic;           // as in AttnArgs
    int32_t page_shift;
    int32_t box;                   // keys of one copy: the largest power of two up to 128 that divides a page
    int32_t unit_rows;             // packed rows of a unit: of whole tokens where one has no more
    int32_t narrow_cost;           // kChunkNarrowCost or 0
    int32_t q_box;                 // tokens of one copy of Q; 0: Q is copied row by row
    int32_t head_step[2], page_step[2];    // of K and V: 0 where the plane's stride is 0, else 1
    float factor;                  // |scale| * log2(e) * K's scale
    int32_t negative;              // the scale is below 0
    uint64_t timeout_ns;           // of a block's wait for others, beyond the time that it took itself
};

struct HeadNormArgs {
    RopeArgs rope;
    const void *q_weight, *k_weight;
    float eps;
};

// The grid never exceeds this many blocks (the workspace holds two counters and
// two pieces for each).
constexpr int kChunkMaxCtas = 160;
constexpr size_t kChunkCounterBytes = (2 * kChunkMaxCtas * sizeof(int32_t) + 255) / 256 * 256;
constexpr int kChunkKeys = 128;                                       // tokens of a K or V tile
// Packed rows (a token's query heads of one KV head, token by token) of a unit:
// two tiles of 128, one where a head is larger than 128.
constexpr int chunk_rows(int padded_dim) { return padded_dim <= 128 ? 256 : 128; }
// A unit's fixed part of its cost (Q, turnaround, stores), in tokens of its keys: as two
// key tiles of 2750 cycles each. The turnaround itself is 9000; what of it counts was found by
// timing. With 128 / 256 / 384 / 512, 13 ragged prompts take 190 / 171 / 187 / 184 us, 4 with
// heads of 256 173 / 143 / 146 / 150, one of 8192 tokens 408 / 411 / 412 / 422, 40 short ones with heads of 64
// 77 / 78 / 76 / 74, 4 new tokens of 32 sequences over e4m3 151 / 150 / 145 / 143.
constexpr int64_t kChunkUnitCost = 256;
constexpr int kChunkNarrowCost = 384;          // over e4m3 more for one with both slots on the same rows
// e4m3 codes on their way to fp16: their shared memory, and the bytes from one row of a
// tile to the next. A TMA copy begins on a 128-byte boundary there, so rows of 64 that are
// copied one by one (pages of an odd size) lie 128 apart, and half as many tiles fit.
constexpr int kChunkCodeBytes = 64 * 1024;
__host__ __device__ constexpr int code_row_bytes(int columns, int box) { return columns * box < 128 ? 128 : columns; }
// Floats of a piece: output, maximum, sum of every row.
constexpr size_t chunk_piece_floats(int padded_dim) { return static_cast<size_t>(chunk_rows(padded_dim)) * (padded_dim + 2); }
constexpr size_t chunk_workspace_bytes(int dim)
{
    return kChunkCounterBytes + sizeof(float) * 2 * kChunkMaxCtas * chunk_piece_floats(attn_padded_dim(dim));
}

// One translation unit per pair of types.
awq_status launch_chunk_f16(const ChunkArgs &a, int sms, cudaStream_t st);
awq_status launch_chunk_bf16(const ChunkArgs &a, int sms, cudaStream_t st);
awq_status launch_chunk_f16_e4m3(const ChunkArgs &a, int sms, cudaStream_t st);
awq_status launch_chunk_bf16_e4m3(const ChunkArgs &a, int sms, cudaStream_t st);

// vec: elements per access (8, 4 or 1).
awq_status launch_head_norm(const HeadNormArgs &a, int dtype, int vec, int sms, cudaStream_t st);

}  // namespace awq
