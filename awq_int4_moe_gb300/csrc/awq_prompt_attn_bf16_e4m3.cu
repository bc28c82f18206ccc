// bf16 queries over an e4m3 cache.
#include "awq_prompt_attn.cuh"

namespace awq {

awq_status launch_chunk_bf16_e4m3(const ChunkArgs &a, int sms, cudaStream_t st) { return launch_chunk<__nv_bfloat16, true>(a, sms, st); }

}  // namespace awq
