// fp16 queries over an e4m3 cache.
#include "awq_prompt_attn.cuh"

namespace awq {

awq_status launch_chunk_f16_e4m3(const ChunkArgs &a, int sms, cudaStream_t st) { return launch_chunk<__half, true>(a, sms, st); }

}  // namespace awq
