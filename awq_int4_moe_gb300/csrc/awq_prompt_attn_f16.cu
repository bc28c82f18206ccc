// fp16 queries over a 16-bit cache, or packed K and V.
#include "awq_prompt_attn.cuh"

namespace awq {

awq_status launch_chunk_f16(const ChunkArgs &a, int sms, cudaStream_t st) { return launch_chunk<__half, false>(a, sms, st); }

}  // namespace awq
