// Attention over the 4-bit cache, chunks.
#include "hc_attention_chunk.cuh"

namespace hc {

size_t attention_chunk_scratch_floats(int sm_count) { return static_cast<size_t>(sm_count) * 2 * kPieceFloats; }

template cudaError_t launch_attention_chunk<kOwn>(const Ctx&, const AttentionArgs&, int, cudaStream_t);
template cudaError_t attention_chunk_setup<kOwn>();

}  // namespace hc
