// Attention over the 4-bit cache, chunks: groups of requests against the prefixes that they share.
#include "hc_attention_chunk.cuh"

namespace hc {

template cudaError_t launch_attention_chunk<kPrefix>(const Ctx&, const SharedArgs&, int, cudaStream_t);
template cudaError_t attention_chunk_setup<kPrefix>();

}  // namespace hc
