// Attention over the 4-bit cache, chunks: requests' own caches, joined with the prefixes' part.
#include "hc_attention_chunk.cuh"

namespace hc {

template cudaError_t launch_attention_chunk<kJoined>(const Ctx&, const SharedArgs&, int, cudaStream_t);
template cudaError_t attention_chunk_setup<kJoined>();

}  // namespace hc
