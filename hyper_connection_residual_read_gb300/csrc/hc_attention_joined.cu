// Attention over the 4-bit cache, windows of few rows: requests' own caches, joined with the prefixes' part.
#include "hc_attention.cuh"

namespace hc {

template cudaError_t launch_attention<kJoined>(const Ctx&, const SharedArgs&, int, cudaStream_t);
template cudaError_t attention_window_setup<kJoined>();

}  // namespace hc
