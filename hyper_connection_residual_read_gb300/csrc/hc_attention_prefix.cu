// Attention over the 4-bit cache, windows of few rows: groups of requests against the prefixes that they share.
#include "hc_attention.cuh"

namespace hc {

template cudaError_t launch_attention<kPrefix>(const Ctx&, const SharedArgs&, int, cudaStream_t);
template cudaError_t attention_window_setup<kPrefix>();

}  // namespace hc
