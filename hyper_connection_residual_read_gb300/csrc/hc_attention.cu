// Attention over the 4-bit cache: windows of few rows, and the choice between the kernels.
#include "hc_attention.cuh"

namespace hc {

extern template cudaError_t launch_attention<kPrefix>(const Ctx&, const AttentionArgs&, int, cudaStream_t);
extern template cudaError_t launch_attention<kJoined>(const Ctx&, const AttentionArgs&, int, cudaStream_t);
extern template cudaError_t attention_window_setup<kPrefix>();
extern template cudaError_t attention_window_setup<kJoined>();

size_t attention_scratch_floats(int sm_count) {
    const size_t window = static_cast<size_t>(sm_count) * kAttnCtasPerSm * 2 * kPieceFloats;
    const size_t chunk = attention_chunk_scratch_floats(sm_count);
    return window > chunk ? window : chunk;
}

cudaError_t attention_setup() {
    cudaError_t e = attention_window_setup<kOwn>();
    if (e == cudaSuccess) e = attention_window_setup<kPrefix>();
    if (e == cudaSuccess) e = attention_window_setup<kJoined>();
    if (e == cudaSuccess) e = attention_chunk_setup<kOwn>();
    if (e == cudaSuccess) e = attention_chunk_setup<kPrefix>();
    if (e == cudaSuccess) e = attention_chunk_setup<kJoined>();
    return e;
}

cudaError_t launch_kv4_attention(const Ctx& ctx, const AttentionArgs& a, int dtype, cudaStream_t st) {
    return launch_attention<kOwn>(ctx, a, dtype, st);
}
cudaError_t launch_kv4_attention_prefix(const Ctx& ctx, const AttentionArgs& a, int dtype, cudaStream_t st) {
    return launch_attention<kPrefix>(ctx, a, dtype, st);
}
cudaError_t launch_kv4_attention_joined(const Ctx& ctx, const AttentionArgs& a, int dtype, cudaStream_t st) {
    return launch_attention<kJoined>(ctx, a, dtype, st);
}

}  // namespace hc
