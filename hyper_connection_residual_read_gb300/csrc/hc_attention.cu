// Attention over the 4-bit cache: windows of few rows, and the choice between the kernels.
#include <limits.h>

#include "hc_attention.cuh"

namespace hc {

// Requests whose tables hold at most so many tokens of their own are short.
constexpr int kShortRoom = 2048;

extern template cudaError_t launch_attention<kPrefix>(const Ctx&, const SharedArgs&, int, cudaStream_t);
extern template cudaError_t launch_attention<kJoined>(const Ctx&, const SharedArgs&, int, cudaStream_t);
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
    if (e == cudaSuccess) e = attention_short_setup();
    if (e == cudaSuccess) e = attention_chunk_setup<kOwn>();
    if (e == cudaSuccess) e = attention_chunk_setup<kPrefix>();
    if (e == cudaSuccess) e = attention_chunk_setup<kJoined>();
    return e;
}

cudaError_t launch_kv4_attention(const Ctx& ctx, const AttentionArgs& a, int dtype, cudaStream_t st) {
    return launch_attention<kOwn>(ctx, a, dtype, st);
}
// A group's rows are many, but where prefixes are short the chunk kernel's start is longer than its work: then each
// group is cut into shares of up to 8 or 16 rows, and each share reads the prefix for itself. The costs are what
// the kernels take, in us: a start, and rounds of units over the resident CTAs.
cudaError_t launch_kv4_attention_prefix(const Ctx& ctx, const SharedArgs& a, int dtype, cudaStream_t st) {
    const int group = a.q_heads / a.c.kv_heads;
    const int64_t rows = static_cast<int64_t>(a.shared) * group, room = static_cast<int64_t>(a.width) * a.c.block_size;
    const int64_t heads = static_cast<int64_t>(a.requests) * a.c.kv_heads;
    if (rows <= kMaxRows) return launch_attention<kPrefix>(ctx, a, dtype, st);
    auto rounds = [&](int64_t units, int ctas) { return static_cast<double>((units + ctas - 1) / ctas); };
    double least = 20 + 2.4 * rounds(heads * ((rows + 255) / 256) * ((room + 127) / 128), ctx.sm_count);
    SharedArgs b = a;
    for (int most = 8; most <= kMaxRows; most += 8) {
        const int each = most / group;                       // tokens of a share
        if (each == 0) continue;
        const int64_t subs = (a.shared + each - 1) / each, units = heads * subs * ((room + kUnit - 1) / kUnit);
        const double cost = most == 8 ? 7 + 2.2 * rounds(units, 2 * ctx.sm_count) : 14 + 3.5 * rounds(units, ctx.sm_count);
        if (cost >= least || a.requests * subs > INT_MAX) continue;
        least = cost;
        b.subs = static_cast<int>(subs), b.requests = static_cast<int>(a.requests * subs), b.max_new = each;
    }
    return launch_attention<kPrefix>(ctx, b, dtype, st);
}
cudaError_t launch_kv4_attention_joined(const Ctx& ctx, const SharedArgs& a, int dtype, cudaStream_t st) {
    const int64_t rows = static_cast<int64_t>(a.max_new) * (a.q_heads / a.c.kv_heads), room = static_cast<int64_t>(a.width) * a.c.block_size;
    const int64_t heads = static_cast<int64_t>(a.requests) * a.c.kv_heads;
    if (rows <= kMaxRows && room <= kShortRoom && heads >= kWholeHeads) return launch_attention_short(ctx, a, dtype, st);
    return launch_attention<kJoined>(ctx, a, dtype, st);
}

}  // namespace hc
