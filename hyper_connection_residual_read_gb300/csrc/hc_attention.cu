// Attention over the 4-bit cache: windows of few rows, and the choice between the kernels.
#include <limits.h>

#include <cmath>

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
// Both rules below go by max_new, max_shared and the room of the tables: lengths lie on the device. (With tables of 32K tokens
// 16 requests behind 2000 take 26 us where tight ones take 19, 64 behind 16384 57 and 48.5.)
//
// A group's rows are many, but where prefixes are short the chunk kernel's start is longer than its work: then each
// group is cut into shares of up to 8 or 16 rows, and each share reads the prefix for itself. The costs are what
// calls take, in us: a start, rounds of units over the resident CTAs, and of the chunk kernel the join of the CTAs that
// share a head. (64 rows of 8 heads: behind 8000 tokens 27.4 by shares, 30.1 by chunks; behind 16000 37.8 and 34.4. 256
// rows of 8 heads behind 2000 31.1 and 29.5, of 2 heads behind 8000 27.8 and 38.5.)
cudaError_t launch_kv4_attention_prefix(const Ctx& ctx, const SharedArgs& a, int dtype, cudaStream_t st) {
    const int group = a.q_heads / a.c.kv_heads;
    const int64_t rows = static_cast<int64_t>(a.shared) * group, room = static_cast<int64_t>(a.width) * a.c.block_size;
    const int64_t heads = static_cast<int64_t>(a.requests) * a.c.kv_heads;
    if (rows <= kMaxRows) return launch_attention<kPrefix>(ctx, a, dtype, st);
    // (in fp64: max_shared bounds tokens and need not be near them, and its products may pass 64 bits)
    auto rounds = [](double units, int ctas) { return std::ceil(units / ctas); };
    const double tiles = static_cast<double>(heads) * static_cast<double>((rows + 255) / 256), keys = static_cast<double>((room + 127) / 128);
    const double sharing = std::ceil(ctx.sm_count / tiles), chunks = 15 + 0.27 * (keys < sharing ? keys : sharing) + 2.4 * rounds(tiles * keys, ctx.sm_count);
    // (shares of 16 rows where a token has more than 8)
    const int each = group <= 8 ? 8 / group : 1;              // tokens of a share
    const int64_t subs = (static_cast<int64_t>(a.shared) + each - 1) / each;
    const double units = static_cast<double>(heads) * subs * ((room + kUnit - 1) / kUnit);
    const double shares = group <= 8 ? 13 + 1.9 * rounds(units, 2 * ctx.sm_count) : 15 + 1.8 * rounds(units, ctx.sm_count);
    SharedArgs b = a;
    if (group <= kMaxRows && shares < chunks && a.requests * subs <= INT_MAX)
        b.subs = static_cast<int>(subs), b.requests = static_cast<int>(a.requests * subs), b.max_new = each;
    return launch_attention<kPrefix>(ctx, b, dtype, st);
}
cudaError_t launch_kv4_attention_joined(const Ctx& ctx, const SharedArgs& a, int dtype, cudaStream_t st) {
    const int64_t rows = static_cast<int64_t>(a.max_new) * (a.q_heads / a.c.kv_heads), room = static_cast<int64_t>(a.width) * a.c.block_size;
    const int64_t heads = static_cast<int64_t>(a.requests) * a.c.kv_heads;
    if (rows <= kMaxRows && room <= kShortRoom && heads >= kWholeHeads) return launch_attention_short(ctx, a, dtype, st);
    return launch_attention<kJoined>(ctx, a, dtype, st);
}

}  // namespace hc
