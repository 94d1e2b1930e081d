// What the kernels of the verify-window operators share.
#pragma once

#include <cuda_fp16.h>
#include <math_constants.h>
#include <stdint.h>

#include <type_traits>

#include "hc_common.cuh"
#include "hc_tc.cuh"
#include "hc_window_internal.h"

namespace hc {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// 2^x by the hardware (ex2.approx: 2^-22 relative; 0 for x below -126 and for -inf).
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// What the bounds-checked build checks against: the groups of a cache (a key or a value of one
// head), the elements of strided [tokens][heads][dim] rows, the entries of the table.
__device__ __forceinline__ size_t group_count(const hc_kv4_cache& c) {
    return static_cast<size_t>(2) * c.blocks * c.kv_heads * c.block_size;
}
__device__ __forceinline__ size_t row_extent(int tokens, int heads, int dim, int64_t token, int64_t head) {
    return static_cast<size_t>(tokens - 1) * token + static_cast<size_t>(heads - 1) * head + dim;
}
__device__ __forceinline__ size_t table_extent(const AttentionArgs& a) { return static_cast<size_t>(a.requests) * a.width; }
__device__ __forceinline__ size_t table_extent(const SharedArgs& a) { return static_cast<size_t>(a.requests / a.subs) * a.width; }
// The table's row of a request, or of a share of a group.
__device__ __forceinline__ int table_row(const AttentionArgs&, int b) { return b; }
__device__ __forceinline__ int table_row(const SharedArgs& a, int b) { return b / a.subs; }

// The window of one request, with what does not fit its arrays cut off and reported. (That kv
// fits the request's row of the table is what the kernels' lookups there rely on.)
struct Window {
    int begin;     // its first token in q
    int n;         // its new tokens
    int rows;      // those of them that are computed (at most max_new)
    int kv;        // its tokens in the cache
    int first;     // position of its first new token (negative where kv < n): all before it is seen
};

// What an attention kernel computes: requests against their caches; groups of requests against
// the prefixes that they share, into the workspace; or the first joined with the second.
enum Side { kOwn, kPrefix, kJoined };

template <Side kSide>
using Args = typename std::conditional<kSide == kOwn, AttentionArgs, SharedArgs>::type;

template <Side kSide>
__device__ __forceinline__ Window load_window(const Args<kSide>& a, int b, int* status) {
    Window w = {};
    if (!HC_IN_RANGE(b, 1, a.requests, status)) return w;
    int at = b, to = b + 1, of = b;
    bool none = false;
    if constexpr (kSide == kPrefix) {
        of = b / a.subs;
        at = a.groups[of], to = a.groups[of + 1];
        none = at < 0 || to < at || to > a.members;
        if (none) at = to = 0;
    }
    const int lo = a.cu[at], hi = a.cu[to], kv = a.kv[of];
    const int64_t room = static_cast<int64_t>(a.width) * a.c.block_size;
    const bool bad = none || lo < 0 || hi < lo || hi > a.tokens;
    w.begin = bad ? 0 : lo;
    w.n = bad ? 0 : hi - lo;
    bool more = w.n > a.max_new;
    if constexpr (kSide == kPrefix) {          // this share of the group's tokens
        more = w.n > a.shared;
        const int skip = static_cast<int>(min(static_cast<int64_t>(b % a.subs) * a.max_new, static_cast<int64_t>(w.n)));
        w.begin += skip, w.n -= skip;
        if (a.subs > 1) w.n = min(w.n, a.max_new);
    }
    w.rows = min(w.n, a.max_new);
    w.kv = kv < 0 ? 0 : static_cast<int>(kv > room ? room : kv);
    w.first = kSide == kPrefix ? w.kv : w.kv - w.n;    // every row sees all of a prefix
    if ((bad || more || kv > room) && status) atomicOr(status, kStatusBounds);
    return w;
}

// 8 codes of a word as 4 pairs of fp16 numbers: pair i holds the codes at i and i + 4. A
// 4-bit number in the low bits of an fp16 pattern is the subnormal code * 2^-24, which a
// tensor core multiplies exactly as any other value; four bits higher it is 16 times
// that. So pairs 0 and 2 are code * 2^-24 and pairs 1 and 3 code * 2^-20: one logical
// operation each, and the powers of two are divided out of the other operand (kOdd) or of
// the result.
constexpr float kCodeUp = 16777216.f;        // 2^24
constexpr float kOdd = 0.0625f;

__device__ __forceinline__ void decode_word(uint32_t w, uint32_t (&h)[4]) {
    const uint32_t w8 = w >> 8;
    h[0] = w & 0x000F000Fu;
    h[1] = w & 0x00F000F0u;
    h[2] = w8 & 0x000F000Fu;
    h[3] = w8 & 0x00F000F0u;
}

template <int kDtype>
__device__ __forceinline__ float2 widen2(uint32_t w) {
    if (kDtype == HC_DTYPE_BF16) return make_float2(bf16_lo(w), bf16_hi(w));
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

template <int kDtype>
__device__ __forceinline__ uint32_t narrow2(float x, float y) {
    if (kDtype == HC_DTYPE_BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint32_t pack_half2(float x, float y) {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Two fp32 operations in one instruction, on a register pair.
__device__ __forceinline__ uint64_t pair(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t z) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t x, uint64_t y) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return r;
}
// Launch with programmatic stream serialisation: the kernel's CTAs may be set up while the previous
// kernel of the stream ends. Every thread begins with pdl_wait, before anything is read or
// written, and most kernels then let the next one be set up. (Called one after the other on a
// stream: 8191 tokens written and read back 26.6 -> 21.3 us, 8 rows scored 12.3 -> 9.0.)
template <typename... KArgs, typename... Args>
cudaError_t launch_early(void (*kernel)(KArgs...), dim3 grid, int block, size_t smem, cudaStream_t st, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}
__device__ __forceinline__ void begin_early() {
    pdl_wait();
    pdl_launch_dependents();
}

// x / y; most sums are short enough for 32 bits, in a fraction of the time.
__device__ __forceinline__ int64_t quotient(int64_t x, int64_t y) {
    if (((x | y) >> 32) == 0) return static_cast<uint32_t>(x) / static_cast<uint32_t>(y);
    return x / y;
}

// Counts a block of the launch that has written its part; the count before it. One thread calls
// it, behind a barrier that the writers have passed: release and acquire cover what the barrier
// ordered, on both sides (a fence by every writer, and one by every reader, cost 0.3 us more).
__device__ __forceinline__ unsigned arrive(unsigned* counter) {
    unsigned before;
    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(before) : "l"(counter) : "memory");
    return before;
}
// The larger, NaN if either is.
__device__ __forceinline__ float max_nan(float x, float y) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float max3(float x, float y, float z) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
    return r;
}

// The queries of a row are multiplied by 2^-e, which brings the largest of them, of
// size `top`, into [2^13, 2^14): exact but for values 2^-27 below it, so that bf16
// queries of any size keep their 8 bits as fp16. The exponents are bounded so that both
// powers are normal; an infinity or NaN leaves e = 0.
__device__ __forceinline__ int query_exponent(float top) {
    const int e = static_cast<int>((__float_as_uint(top) >> 23) & 0xFF) - 127;
    return (top > 0.f && e < 128) ? min(max(e - 13, -110), 114) : 0;
}
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// A prefix's part of a row in the workspace: where its (maximum, sum) lie, behind all rows' values.
__device__ __forceinline__ float2* partial_stats(const SharedArgs& a, int dim) {
    return reinterpret_cast<float2*>(a.partial + static_cast<int64_t>(a.tokens) * a.q_heads * dim);
}
// A row's own part, sums x about 2^peak with the weights' sum `total`, joined with the prefix's,
// means y: out = by_own x + by_prefix y, and ln of the joined sum. A part that has seen nothing has
// a maximum of -inf, and counts for nothing; one with a NaN makes the row NaN.
struct Join {
    float by_own, by_prefix, lse;
};
__device__ __forceinline__ Join join_parts_of_row(float peak, float total, float2 prefix) {
    const float top = fmaxf(peak, prefix.x);
    const float own = peak == -CUDART_INF_F ? 0.f : exp2_fast(peak - top);
    const float other = prefix.x == -CUDART_INF_F ? 0.f : prefix.y * exp2_fast(prefix.x - top);
    const float sum = total * own + other;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    return Join{own * inv, other * inv, sum == 0.f ? -CUDART_INF_F : (top + log2f(sum)) * kLn2};
}

// 16 bytes global -> shared, past L1, in groups that the thread waits for in order.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// Launches by part (hc_attention.cuh; hc_attention_chunk.cuh: more than 16 rows).
template <Side kSide>
cudaError_t launch_attention(const Ctx& ctx, const Args<kSide>& a, int dtype, cudaStream_t st);
template <Side kSide>
cudaError_t attention_window_setup();
template <Side kSide>
cudaError_t launch_attention_chunk(const Ctx& ctx, const Args<kSide>& a, int dtype, cudaStream_t st);
template <Side kSide>
cudaError_t attention_chunk_setup();
size_t attention_chunk_scratch_floats(int sm_count);
// Own parts behind a prefix, of short requests with few rows (hc_attention_short.cu).
cudaError_t launch_attention_short(const Ctx& ctx, const SharedArgs& a, int dtype, cudaStream_t st);
cudaError_t attention_short_setup();

}  // namespace hc
