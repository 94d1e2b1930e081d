// The window plan (blocks, slots and positions from lengths) and the 4-bit cache's write
// and read-back.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <limits.h>
#include <stdint.h>

#include "hc_cache.cuh"

namespace hc {
namespace {

// ---------------------------------------------------------------------------
// plan
// ---------------------------------------------------------------------------
//
// A step's lengths are a few KB and its outputs 16 bytes a token, so launches and
// latency bound it: one launch, and no block waits for another. Every CTA scans all
// requests for itself (two prefix sums over at most 8192 requests in shared memory) and
// then writes its own share of the tokens and of the new blocks, finding the request of
// each by bisection of the prefix sums. New blocks are looked up on the free list by
// rank, not in the table, which other CTAs are writing. 32 requests of 8 tokens take 3.6 us,
// 1024 of 128 tokens 7.4 us.

constexpr int kPlanThreads = 512;
constexpr int kPlanTokens = 2048;      // tokens of one CTA: four a thread

__device__ __forceinline__ int add_sat(int a, int b) {
    return static_cast<int>(min(static_cast<unsigned>(a) + static_cast<unsigned>(b), 0x7FFFFFFFu));
}

// Blocks of 2^sh tokens that hold n >= 0 tokens (unsigned: n may be 2^31 - 1).
__device__ __forceinline__ int blocks_of(int n, int sh) {
    return static_cast<int>((static_cast<unsigned>(n) + (1u << sh) - 1u) >> sh);
}

// Number of entries of the ascending a[0..n) that are <= x.
__device__ __forceinline__ int count_le(const int* a, int n, int x) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] <= x) lo = mid + 1;
        else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanArgs a, int* status) {
    begin_early();
    extern __shared__ int smem[];
    const int n = a.requests, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int* s_cached = smem;                   // [n]
    int* s_cu = s_cached + n;               // [n]  tokens up to and including request b
    int* s_want = s_cu + n;                 // [n]  new blocks up to and including request b
    unsigned char* s_granted = reinterpret_cast<unsigned char*>(s_want + n);   // [n]
    __shared__ int s_tok[kPlanThreads / 32], s_blk[kPlanThreads / 32];

    const int sh = 31 - __clz(a.block_size);
    const int count = min(max(a.free_count[0], 0), a.free_capacity);
    for (int b = tid; b < n; b += kPlanThreads) {
        const int c = max(a.cached[b], 0), w = max(a.added[b], 0);
        const int64_t have = (static_cast<int64_t>(c) + a.block_size - 1) >> sh;
        const int64_t total = (static_cast<int64_t>(c) + w + a.block_size - 1) >> sh;
        const bool fits = total <= a.width;
        s_cached[b] = c;
        s_cu[b] = w;
        s_want[b] = fits ? static_cast<int>(total - have) : 0;
        s_granted[b] = fits;
    }
    __syncthreads();
    // inclusive sums: each thread over its own run, then over the threads' totals
    const int per = (n + kPlanThreads - 1) / kPlanThreads;
    const int b0 = min(tid * per, n), b1 = min(b0 + per, n);
    int tok = 0, blk = 0;
    for (int b = b0; b < b1; ++b) {
        tok = add_sat(tok, s_cu[b]);
        blk += s_want[b];
    }
    int tok_in = tok, blk_in = blk;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int t = __shfl_up_sync(~0u, tok_in, d), k = __shfl_up_sync(~0u, blk_in, d);
        if (lane >= d) {
            tok_in = add_sat(tok_in, t);
            blk_in += k;
        }
    }
    if (lane == 31) {
        s_tok[warp] = tok_in;
        s_blk[warp] = blk_in;
    }
    int run_tok = __shfl_up_sync(~0u, tok_in, 1), run_blk = __shfl_up_sync(~0u, blk_in, 1);
    if (lane == 0) run_tok = run_blk = 0;
    __syncthreads();
    for (int w = 0; w < warp; ++w) {
        run_tok = add_sat(run_tok, s_tok[w]);
        run_blk += s_blk[w];
    }
    for (int b = b0; b < b1; ++b) {
        const int want = s_want[b];
        run_tok = add_sat(run_tok, s_cu[b]);
        run_blk += want;
        s_cu[b] = run_tok;
        s_want[b] = run_blk;
        s_granted[b] = s_granted[b] && (want == 0 || run_blk <= count);
    }
    __syncthreads();

    if (blockIdx.x == 0) {
        for (int b = tid; b < n; b += kPlanThreads) {
            a.cu[b + 1] = s_cu[b];
            a.kv[b] = s_granted[b] ? add_sat(s_cached[b], max(a.added[b], 0)) : s_cached[b];
        }
        if (tid == 0) {
            a.cu[0] = 0;
            // blocks wanted by the last request whose wants were still covered
            const int covered = count_le(s_want, n, count);
            a.free_left[0] = count - (covered ? s_want[covered - 1] : 0);
        }
    }
    // new blocks: the i-th wanted goes to the request whose sum first passes i
    const int covered = count_le(s_want, n, count);
    const int taken = covered ? s_want[covered - 1] : 0;
    for (int i = blockIdx.x * kPlanThreads + tid; i < taken; i += gridDim.x * kPlanThreads) {
        const int b = count_le(s_want, n, i);
        const int j = i - (b ? s_want[b - 1] : 0);
        const int have = blocks_of(s_cached[b], sh);
        const size_t at = static_cast<size_t>(b) * a.width + have + j;
        if (HC_IN_RANGE(at, 1, static_cast<size_t>(n) * a.width, status) &&
            HC_IN_RANGE(count - 1 - i, 1, a.free_capacity, status))
            a.table[at] = a.free_blocks[count - 1 - i];
    }
    // tokens
    const int total = s_cu[n - 1];
    const int t1 = min(a.capacity - blockIdx.x * kPlanTokens, kPlanTokens);
    for (int i = tid; i < t1; i += kPlanThreads) {
        const int t = blockIdx.x * kPlanTokens + i;
        int64_t slot = -1;
        int request = -1, pos = -1;
        if (t < total) {
            const int b = count_le(s_cu, n, t);
            const int c = s_cached[b];
            request = b;
            pos = add_sat(c, t - (b ? s_cu[b - 1] : 0));
            if (s_granted[b]) {
                const int at = pos >> sh, have = blocks_of(c, sh);
                const int rank = (b ? s_want[b - 1] : 0) + at - have;
                int block = 0;
                if (at >= have) {
                    if (HC_IN_RANGE(count - 1 - rank, 1, a.free_capacity, status))
                        block = a.free_blocks[count - 1 - rank];
                } else if (HC_IN_RANGE(at, 1, a.width, status)) {
                    block = a.table[static_cast<size_t>(b) * a.width + at];
                }
                if (block < 0) atomicOr(status, kStatusBounds);           // no block: no slot
                else slot = static_cast<int64_t>(block) * a.block_size + (pos & (a.block_size - 1));
            }
        }
        if (!HC_IN_RANGE(t, 1, a.capacity, status)) continue;
        a.slots[t] = slot;
        a.request_of[t] = request;
        a.positions[t] = pos;
    }
}

// ---------------------------------------------------------------------------
// cache write and read-back
// ---------------------------------------------------------------------------
//
// One group (a token's key or value of one head) is D values, held by D / 8 lanes of 8
// values each: its minimum and maximum are a few shuffles, and every lane stores its 8
// codes as one word. A CTA takes the tokens of one tile for one head, key and value of a
// token in the same lanes, both loads on their way before either is rounded. Every value is
// read and written once, 16 bytes a lane, so that memory bounds long calls: 8191 tokens of 8
// heads of 128 in fp16, written and read back, take 20.9 us for 85 MB, 4.1 TB/s. (Four
// tokens a thread at once took 23.6 us, and min, max and codes one value at a time 25.3.) 32
// tokens take 3.1 us for both launches.

constexpr int kCacheThreads = 256;

template <int kD, int kDtype>
__global__ void __launch_bounds__(kCacheThreads) append_kernel(const CacheArgs a, int* status) {
    begin_early();
    constexpr int kLanes = kD / 8, kTile = kCacheThreads / kLanes;
    const int sub = threadIdx.x % kLanes, head = blockIdx.y;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kTile + threadIdx.x / kLanes;
    const int sh = 31 - __clz(a.c.block_size);
    // a lane without a token still takes part in the shuffles
    Raw8<kDtype> raw[2] = {};
    int64_t slot = -1;
    if (t < a.tokens) {
        slot = a.slots[t];
        const int64_t k = t * a.k_token + head * a.k_head + sub * 8, v = t * a.v_token + head * a.v_head + sub * 8;
        if (HC_IN_RANGE(k, 8, row_extent(a.tokens, a.c.kv_heads, kD, a.k_token, a.k_head), status)) raw[0].load(a.k, k);
        if (HC_IN_RANGE(v, 8, row_extent(a.tokens, a.c.kv_heads, kD, a.v_token, a.v_head), status)) raw[1].load(a.v, v);
    }
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        uint32_t sm;
        const uint32_t code = round_group<kLanes>(raw[kv], sm);
        if (slot < 0) continue;
        const int64_t g = group_index(a.c, sh, slot, kv, head, status);
        if (g < 0 || !HC_IN_RANGE(g, 1, group_count(a.c), status)) continue;
        reinterpret_cast<uint32_t*>(a.c.codes)[g * kLanes + sub] = code;
        if (sub == 0) reinterpret_cast<uint32_t*>(a.c.scales)[g] = sm;
    }
}

template <int kD, int kDtype>
__global__ void __launch_bounds__(kCacheThreads) load_kernel(const CacheArgs a, int* status) {
    begin_early();
    constexpr int kLanes = kD / 8, kTile = kCacheThreads / kLanes;
    const int sub = threadIdx.x % kLanes, head = blockIdx.y;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kTile + threadIdx.x / kLanes;
    const int sh = 31 - __clz(a.c.block_size);
    if (t >= a.tokens) return;
    const int64_t slot = a.slots[t];
    uint32_t code[2] = {}, sm[2] = {};
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        const int64_t g = slot < 0 ? -1 : group_index(a.c, sh, slot, kv, head, status);
        if (g < 0 || !HC_IN_RANGE(g, 1, group_count(a.c), status)) continue;
        code[kv] = reinterpret_cast<const uint32_t*>(a.c.codes)[g * kLanes + sub];
        sm[kv] = reinterpret_cast<const uint32_t*>(a.c.scales)[g];
    }
    const int64_t at = (t * a.c.kv_heads + head) * kD + sub * 8;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        // A code stays where it is in its half word: 16^i c as the low bits of 2^23 + 16^i c, met by
        // s / 16^i (exact: s has 8 bits and is 2^-126 at least, or 0), so that the sum is rounded
        // once and the same.
        const float s = bf16_lo(sm[kv]), m = bf16_hi(sm[kv]);
        const uint64_t s01 = pair(s, s * 0x1p-4f), s23 = pair(s * 0x1p-8f, s * 0x1p-12f);
        const uint64_t m2 = pair(m, m), less = pair(-8388608.f, -8388608.f);
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const uint32_t w = code[kv] >> (i / 4 * 16);
            const int at = i % 4 * 4;
            const uint64_t c = add2(pair(__uint_as_float((w & (15u << at)) | 0x4B000000u),
                                         __uint_as_float((w & (240u << at)) | 0x4B000000u)), less);
            const float2 y = unpair(fma2(i % 4 ? s23 : s01, c, m2));
            x[i] = y.x, x[i + 1] = y.y;
        }
        Raw8<kDtype> raw;
        raw.set(x);
        if (HC_IN_RANGE(at, 8, static_cast<size_t>(a.tokens) * a.c.kv_heads * kD, status)) raw.store(kv ? a.v_out : a.k_out, at);
    }
}

template <int kD, int kDtype>
cudaError_t cache_call(const Ctx& ctx, const CacheArgs& a, bool append, cudaStream_t st) {
    constexpr int kTile = kCacheThreads / (kD / 8);
    const dim3 grid((a.tokens - 1) / kTile + 1, a.c.kv_heads);
    return append ? launch_early(append_kernel<kD, kDtype>, grid, kCacheThreads, 0, st, a, ctx.s.status)
                  : launch_early(load_kernel<kD, kDtype>, grid, kCacheThreads, 0, st, a, ctx.s.status);
}

template <int kDtype>
cudaError_t cache_call_dim(const Ctx& ctx, const CacheArgs& a, bool append, cudaStream_t st) {
    return a.c.head_dim == 64 ? cache_call<64, kDtype>(ctx, a, append, st)
                              : cache_call<128, kDtype>(ctx, a, append, st);
}

cudaError_t cache_dispatch(const Ctx& ctx, const CacheArgs& a, int dtype, bool append, cudaStream_t st) {
    switch (dtype) {
        case HC_DTYPE_BF16: return cache_call_dim<HC_DTYPE_BF16>(ctx, a, append, st);
        case HC_DTYPE_FP16: return cache_call_dim<HC_DTYPE_FP16>(ctx, a, append, st);
        default: return cache_call_dim<HC_DTYPE_FP32>(ctx, a, append, st);
    }
}

}  // namespace

cudaError_t window_setup() {
    return cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, HC_PLAN_MAX_REQUESTS * 13);
}

cudaError_t launch_plan(const Ctx& ctx, const PlanArgs& a, cudaStream_t st) {
    const size_t smem = static_cast<size_t>(a.requests) * 13;
    const int grid = a.capacity > kPlanTokens ? (a.capacity - 1) / kPlanTokens + 1 : 1;
    return launch_early(plan_kernel, dim3(grid), kPlanThreads, smem, st, a, ctx.s.status);
}

cudaError_t launch_kv4_append(const Ctx& ctx, const CacheArgs& a, int dtype, cudaStream_t st) {
    return cache_dispatch(ctx, a, dtype, true, st);
}

cudaError_t launch_kv4_load(const Ctx& ctx, const CacheArgs& a, int dtype, cudaStream_t st) {
    return cache_dispatch(ctx, a, dtype, false, st);
}

}  // namespace hc
