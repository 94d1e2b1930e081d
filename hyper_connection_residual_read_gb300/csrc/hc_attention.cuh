// What the two kernels of the attention over the 4-bit cache share.
#pragma once

#include <cuda_fp16.h>
#include <math_constants.h>
#include <stdint.h>

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

// The window of one request, with what does not fit its arrays cut off and reported.
struct Window {
    int begin;     // its first token in q
    int n;         // its new tokens
    int rows;      // those of them that are computed (at most max_new)
    int kv;        // its tokens in the cache
    int first;     // position of its first new token (negative where kv < n)
};

__device__ __forceinline__ Window load_window(const AttentionArgs& a, int b, int* status) {
    Window w;
    const int lo = a.cu[b], hi = a.cu[b + 1], kv = a.kv[b];
    const int64_t room = static_cast<int64_t>(a.width) * a.c.block_size;
    const bool bad = lo < 0 || hi < lo || hi > a.tokens;
    w.begin = bad ? 0 : lo;
    w.n = bad ? 0 : hi - lo;
    w.rows = min(w.n, a.max_new);
    w.kv = kv < 0 ? 0 : static_cast<int>(kv > room ? room : kv);
    w.first = w.kv - w.n;
    if ((bad || w.n > a.max_new || kv > room) && status) atomicOr(status, kStatusBounds);
    return w;
}

// The block that holds page `page` of request b; block 0, reported, for an entry that
// is none (its values are wrong then, but they are read from the cache's own memory).
__device__ __forceinline__ int load_block(const AttentionArgs& a, int b, int page, int* status) {
    int block = -1;
    if (page < a.width) block = a.table[static_cast<int64_t>(b) * a.width + page];
    if (block < 0 || block >= a.c.blocks) {
        atomicOr(status, kStatusBounds);
        block = 0;
    }
    return block;
}

// 8 codes of a word as 4 pairs of fp16 numbers code - 8, exactly: pair i holds the codes
// at i and i + 4. A code in the low bits of an fp16 pattern 0x6400 is 1024 + code; four
// bits higher it is 1024 + 16 code.
__device__ __forceinline__ void decode_word(uint32_t w, uint32_t (&h)[4]) {
    constexpr uint32_t kLo = 0x000F000Fu, kHi = 0x00F000F0u, kMagic = 0x64006400u;
    const __half2 minus = __float2half2_rn(-1032.f), sixteenth = __float2half2_rn(0.0625f),
                  minus_hi = __float2half2_rn(-72.f);
    const uint32_t w8 = w >> 8;
    uint32_t t[4];
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(t[0]) : "r"(w), "r"(kLo), "r"(kMagic));
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(t[1]) : "r"(w), "r"(kHi), "r"(kMagic));
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(t[2]) : "r"(w8), "r"(kLo), "r"(kMagic));
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(t[3]) : "r"(w8), "r"(kHi), "r"(kMagic));
    __half2 r[4];
    r[0] = __hadd2(*reinterpret_cast<__half2*>(&t[0]), minus);
    r[1] = __hfma2(*reinterpret_cast<__half2*>(&t[1]), sixteenth, minus_hi);
    r[2] = __hadd2(*reinterpret_cast<__half2*>(&t[2]), minus);
    r[3] = __hfma2(*reinterpret_cast<__half2*>(&t[3]), sixteenth, minus_hi);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = *reinterpret_cast<uint32_t*>(&r[i]);
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

// The queries of a tile are multiplied by 2^-e, which brings the largest of them, of
// size `top`, into [2^13, 2^14): exact but for values 2^-27 below it, so that bf16
// queries of any size keep their 8 bits as fp16. The exponents are bounded so that both
// powers are normal; an infinity or NaN leaves e = 0.
__device__ __forceinline__ int query_exponent(float top) {
    const int e = static_cast<int>((__float_as_uint(top) >> 23) & 0xFF) - 127;
    return (top > 0.f && e < 128) ? min(max(e - 13, -110), 114) : 0;
}
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// One contiguous global -> shared copy counted on `bar` (16-byte aligned, whole 16 bytes).
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            tc::smem_u32(dst)),
        "l"(src), "r"(bytes), "r"(tc::smem_u32(bar))
        : "memory");
}

cudaError_t launch_attention_window(const Ctx& ctx, const AttentionArgs& a, int dtype, cudaStream_t st);

}  // namespace hc
