// Log probabilities of given tokens, with the entropy, the rank and the most likely
// alternatives.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "hc_common.cuh"
#include "hc_window_internal.h"

namespace hc {
namespace {

constexpr int kThreads = 512;

template <int kDtype>
__device__ __forceinline__ float logit(const void* p, int64_t i) {
    if (kDtype == HC_DTYPE_FP32) return static_cast<const float*>(p)[i];
    if (kDtype == HC_DTYPE_BF16) return bf16_lo(static_cast<const uint16_t*>(p)[i]);
    return __half2float(static_cast<const __half*>(p)[i]);
}

template <typename T, typename F>
__device__ T block_reduce(T v, T* s, F f) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v = f(v, __shfl_xor_sync(~0u, v, d));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    v = s[0];
    for (int w = 1; w < kThreads / 32; ++w) v = f(v, s[w]);
    return v;
}

// Value, then index, in one whole number that grows with the value and falls with the
// index (0 is below every entry).
__device__ __forceinline__ uint64_t order_key(float x, int i) {
    uint32_t u = __float_as_uint(x + 0.0f);
    u = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
    return (static_cast<uint64_t>(u) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(i));
}
__device__ __forceinline__ float key_value(uint64_t k) {
    const uint32_t u = static_cast<uint32_t>(k >> 32);
    return __uint_as_float((u & 0x80000000u) ? (u & 0x7FFFFFFFu) : ~u);
}

template <int kDtype>
__global__ void __launch_bounds__(kThreads) logprob_kernel(const LogprobArgs a) {
    __shared__ float sf[kThreads / 32];
    __shared__ int si[kThreads / 32];
    __shared__ uint64_t sk[kThreads / 32];
    const int64_t base = blockIdx.x * a.row;
    const int id = a.ids[blockIdx.x];
    const bool known = id >= 0 && id < a.vocab;
    const float mine = known ? logit<kDtype>(a.logits, base + id) : -CUDART_INF_F;
    float top = -CUDART_INF_F;
    for (int i = threadIdx.x; i < a.vocab; i += kThreads) top = fmaxf(top, logit<kDtype>(a.logits, base + i));
    top = block_reduce(top, sf, [](float x, float y) { return fmaxf(x, y); });
    const float ref = top == -CUDART_INF_F ? 0.f : top;
    float sum = 0.f, below = 0.f;
    int above = 0;
    for (int i = threadIdx.x; i < a.vocab; i += kThreads) {
        const float x = logit<kDtype>(a.logits, base + i), e = expf(x - ref);
        sum += e;
        if (e != 0.f) below += e * (x - ref);
        above += x > mine;
    }
    sum = block_reduce(sum, sf, [](float x, float y) { return x + y; });
    below = block_reduce(below, sf, [](float x, float y) { return x + y; });
    above = block_reduce(above, si, [](int x, int y) { return x + y; });
    const float lse = ref + logf(sum);
    const bool empty = top == -CUDART_INF_F && sum == 0.f;
    auto lp = [&](float x) { return x == -CUDART_INF_F && !(lse != lse) ? x : x - lse; };
    if (threadIdx.x == 0) {
        a.lse[blockIdx.x] = empty ? -CUDART_INF_F : lse;
        a.logprob[blockIdx.x] = lp(mine);
        a.entropy[blockIdx.x] = empty ? 0.f : logf(sum) - below / sum;
        a.rank[blockIdx.x] = known ? above : a.vocab;
    }
    uint64_t last = ~0ull;
    for (int k = 0; k < a.top; ++k) {
        uint64_t best = 0;
        for (int i = threadIdx.x; i < a.vocab; i += kThreads) {
            const uint64_t key = order_key(logit<kDtype>(a.logits, base + i), i);
            if (key < last && key > best) best = key;
        }
        best = block_reduce(best, sk, [](uint64_t x, uint64_t y) { return x > y ? x : y; });
        if (threadIdx.x == 0) {
            a.top_ids[static_cast<int64_t>(blockIdx.x) * a.top + k] =
                static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(best));
            a.top_logprobs[static_cast<int64_t>(blockIdx.x) * a.top + k] = lp(key_value(best));
        }
        last = best;
    }
}

}  // namespace

cudaError_t launch_logprobs(const Ctx&, const LogprobArgs& a, int dtype, cudaStream_t st) {
    switch (dtype) {
        case HC_DTYPE_BF16: logprob_kernel<HC_DTYPE_BF16><<<a.tokens, kThreads, 0, st>>>(a); break;
        case HC_DTYPE_FP16: logprob_kernel<HC_DTYPE_FP16><<<a.tokens, kThreads, 0, st>>>(a); break;
        default: logprob_kernel<HC_DTYPE_FP32><<<a.tokens, kThreads, 0, st>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace hc
