// Tokens drawn from logits with temperature, top-k, top-p and min-p.
//
// Weights are whole numbers, multiples of 2^-45 of the largest, so that sums are exact and the
// same in any order: which token a uniform number falls on, and where a filter cuts, are decided
// by comparing whole numbers.
//
// exp((x - M) / T) = 2^z, z = (x - M) log2(e) / T in two floats. z is cut into a multiple m / 32
// and a rest |g| <= 1/64, 2^z = 2^(m / 32) (1 + p(g)): the first from a table of 45 bits, p by its
// series to the fourth power (2^-33), in fp32 where it is below 2^-6: within 2^-29 in all.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "hc_serve_internal.h"
#include "hc_window.cuh"

namespace hc {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kUnitBits = 45;
constexpr uint64_t kOne = 1ull << kUnitBits;
constexpr int kIdBits = 18;                  // of an index: HC_SAMPLE_MAX_VOCAB
static_assert(HC_SAMPLE_MAX_VOCAB == 1 << kIdBits);

// 2^(j / 32) 2^45
__constant__ uint64_t kPowers[32] = {
    0x200000000000ull, 0x20B361A62B0Bull, 0x216AB0D9F312ull, 0x222603A024B7ull,
    0x22E57078FAA3ull, 0x23A90E62D173ull, 0x2470F4DCEAC4ull, 0x253D3BEA3FBEull,
    0x260DFC14636Eull, 0x26E34E6E7554ull, 0x27BD4C982468ull, 0x289C10C0C312ull,
    0x297FB5AA6C54ull, 0x2A6856AD3A9Full, 0x2B560FBA90A8ull, 0x2C48FD6074ABull,
    0x2D413CCCFE78ull, 0x2E3EEBD1D8BFull, 0x2F4228E7D603ull, 0x304B1332999Cull,
    0x3159CA845542ull, 0x326E6F619B8Cull, 0x3389230547E1ull, 0x34AA07647C4Bull,
    0x35D13F32B5A7ull, 0x36FEEDE5F6BDull, 0x383337BB0AA5ull, 0x396E41B9DF21ull,
    0x3AB031B9F749ull, 0x3BF92E66F737ull, 0x3D495F454922ull, 0x3EA0ECB6DC8Bull,
};

template <int kDtype>
__device__ __forceinline__ float logit(const void* p, int64_t i) {
    if (kDtype == HC_DTYPE_FP32) return static_cast<const float*>(p)[i];
    const uint16_t u = static_cast<const uint16_t*>(p)[i];
    return kDtype == HC_DTYPE_BF16 ? __uint_as_float(static_cast<uint32_t>(u) << 16) : __half2float(__ushort_as_half(u));
}

// log2(e) / T in two floats.
struct Heat {
    float hi, lo;
};
__device__ __forceinline__ Heat heat_of(float t) {
    const double c = 1.4426950408889634 / static_cast<double>(t);
    Heat h;
    h.hi = static_cast<float>(c);
    h.lo = static_cast<float>(c - static_cast<double>(h.hi));
    return h;
}

// The weight of logit x beside the largest, top, in multiples of 2^-45; x <= top, top finite.
__device__ __forceinline__ uint64_t weight(float x, float top, Heat c, const uint64_t* powers) {
    const float d = __fsub_rn(x, top);
    const float z = __fmul_rn(d, c.hi);
    if (!(z > -47.f)) return 0;
    const float b = __fsub_rn(d, x);
    const float dl = __fsub_rn(__fsub_rn(x, __fsub_rn(d, b)), __fadd_rn(top, b));     // x - top = d + dl
    const float zl = fmaf(dl, c.hi, fmaf(d, c.lo, fmaf(d, c.hi, -z)));
    const int m = __float2int_rn(z * 32.f);
    const float g = fmaf(static_cast<float>(m), -1.f / 32.f, z) + zl;
    const float p = g * fmaf(g, fmaf(g, fmaf(g, 0.009618129f, 0.05550411f), 0.24022651f), kLn2);
    const uint64_t t = powers[m & 31];
    const int64_t more = static_cast<int64_t>(static_cast<int>(t >> 15)) * __float2int_rn(p * 68719476736.f);   // 2^30 2^36
    const uint64_t w = t + static_cast<uint64_t>(more >> 21);
    const int down = -(m >> 5);
    return down == 0 ? w : (w + (1ull << (down - 1))) >> down;
}

// A logit and its index in one whole number: larger logits first, of equal ones lower ids.
__device__ __forceinline__ uint64_t rank_of(float x, int id) {
    uint32_t u = __float_as_uint(x + 0.0f);
    u = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
    return (static_cast<uint64_t>(u) << kIdBits) | static_cast<uint32_t>(HC_SAMPLE_MAX_VOCAB - 1 - id);
}

__device__ __forceinline__ uint64_t block_sum(uint64_t x, uint64_t* buffer) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(~0u, x, d);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) buffer[threadIdx.x >> 5] = x;
    __syncthreads();
    x = 0;
    for (int w = 0; w < kWarps; ++w) x += buffer[w];
    return x;
}
__device__ __forceinline__ uint64_t block_max(uint64_t x, uint64_t* buffer) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const uint64_t o = __shfl_xor_sync(~0u, x, d);
        x = x > o ? x : o;
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 0) buffer[threadIdx.x >> 5] = x;
    __syncthreads();
    x = 0;
    for (int w = 0; w < kWarps; ++w) x = buffer[w] > x ? buffer[w] : x;
    return x;
}

// A CTA a row. Every border is found by bisection: the largest rank down to which the logits are
// as many, or as heavy, as the filter lets stay; the first id up to which they are as heavy as the
// uniform number asks.
template <int kDtype>
__global__ void __launch_bounds__(kThreads) sample_kernel(const SampleArgs a, int* status) {
    begin_early();
    __shared__ uint64_t buffer[kWarps], powers[32];
    const int row = blockIdx.x, tid = threadIdx.x;
    if (!HC_IN_RANGE(row, 1, a.tokens, status)) return;
    constexpr int kItem = kDtype == HC_DTYPE_FP32 ? 4 : 2;
    const void* x = static_cast<const unsigned char*>(a.logits) + row * a.row * kItem;
    if (tid < 32) powers[tid] = kPowers[tid];
    const float u = a.uniform[row], t = a.temperature ? a.temperature[row] : 1.f;
    const float p = a.top_p ? a.top_p[row] : 1.f, least = a.min_p ? a.min_p[row] : 0.f;
    const int k = a.top_k ? a.top_k[row] : 0;

    uint64_t best = 0;
    bool bad = !(u == u && p == p && least == least) || !(fabsf(t) <= 3.402823466e38f);
    for (int i = tid; i < a.vocab; i += kThreads) {
        const float y = logit<kDtype>(x, i);
        bad |= !(y <= 3.402823466e38f);
        const uint64_t r = rank_of(y, i);
        best = r > best ? r : best;
    }
    best = block_max(best, buffer);
    bad = __syncthreads_or(bad);
    const int first = HC_SAMPLE_MAX_VOCAB - 1 - static_cast<int>(best & (HC_SAMPLE_MAX_VOCAB - 1));
    const float top = logit<kDtype>(x, first);
    if (bad || top == -CUDART_INF_F || t < 5.421010862427522e-20f) {
        const bool none = bad || top == -CUDART_INF_F;
        if (tid == 0) {
            a.ids[row] = none ? -1 : first;
            a.logprob[row] = none ? CUDART_NAN_F : 0.f;
        }
        return;
    }
    const Heat heat = heat_of(t);
    // count or mass of the logits of rank `cut` and above, up to id `last`, that weigh `low` at least
    auto count = [&](uint64_t cut) {
        uint64_t n = 0;
        for (int i = tid; i < a.vocab; i += kThreads) n += rank_of(logit<kDtype>(x, i), i) >= cut;
        return block_sum(n, buffer);
    };
    auto mass = [&](uint64_t cut, uint64_t low, int last) {
        uint64_t n = 0;
        for (int i = tid; i <= last; i += kThreads) {
            const float y = logit<kDtype>(x, i);
            const uint64_t w = weight(y, top, heat, powers);
            if (rank_of(y, i) >= cut && w >= low) n += w;
        }
        return block_sum(n, buffer);
    };
    uint64_t cut = 0;
    if (k > 0 && k < a.vocab) {
        for (int bit = 31 + kIdBits; bit >= 0; --bit)
            if (count(cut | 1ull << bit) >= static_cast<uint64_t>(k)) cut |= 1ull << bit;
    }
    if (p < 1.f) {
        const double part = ceil(static_cast<double>(fmaxf(p, 0.f)) * static_cast<double>(mass(cut, 0, a.vocab - 1)));
        const uint64_t want = part < 1.0 ? 1 : static_cast<uint64_t>(part);
        uint64_t to = 0;
        for (int bit = 31 + kIdBits; bit >= 0; --bit) {
            const uint64_t next = to | 1ull << bit;
            if (next <= cut || mass(next, 0, a.vocab - 1) >= want) to = next;
        }
        cut = to > cut ? to : cut;
    }
    uint64_t low = 1;
    if (least > 0.f) {
        low = static_cast<uint64_t>(ceil(static_cast<double>(fminf(least, 1.f)) * static_cast<double>(kOne)));
        low = low < 1 ? 1 : low;
    }
    const uint64_t total = mass(cut, low, a.vocab - 1);
    const double at = floor(static_cast<double>(fmaxf(u, 0.f)) * static_cast<double>(total));
    uint64_t below = at < static_cast<double>(total) ? static_cast<uint64_t>(at) : total - 1;
    below = below < total ? below : total - 1;
    int lo = 0, hi = a.vocab - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (mass(cut, low, mid) > below) hi = mid;
        else lo = mid + 1;
    }
    if (tid == 0) {
        a.ids[row] = lo;
        const float y = logit<kDtype>(x, lo);
        const float z = (y - top) * heat.hi * kLn2;
        a.logprob[row] = z - logf(static_cast<float>(total) * (1.f / kOne));
    }
}

}  // namespace

cudaError_t launch_sample_tokens(const Ctx& ctx, const SampleArgs& a, int dtype, cudaStream_t st) {
    switch (dtype) {
        case HC_DTYPE_BF16: return launch_early(sample_kernel<HC_DTYPE_BF16>, dim3(a.tokens), kThreads, 0, st, a, ctx.s.status);
        case HC_DTYPE_FP16: return launch_early(sample_kernel<HC_DTYPE_FP16>, dim3(a.tokens), kThreads, 0, st, a, ctx.s.status);
        default: return launch_early(sample_kernel<HC_DTYPE_FP32>, dim3(a.tokens), kThreads, 0, st, a, ctx.s.status);
    }
}

}  // namespace hc
