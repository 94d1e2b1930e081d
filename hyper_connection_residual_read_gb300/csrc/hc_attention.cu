// Attention over the cache held in 4 bits.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "hc_common.cuh"
#include "hc_window_internal.h"

namespace hc {
namespace {

template <int kDtype>
__device__ __forceinline__ float widen(const void* p, int64_t i) {
    if (kDtype == HC_DTYPE_BF16) return bf16_lo(static_cast<const uint16_t*>(p)[i]);
    return __half2float(static_cast<const __half*>(p)[i]);
}

// One warp for each token and query head: one pass over the keys with the running maximum
// and sum, each lane holding kD / 32 neighbouring dimensions.
template <int kD, int kDtype>
__global__ void __launch_bounds__(128) attention_kernel(const AttentionArgs a, int* status) {
    constexpr int kN = kD / 32;
    const int lane = threadIdx.x & 31;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    if (row >= static_cast<int64_t>(a.tokens) * a.q_heads) return;
    const int t = static_cast<int>(row / a.q_heads), hq = static_cast<int>(row % a.q_heads);
    const int h = hq / (a.q_heads / a.c.kv_heads);
    int b = 0;
    while (b < a.requests && a.cu[b + 1] <= t) ++b;
    if (b == a.requests) return;
    const int n = a.cu[b + 1] - a.cu[b], kv = max(a.kv[b], 0), first = kv - n, i = t - a.cu[b];
    if (i >= a.max_new) {
        if (lane == 0) atomicOr(status, kStatusBounds);
        return;
    }
    float q[kN], o[kN] = {};
#pragma unroll
    for (int e = 0; e < kN; ++e) q[e] = widen<kDtype>(a.q, t * a.q_token + hq * a.q_head + lane * kN + e);
    float top = -CUDART_INF_F, sum = 0.f;
    const uint64_t mask = a.mask ? a.mask[t] : 0;
    for (int j = 0; j < kv; ++j) {
        if (a.mask ? (j >= first && !((mask >> (j - first)) & 1)) : j > first + i) continue;
        const int page = j / a.c.block_size, off = j % a.c.block_size;
        const int block = page < a.width ? a.table[static_cast<int64_t>(b) * a.width + page] : -1;
        if (block < 0 || block >= a.c.blocks) {
            if (lane == 0) atomicOr(status, kStatusBounds);
            continue;
        }
        const int64_t gk = ((static_cast<int64_t>(block) * 2) * a.c.kv_heads + h) * a.c.block_size + off;
        const int64_t gv = gk + static_cast<int64_t>(a.c.kv_heads) * a.c.block_size;
        float k[kN], v[kN];
        const float sk = bf16_lo(a.c.scales[2 * gk]), mk = bf16_lo(a.c.scales[2 * gk + 1]);
        const float sv = bf16_lo(a.c.scales[2 * gv]), mv = bf16_lo(a.c.scales[2 * gv + 1]);
#pragma unroll
        for (int e = 0; e < kN; ++e) {
            const int at = (lane * kN + e) / 2, sh = 4 * (e & 1);
            k[e] = fmaf(sk, static_cast<float>((a.c.codes[gk * (kD / 2) + at] >> sh) & 15), mk);
            v[e] = fmaf(sv, static_cast<float>((a.c.codes[gv * (kD / 2) + at] >> sh) & 15), mv);
        }
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < kN; ++e) s = fmaf(q[e], k[e], s);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
        s *= a.scale;
        const float up = fmaxf(top, s);
        const float old = top == -CUDART_INF_F ? 0.f : expf(top - up), p = s == -CUDART_INF_F ? 0.f : expf(s - up);
        sum = sum * old + p;
#pragma unroll
        for (int e = 0; e < kN; ++e) o[e] = fmaf(p, v[e], o[e] * old);
        top = up;
    }
    const float r = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int e = 0; e < kN; ++e) {
        const float x = o[e] * r;
        static_cast<uint16_t*>(a.out)[row * kD + lane * kN + e] =
            kDtype == HC_DTYPE_BF16 ? to_bf16_bits(x) : to_fp16_bits(x);
    }
    if (lane == 0 && a.lse) a.lse[row] = sum == 0.f ? -CUDART_INF_F : top + logf(sum);
}

template <int kD>
void launch_dim(const Ctx& ctx, const AttentionArgs& a, int dtype, cudaStream_t st) {
    const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(a.tokens) * a.q_heads + 3) / 4);
    if (dtype == HC_DTYPE_BF16)
        attention_kernel<kD, HC_DTYPE_BF16><<<grid, 128, 0, st>>>(a, ctx.s.status);
    else
        attention_kernel<kD, HC_DTYPE_FP16><<<grid, 128, 0, st>>>(a, ctx.s.status);
}

}  // namespace

cudaError_t launch_kv4_attention(const Ctx& ctx, const AttentionArgs& a, int dtype, cudaStream_t st) {
    if (a.c.head_dim == 64) launch_dim<64>(ctx, a, dtype, st);
    else launch_dim<128>(ctx, a, dtype, st);
    return cudaGetLastError();
}

}  // namespace hc
