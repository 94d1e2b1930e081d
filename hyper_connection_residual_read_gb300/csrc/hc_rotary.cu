// Queries and keys normed by head and rotated by their positions, keys and values rounded into
// the 4-bit cache, in one pass over the projection's output.
//
// A head of a token is D values, held by D / 8 neighbouring lanes of 8 values each: its squares
// are summed within a lane and then by shuffles, neighbours first, which is the order that the
// operator states; the second element of a pair is in the same lane (neighbouring pairs) or D_rot
// / 16 lanes on (halves). Every step is a single rounded operation (no fma): the codes of a key
// are a step function of it, and would differ from place to place with the last bit of it.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "hc_cache.cuh"
#include "hc_serve_internal.h"

namespace hc {
namespace {

constexpr int kThreads = 256;

// A token's row of the table for frequency i.
__device__ __forceinline__ int table_row(const RotaryArgs& a, int64_t t, int axis, int* status) {
    if (axis < 0 || axis >= a.r.axes) {
        atomicOr(status, kStatusBounds);
        axis = 0;
    }
    const int64_t at = static_cast<int64_t>(axis) * a.tokens + t;
    int p = HC_IN_RANGE(at, 1, static_cast<size_t>(a.r.axes) * a.tokens, status) ? a.positions[at] : 0;
    if (p >= a.r.length) {
        atomicOr(status, kStatusBounds);
        p = a.r.length - 1;
    }
    return p;
}

template <int kDtype>
__device__ __forceinline__ void load_weights(const void* w, int sub, float (&x)[8]) {
    Raw8<kDtype> raw;
    raw.load(w, sub * 8);
    raw.get(x);
}

// The sum of squares of a lane's 8 values, neighbours first. (Products two at a time; a sum directly behind them
// would be joined to an fma.)
__device__ __forceinline__ float squares(const float (&x)[8]) {
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const uint64_t v = pair(x[i], x[i + 1]);
        const float2 z = unpair(mul2(v, v));
        y[i] = z.x, y[i + 1] = z.y;
    }
    return __fadd_rn(__fadd_rn(__fadd_rn(y[0], y[1]), __fadd_rn(y[2], y[3])), __fadd_rn(__fadd_rn(y[4], y[5]), __fadd_rn(y[6], y[7])));
}
template <int kLanes>
__device__ __forceinline__ float scale_of(float sum, float eps) {
    return __frcp_rn(__fsqrt_rn(__fadd_rn(__fmul_rn(sum, 1.f / (8 * kLanes)), eps)));
}
// The norms' scales of kQ heads, of whose squares each lane has its sum. The lanes share the heads: after an
// exchange with the neighbour a lane goes on with half of them, so that four heads take five exchanges, a root
// and a quotient instead of sixteen and four of each (8191 tokens of 32/8 heads: 52 us against @@).
template <int kLanes, int kQ>
__device__ __forceinline__ void scales_of(float (&sum)[kQ], int sub, float eps) {
    const bool odd = sub & 1, upper = sub & 2;
    float x;
    if constexpr (kQ == 4) {
        float a0 = odd ? sum[2] : sum[0], a1 = odd ? sum[3] : sum[1];
        a0 = __fadd_rn(a0, __shfl_xor_sync(~0u, odd ? sum[0] : sum[2], 1));
        a1 = __fadd_rn(a1, __shfl_xor_sync(~0u, odd ? sum[1] : sum[3], 1));
        x = __fadd_rn(upper ? a1 : a0, __shfl_xor_sync(~0u, upper ? a0 : a1, 2));
    } else {
        x = __fadd_rn(odd ? sum[1] : sum[0], __shfl_xor_sync(~0u, odd ? sum[0] : sum[1], 1));
        x = __fadd_rn(x, __shfl_xor_sync(~0u, x, 2));
    }
#pragma unroll
    for (int d = 4; d < kLanes; d <<= 1) x = __fadd_rn(x, __shfl_xor_sync(~0u, x, d));
    x = scale_of<kLanes>(x, eps);
#pragma unroll
    for (int n = 0; n < kQ; ++n) sum[n] = __shfl_sync(~0u, x, kQ == 4 ? (n >> 1) | ((n & 1) << 1) : n, kLanes);
}
// x r w.
__device__ __forceinline__ void scaled(float (&x)[8], float r, const float (&w)[8]) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const float2 y = unpair(mul2(mul2(pair(x[i], x[i + 1]), pair(r, r)), pair(w[i], w[i + 1])));
        x[i] = y.x, x[i + 1] = y.y;
    }
}
// The 8 values of this lane rotated. c and s: this lane's cosines and sines (of its 8 elements for halves, of its 4
// pairs for neighbours); `partner`: the lane of the group with the other halves, or its own for lanes past
// the rotated dimensions.
template <int kLanes, bool kInterleaved>
__device__ __forceinline__ void rotate(float (&x)[8], bool rotated, int partner, const float (&c)[kInterleaved ? 4 : 8],
                                       const float (&s)[kInterleaved ? 4 : 8]) {
    if constexpr (kInterleaved) {
        if (rotated) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 u = unpair(mul2(pair(x[2 * i], x[2 * i + 1]), pair(c[i], c[i])));
                const float2 v = unpair(mul2(pair(x[2 * i + 1], x[2 * i]), pair(s[i], s[i])));
                x[2 * i] = __fsub_rn(u.x, v.x);
                x[2 * i + 1] = __fadd_rn(u.y, v.y);
            }
        }
    } else {
        // a c - b s of the first half, b c + a s of the second: s has the sign (a - b is a + (-b), rounded alike)
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = __shfl_sync(~0u, x[i], partner, kLanes);
        if (rotated) {
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const float2 u = unpair(mul2(pair(x[i], x[i + 1]), pair(c[i], c[i + 1])));
                const float2 v = unpair(mul2(pair(o[i], o[i + 1]), pair(s[i], s[i + 1])));
                x[i] = __fadd_rn(u.x, v.x), x[i + 1] = __fadd_rn(u.y, v.y);
            }
        }
    }
}

// A thread keeps its token's cosines and sines and goes through heads. They are numbered through, the kv heads
// first, and a CTA has each gridDim.y-th: the query heads of these, kQ of them on their way at once, then the kv
// heads.
template <int kD, int kDtype, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, 3) rotary_kernel(const RotaryArgs a, int* status) {
    begin_early();
    constexpr int kLanes = kD / 8, kTile = kThreads / kLanes, kAngles = kInterleaved ? 4 : 8;
    constexpr int kQ = kDtype == HC_DTYPE_FP32 ? 2 : 4;
    const int sub = threadIdx.x % kLanes;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kTile + threadIdx.x / kLanes;
    const int sh = 31 - __clz(a.c.block_size);
    // a lane without a token still takes part in the shuffles
    bool here = t < a.tokens;
    const int half = a.r.dim / 2, half_lanes = half / 8;
    const bool rotated = sub < 2 * half_lanes, second = sub >= half_lanes;
    const int partner = !rotated ? sub : second ? sub - half_lanes : sub + half_lanes;
    float c[kAngles] = {}, s[kAngles] = {};
    int64_t slot = -1;
    if (here) {
        if (HC_IN_RANGE(t, 1, a.tokens, status)) slot = a.slots[t];
        if (a.r.dim > 0)
            for (int x = 0; x < a.r.axes; ++x) {
                const int64_t at = static_cast<int64_t>(x) * a.tokens + t;
                here = here && HC_IN_RANGE(at, 1, static_cast<size_t>(a.r.axes) * a.tokens, status) && a.positions[at] >= 0;
            }
        if (here && rotated) {
            const int i0 = kInterleaved ? sub * 4 : (second ? sub - half_lanes : sub) * 8;
            int axis = 0, row = table_row(a, t, a.r.axis_of ? a.r.axis_of[i0] : 0, status);
            if (a.r.axis_of) axis = a.r.axis_of[i0];
#pragma unroll
            for (int i = 0; i < kAngles; ++i) {
                if (i > 0 && a.r.axis_of && a.r.axis_of[i0 + i] != axis) {
                    axis = a.r.axis_of[i0 + i];
                    row = table_row(a, t, axis, status);
                }
                const int64_t at = static_cast<int64_t>(row) * a.r.dim + i0 + i;
                if (!HC_IN_RANGE(at + half, 1, static_cast<size_t>(a.r.length) * a.r.dim, status)) continue;
                c[i] = a.r.cos_sin[at], s[i] = a.r.cos_sin[at + half];
                if (!kInterleaved && !second) s[i] = -s[i];
            }
        }
    }
    float w[8] = {};
    if (a.r.q_norm && a.q_heads > 0) load_weights<kDtype>(a.r.q_norm, sub, w);
    const int64_t q0 = t * a.q_token + sub * 8;
    const int step = gridDim.y;
    const int first = static_cast<int>(blockIdx.y) - a.c.kv_heads % step;
    for (int h0 = first < 0 ? first + step : first; h0 < a.q_heads; h0 += kQ * step) {
        Raw8<kDtype> raw[kQ] = {};
#pragma unroll
        for (int n = 0; n < kQ; ++n) {
            const int h = h0 + n * step;
            const int64_t at = q0 + h * a.q_head;
            if (here && h < a.q_heads && HC_IN_RANGE(at, 8, row_extent(a.tokens, a.q_heads, kD, a.q_token, a.q_head), status)) raw[n].load(a.q, at);
        }
        float r[kQ] = {};
        if (a.r.q_norm) {
#pragma unroll
            for (int n = 0; n < kQ; ++n) {
                float x[8];
                raw[n].get(x);
                r[n] = squares(x);
            }
            scales_of<kLanes, kQ>(r, sub, a.r.eps);
        }
#pragma unroll
        for (int n = 0; n < kQ; ++n) {
            const int h = h0 + n * step;
            if (h >= a.q_heads) break;
            float x[8];
            raw[n].get(x);
            if (a.r.q_norm) scaled(x, r[n], w);
            rotate<kLanes, kInterleaved>(x, rotated, partner, c, s);
            const int64_t to = (t * a.q_heads + h) * kD + sub * 8;
            raw[n].set(x);
            if (here && HC_IN_RANGE(to, 8, static_cast<size_t>(a.tokens) * a.q_heads * kD, status)) raw[n].store(a.q_out, to);
        }
    }
    if (a.r.k_norm) load_weights<kDtype>(a.r.k_norm, sub, w);
    for (int h = blockIdx.y; h < a.c.kv_heads; h += step) {
        Raw8<kDtype> raw = {}, value = {};
        if (here) {
            const int64_t k = t * a.k_token + h * a.k_head + sub * 8, v = t * a.v_token + h * a.v_head + sub * 8;
            if (HC_IN_RANGE(k, 8, row_extent(a.tokens, a.c.kv_heads, kD, a.k_token, a.k_head), status)) raw.load(a.k, k);
            if (HC_IN_RANGE(v, 8, row_extent(a.tokens, a.c.kv_heads, kD, a.v_token, a.v_head), status)) value.load(a.v, v);
        }
        float x[8];
        raw.get(x);
        if (a.r.k_norm) {
            float sum = squares(x);
#pragma unroll
            for (int d = 1; d < kLanes; d <<= 1) sum = __fadd_rn(sum, __shfl_xor_sync(~0u, sum, d));
            scaled(x, scale_of<kLanes>(sum, a.r.eps), w);
        }
        rotate<kLanes, kInterleaved>(x, rotated, partner, c, s);
        Raw8<HC_DTYPE_FP32> key;
        key.set(x);
        uint32_t sm[2], code[2];
        code[0] = round_group<kLanes>(key, sm[0]);
        code[1] = round_group<kLanes>(value, sm[1]);
        if (!here || slot < 0) continue;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            const int64_t g = group_index(a.c, sh, slot, kv, h, status);
            if (g < 0 || !HC_IN_RANGE(g, 1, group_count(a.c), status)) continue;
            reinterpret_cast<uint32_t*>(a.c.codes)[g * kLanes + sub] = code[kv];
            if (sub == 0) reinterpret_cast<uint32_t*>(a.c.scales)[g] = sm[kv];
        }
    }
}

template <int kD, int kDtype>
cudaError_t call(const Ctx& ctx, const RotaryArgs& a, cudaStream_t st) {
    constexpr int kTile = kThreads / (kD / 8);
    const int tiles = (a.tokens - 1) / kTile + 1;
    // as many CTAs for the heads of a tile as fill the GPU, and no more than heads
    const int heads = a.q_heads + a.c.kv_heads;
    int split = (4 * ctx.sm_count + tiles - 1) / tiles;
    split = split < heads ? split : heads;
    split = split < 65535 ? split : 65535;
    const dim3 grid(tiles, split);
    return a.r.interleaved ? launch_early(rotary_kernel<kD, kDtype, true>, grid, kThreads, 0, st, a, ctx.s.status)
                           : launch_early(rotary_kernel<kD, kDtype, false>, grid, kThreads, 0, st, a, ctx.s.status);
}

template <int kDtype>
cudaError_t call_dim(const Ctx& ctx, const RotaryArgs& a, cudaStream_t st) {
    return a.c.head_dim == 64 ? call<64, kDtype>(ctx, a, st) : call<128, kDtype>(ctx, a, st);
}

}  // namespace

cudaError_t launch_kv4_append_rotary(const Ctx& ctx, const RotaryArgs& a, int dtype, cudaStream_t st) {
    switch (dtype) {
        case HC_DTYPE_BF16: return call_dim<HC_DTYPE_BF16>(ctx, a, st);
        case HC_DTYPE_FP16: return call_dim<HC_DTYPE_FP16>(ctx, a, st);
        default: return call_dim<HC_DTYPE_FP32>(ctx, a, st);
    }
}

}  // namespace hc
