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

// The 8 values of this lane, normed and rotated. c and s: this lane's cosines and sines (of its 8
// elements for halves, of its 4 pairs for neighbours); `partner`: the lane of the group with the
// other halves, or its own for lanes past the rotated dimensions.
template <int kLanes, bool kInterleaved>
__device__ __forceinline__ void norm_rotate(float (&x)[8], bool norm, const float (&w)[8], float eps, bool rotated, bool second,
                                            int partner, const float (&c)[kInterleaved ? 4 : 8], const float (&s)[kInterleaved ? 4 : 8]) {
    if (norm) {
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = __fmul_rn(x[i], x[i]);
        float sum = __fadd_rn(__fadd_rn(__fadd_rn(y[0], y[1]), __fadd_rn(y[2], y[3])), __fadd_rn(__fadd_rn(y[4], y[5]), __fadd_rn(y[6], y[7])));
#pragma unroll
        for (int d = 1; d < kLanes; d <<= 1) sum = __fadd_rn(sum, __shfl_xor_sync(~0u, sum, d));
        const float r = __frcp_rn(__fsqrt_rn(__fadd_rn(__fmul_rn(sum, 1.f / (8 * kLanes)), eps)));
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __fmul_rn(__fmul_rn(x[i], r), w[i]);
    }
    if constexpr (kInterleaved) {
        if (rotated) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float a = x[2 * i], b = x[2 * i + 1];
                x[2 * i] = __fsub_rn(__fmul_rn(a, c[i]), __fmul_rn(b, s[i]));
                x[2 * i + 1] = __fadd_rn(__fmul_rn(b, c[i]), __fmul_rn(a, s[i]));
            }
        }
    } else {
        // a c - b s of the first half, b c + a s of the second: s has the sign (a - b is a + (-b), rounded alike)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float o = __shfl_sync(~0u, x[i], partner, kLanes);
            if (rotated) x[i] = __fadd_rn(__fmul_rn(x[i], c[i]), __fmul_rn(o, s[i]));
        }
    }
}

// A thread keeps its token's cosines and sines and goes through heads: query heads blockIdx.y, blockIdx.y +
// gridDim.y, ..., kQ of them on their way at once, then kv heads.
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
    for (int h0 = blockIdx.y; h0 < a.q_heads; h0 += kQ * gridDim.y) {
        Raw8<kDtype> raw[kQ] = {};
#pragma unroll
        for (int n = 0; n < kQ; ++n) {
            const int h = h0 + n * gridDim.y;
            const int64_t at = q0 + h * a.q_head;
            if (here && h < a.q_heads && HC_IN_RANGE(at, 8, row_extent(a.tokens, a.q_heads, kD, a.q_token, a.q_head), status)) raw[n].load(a.q, at);
        }
#pragma unroll
        for (int n = 0; n < kQ; ++n) {
            const int h = h0 + n * gridDim.y;
            if (h >= a.q_heads) break;
            float x[8];
            raw[n].get(x);
            norm_rotate<kLanes, kInterleaved>(x, a.r.q_norm != nullptr, w, a.r.eps, rotated, second, partner, c, s);
            const int64_t to = (t * a.q_heads + h) * kD + sub * 8;
            raw[n].set(x);
            if (here && HC_IN_RANGE(to, 8, static_cast<size_t>(a.tokens) * a.q_heads * kD, status)) raw[n].store(a.q_out, to);
        }
    }
    if (a.r.k_norm) load_weights<kDtype>(a.r.k_norm, sub, w);
    for (int h = blockIdx.y; h < a.c.kv_heads; h += gridDim.y) {
        Raw8<kDtype> raw = {}, value = {};
        if (here) {
            const int64_t k = t * a.k_token + h * a.k_head + sub * 8, v = t * a.v_token + h * a.v_head + sub * 8;
            if (HC_IN_RANGE(k, 8, row_extent(a.tokens, a.c.kv_heads, kD, a.k_token, a.k_head), status)) raw.load(a.k, k);
            if (HC_IN_RANGE(v, 8, row_extent(a.tokens, a.c.kv_heads, kD, a.v_token, a.v_head), status)) value.load(a.v, v);
        }
        float x[8];
        raw.get(x);
        norm_rotate<kLanes, kInterleaved>(x, a.r.k_norm != nullptr, w, a.r.eps, rotated, second, partner, c, s);
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
    const int most = a.q_heads > a.c.kv_heads ? a.q_heads : a.c.kv_heads;
    int split = (4 * ctx.sm_count + tiles - 1) / tiles;
    split = split < most ? split : most;
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
