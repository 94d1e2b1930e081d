// Queries and keys normed by head and rotated by their positions, keys and values rounded into
// the 4-bit cache, in one pass over the projection's output.
//
// A head of a token is D values, held by D / 16 neighbouring lanes: 8 of the first half and the 8 as far into the
// second, 16 bytes each. So the pairs of halves lie in one lane (where all dimensions are rotated), and so do
// neighbouring pairs. Squares are summed within a lane and then by shuffles, neighbours first, which is the
// order that the operator states. Every step is a single rounded operation (no fma): the codes of a key are a
// step function of it, and would differ from place to place with the last bit of it.
//
// A CTA takes some heads of a share of the tokens, so that a token's cosines and sines are fetched once for them,
// and brings heads through a ring of three steps of asynchronous copies. (Of one step in fp32, whose heads are twice as
// large: nothing is brought ahead there, and each step waits for its loads.)
//
// Measured: 8191 tokens, 32 query and 8 kv heads of 128, bf16, with norms, 34.9 us, 176 MB at 5.0 TB/s (74% of the
// copy rate): issue bounds it (65% of the slots; ALU 46%, FMA 32%), since without fma and with each rounding of its
// own a value costs some ten instructions. 4099 tokens of 16 + 16 heads of 64, fp16, three axes, no norm, 12.1 us:
// a CTA's few steps hardly outlast its start. 32 tokens 3.3 us, a launch and a chain of loads. In fp32 8191 tokens of
// 32 + 8 heads take 81 us, 349 MB at 4.3 TB/s. Halves of a part of the head (8191 tokens, 64 of 128 dimensions) 40 us.
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

enum Pairs { kHalves, kNeighbours, kPartHalves };     // (i, i + D / 2); (2i, 2i + 1); (i, i + dim / 2), dim < D
template <Pairs kPairs>
constexpr int kCtasPerSm = kPairs == kPartHalves ? 2 : 3;      // (of 120 to 124 registers a thread, and of 80)

template <int kDtype>
__device__ __forceinline__ void load_weights(const void* w, int at, float (&x)[8]) {
    Raw8<kDtype> raw;
    raw.load(w, at);
    raw.get(x);
}

// This thread's 8 values of a ring's slot.
template <int kDtype, int kPieces>
__device__ __forceinline__ Raw8<kDtype> from_ring(const uint4 (&slot)[kPieces][kThreads]) {
    Raw8<kDtype> raw;
    if constexpr (kPieces == 1) {
        raw.v = slot[0][threadIdx.x];
    } else {
        raw.a = *reinterpret_cast<const float4*>(&slot[0][threadIdx.x]);
        raw.b = *reinterpret_cast<const float4*>(&slot[1][threadIdx.x]);
    }
    return raw;
}

// The sum of squares of 8 values, neighbours first. (Products two at a time; a sum directly behind them would be
// joined to an fma.)
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
__device__ __forceinline__ float add_xor(float x, float sent, int d) { return __fadd_rn(x, __shfl_xor_sync(~0u, sent, d)); }

// The norms' scales of kN heads from each lane's sums of its two halves. The lanes share them: in an exchange with
// a neighbour a lane gives half of what it has and goes on with the others, so that one root and one quotient
// do for two heads.
template <int kLanes, int kN>
__device__ __forceinline__ void scales_of(const float (&sum)[kN][2], int sub, float eps, float (&r)[kN]) {
    const bool odd = sub & 1, last = sub & 4;
    float x[2];                              // of this lane's head
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        x[h] = kN == 2 ? add_xor(odd ? sum[kN - 1][h] : sum[0][h], odd ? sum[0][h] : sum[kN - 1][h], 1) : add_xor(sum[0][h], sum[0][h], 1);
        x[h] = add_xor(x[h], x[h], 2);
    }
    float total;
    if constexpr (kLanes == 8) {             // a half a lane, then both
        total = add_xor(last ? x[1] : x[0], last ? x[0] : x[1], 4);
        total = add_xor(total, total, 4);
    } else {
        total = __fadd_rn(x[0], x[1]);
    }
    total = __frcp_rn(__fsqrt_rn(__fadd_rn(__fmul_rn(total, 1.f / (16 * kLanes)), eps)));
#pragma unroll
    for (int n = 0; n < kN; ++n) r[n] = kN == 1 ? total : __shfl_sync(~0u, total, n, kLanes);
}
// x r w.
__device__ __forceinline__ void scaled(float (&x)[8], float r, const float (&w)[8]) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const float2 y = unpair(mul2(mul2(pair(x[i], x[i + 1]), pair(r, r)), pair(w[i], w[i + 1])));
        x[i] = y.x, x[i + 1] = y.y;
    }
}

// What a lane keeps of its token's angles: of its 8 pairs of halves; of the 4 pairs of each of its vectors; of
// the 8 elements of each, with the sign of what the other half adds in the sine.
template <Pairs kPairs>
struct Angles {
    static constexpr int kN = kPairs == kPartHalves ? 16 : 8;
    float c[kN], s[kN];
    bool turns[2];                           // whether the vectors are rotated
};
// Lane and vector of the other half of vector `chunk` of a head, of dim / 16 vectors a half.
__device__ __forceinline__ int other_half(int chunk, int half) { return chunk < half ? chunk + half : chunk < 2 * half ? chunk - half : chunk; }

template <int kLanes, Pairs kPairs>
__device__ __forceinline__ void rotate(float (&x)[2][8], const Angles<kPairs>& t, int sub, int half) {
    if constexpr (kPairs == kHalves) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const uint64_t a = pair(x[0][i], x[0][i + 1]), b = pair(x[1][i], x[1][i + 1]);
            const uint64_t c = pair(t.c[i], t.c[i + 1]), s = pair(t.s[i], t.s[i + 1]);
            const float2 ac = unpair(mul2(a, c)), bs = unpair(mul2(b, s)), bc = unpair(mul2(b, c)), as = unpair(mul2(a, s));
            x[0][i] = __fsub_rn(ac.x, bs.x), x[0][i + 1] = __fsub_rn(ac.y, bs.y);
            x[1][i] = __fadd_rn(bc.x, as.x), x[1][i + 1] = __fadd_rn(bc.y, as.y);
        }
    } else if constexpr (kPairs == kNeighbours) {
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            if (!t.turns[v]) continue;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float a = x[v][2 * i], b = x[v][2 * i + 1];
                const float2 c = unpair(mul2(pair(a, b), pair(t.c[4 * v + i], t.c[4 * v + i])));
                const float2 s = unpair(mul2(pair(b, a), pair(t.s[4 * v + i], t.s[4 * v + i])));
                x[v][2 * i] = __fsub_rn(c.x, s.x), x[v][2 * i + 1] = __fadd_rn(c.y, s.y);
            }
        }
    } else {
        float o[2][8];
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const int from = other_half(v * kLanes + sub, half);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float low = __shfl_sync(~0u, x[0][i], from % kLanes, kLanes), high = __shfl_sync(~0u, x[1][i], from % kLanes, kLanes);
                o[v][i] = from < kLanes ? low : high;
            }
        }
        // a c - b s of the first half, b c + a s of the second (a - b is a + (-b), rounded alike)
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            if (!t.turns[v]) continue;
#pragma unroll
            for (int i = 0; i < 8; ++i) x[v][i] = __fadd_rn(__fmul_rn(x[v][i], t.c[8 * v + i]), __fmul_rn(o[v][i], t.s[8 * v + i]));
        }
    }
}

// A thread keeps its token's angles and goes through heads. They are numbered through, the kv heads first, and a
// CTA has each gridDim.y-th: the query heads of these, two at a time, then the kv heads, a key and a value. What a
// thread needs comes to a ring of its own in shared memory, two such steps ahead (fp32: as it is needed).
template <int kD, int kDtype, Pairs kPairs>
__global__ void __launch_bounds__(kThreads, kCtasPerSm<kPairs>) rotary_kernel(const RotaryArgs a, int* status) {
    begin_early();
    constexpr int kLanes = kD / 16, kTile = kThreads / kLanes;
    const int sub = threadIdx.x % kLanes;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kTile + threadIdx.x / kLanes;
    const int sh = 31 - __clz(a.c.block_size);
    // a lane without a token still takes part in the shuffles
    bool here = t < a.tokens;
    const int half = a.r.dim / 16;               // vectors of a half of the rotated dimensions
    Angles<kPairs> angles = {};
    int64_t slot = -1;
    if (here) {
        if (HC_IN_RANGE(t, 1, a.tokens, status)) slot = a.slots[t];
        if (a.r.dim > 0)
            for (int x = 0; x < a.r.axes; ++x) {
                const int64_t at = static_cast<int64_t>(x) * a.tokens + t;
                here = here && HC_IN_RANGE(at, 1, static_cast<size_t>(a.r.axes) * a.tokens, status) && a.positions[at] >= 0;
            }
    }
#pragma unroll
    for (int v = 0; v < 2; ++v) {
        const int chunk = v * kLanes + sub;
        angles.turns[v] = chunk < 2 * half;
        if (!here || !angles.turns[v] || (kPairs == kHalves && v == 1)) continue;
        constexpr int kEach = kPairs == kNeighbours ? 4 : 8;
        const int i0 = kPairs == kNeighbours ? chunk * 4 : (chunk < half ? chunk : chunk - half) * 8;
        const bool minus = kPairs == kPartHalves && chunk < half;
        int axis = a.r.axis_of ? a.r.axis_of[i0] : 0, row = table_row(a, t, axis, status);
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            if (i > 0 && a.r.axis_of && a.r.axis_of[i0 + i] != axis) {
                axis = a.r.axis_of[i0 + i];
                row = table_row(a, t, axis, status);
            }
            const int64_t at = static_cast<int64_t>(row) * a.r.dim + i0 + i;
            if (!HC_IN_RANGE(at + a.r.dim / 2, 1, static_cast<size_t>(a.r.length) * a.r.dim, status)) continue;
            const float s = a.r.cos_sin[at + a.r.dim / 2];
            angles.c[kEach * v + i] = a.r.cos_sin[at], angles.s[kEach * v + i] = minus ? -s : s;
        }
    }
    // the CTA's heads: q0 + j step, j < nq, and k0 + j step, j < nk
    const int step = gridDim.y, kv_heads = a.c.kv_heads, k0 = blockIdx.y, q0 = (k0 + step - kv_heads % step) % step;
    const int nq = a.q_heads > q0 ? (a.q_heads - q0 - 1) / step + 1 : 0, nk = kv_heads > k0 ? (kv_heads - k0 - 1) / step + 1 : 0;
    constexpr int kPieces = kDtype == HC_DTYPE_FP32 ? 2 : 1, kRing = kDtype == HC_DTYPE_FP32 ? 1 : 3;   // 16 bytes a piece
    __shared__ uint4 ring[kRing][2][2][kPieces][kThreads];       // [step][head, or key and value][half]
    const int q_steps = (nq + 1) / 2, steps = q_steps + nk;
    auto bring = [&](uint4 (&to)[2][kPieces][kThreads], const void* from, int64_t at, size_t extent) {
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            if (!HC_IN_RANGE(at + v * (kD / 2), 8, extent, status)) continue;
            const unsigned char* bytes = static_cast<const unsigned char*>(from) + (at + v * (kD / 2)) * (2 * kPieces);
#pragma unroll
            for (int e = 0; e < kPieces; ++e) copy16(tc::smem_u32(&to[v][e][threadIdx.x]), bytes + 16 * e);
        }
    };
    auto issue = [&](int b) {
        if (here && b < steps) {
            auto& to = ring[b % kRing];
            if (b < q_steps) {
#pragma unroll
                for (int n = 0; n < 2; ++n)
                    if (2 * b + n < nq)
                        bring(to[n], a.q, t * a.q_token + static_cast<int64_t>(q0 + (2 * b + n) * step) * a.q_head + sub * 8,
                              row_extent(a.tokens, a.q_heads, kD, a.q_token, a.q_head));
            } else {
                const int h = k0 + (b - q_steps) * step;
                bring(to[0], a.k, t * a.k_token + h * a.k_head + sub * 8, row_extent(a.tokens, kv_heads, kD, a.k_token, a.k_head));
                bring(to[1], a.v, t * a.v_token + h * a.v_head + sub * 8, row_extent(a.tokens, kv_heads, kD, a.v_token, a.v_head));
            }
        }
        copy_commit();
    };
    float w[2][8] = {};
    auto take_weights = [&](const void* from) {
#pragma unroll
        for (int v = 0; v < 2; ++v) load_weights<kDtype>(from, v * (kD / 2) + sub * 8, w[v]);
    };
#pragma unroll
    for (int b = 0; b < kRing - 1; ++b) issue(b);
    if (a.r.q_norm && nq > 0) take_weights(a.r.q_norm);
    for (int b = 0; b < steps; ++b) {
        issue(b + kRing - 1);
        copy_wait<kRing - 1>();
        auto& in = ring[b % kRing];
        if (b < q_steps) {
            float r[2] = {};
            if (a.r.q_norm) {
                float sum[2][2];
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int v = 0; v < 2; ++v) {
                        float x[8];
                        from_ring<kDtype>(in[n][v]).get(x);
                        sum[n][v] = squares(x);
                    }
                scales_of<kLanes, 2>(sum, sub, a.r.eps, r);
            }
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const int h = q0 + (2 * b + n) * step;
                if (2 * b + n >= nq) break;
                float x[2][8];
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    from_ring<kDtype>(in[n][v]).get(x[v]);
                    if (a.r.q_norm) scaled(x[v], r[n], w[v]);
                }
                rotate<kLanes, kPairs>(x, angles, sub, half);
                const int64_t to = (t * a.q_heads + h) * kD + sub * 8;
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    Raw8<kDtype> out;
                    out.set(x[v]);
                    if (here && HC_IN_RANGE(to + v * (kD / 2), 8, static_cast<size_t>(a.tokens) * a.q_heads * kD, status)) out.store(a.q_out, to + v * (kD / 2));
                }
            }
            continue;
        }
        if (b == q_steps && a.r.k_norm) take_weights(a.r.k_norm);
        const int h = k0 + (b - q_steps) * step;
        float x[2][8];
#pragma unroll
        for (int v = 0; v < 2; ++v) from_ring<kDtype>(in[0][v]).get(x[v]);
        if (a.r.k_norm) {
            const float sum[1][2] = {{squares(x[0]), squares(x[1])}};
            float r[1];
            scales_of<kLanes, 1>(sum, sub, a.r.eps, r);
#pragma unroll
            for (int v = 0; v < 2; ++v) scaled(x[v], r[0], w[v]);
        }
        rotate<kLanes, kPairs>(x, angles, sub, half);
        Raw8<HC_DTYPE_FP32> key[2];
#pragma unroll
        for (int v = 0; v < 2; ++v) key[v].set(x[v]);
        const Raw8<kDtype> value[2] = {from_ring<kDtype>(in[1][0]), from_ring<kDtype>(in[1][1])};
        uint32_t sm[2];
        uint2 code[2];
        code[0] = round_group<kLanes>(key, sm[0]);
        code[1] = round_group<kLanes>(value, sm[1]);
        if (!here || slot < 0) continue;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            const int64_t g = group_index(a.c, sh, slot, kv, h, status);
            if (g < 0 || !HC_IN_RANGE(g, 1, group_count(a.c), status)) continue;
            uint32_t* to = reinterpret_cast<uint32_t*>(a.c.codes) + g * (2 * kLanes) + sub;
            to[0] = code[kv].x, to[kLanes] = code[kv].y;
            if (sub == 0) reinterpret_cast<uint32_t*>(a.c.scales)[g] = sm[kv];
        }
    }
    copy_wait<0>();
}

// CTAs that share a tile's heads: those that take the fewest rounds of all resident CTAs, each as long as its
// heads and two more for its start (8191 tokens of 40 heads: 5 CTAs take 34.9 us, 3 36.2, 10 38.9). `resident` are those
// of the kernel that is launched (4099 tokens of 32 + 8 heads half of which are rotated, by halves: 21.7 us, and 27.8 with
// the other kernels' three an SM).
int head_split(int tiles, int heads, int resident) {
    int best = 1;
    int64_t least = -1;
    for (int n = 1; n <= heads && n <= 64; ++n) {
        const int64_t rounds = (static_cast<int64_t>(tiles) * n + resident - 1) / resident, cost = rounds * ((heads + n - 1) / n + 2);
        if (least < 0 || cost < least) least = cost, best = n;
    }
    return best;
}

template <int kD, int kDtype, Pairs kPairs>
cudaError_t call_pairs(const Ctx& ctx, const RotaryArgs& a, cudaStream_t st) {
    constexpr int kTile = kThreads / (kD / 16);
    const int tiles = (a.tokens - 1) / kTile + 1;
    const dim3 grid(tiles, head_split(tiles, a.q_heads + a.c.kv_heads, kCtasPerSm<kPairs> * ctx.sm_count));
    return launch_early(rotary_kernel<kD, kDtype, kPairs>, grid, kThreads, 0, st, a, ctx.s.status);
}

template <int kD, int kDtype>
cudaError_t call(const Ctx& ctx, const RotaryArgs& a, cudaStream_t st) {
    if (a.r.interleaved || a.r.dim == 0) return call_pairs<kD, kDtype, kNeighbours>(ctx, a, st);
    return a.r.dim == kD ? call_pairs<kD, kDtype, kHalves>(ctx, a, st) : call_pairs<kD, kDtype, kPartHalves>(ctx, a, st);
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
