// Log probabilities of given tokens, with the entropy, the rank and the most likely
// alternatives: one pass over the logits, whose bytes bound it.
//
// A CTA takes a row, or a segment of one where there are few rows. Each thread runs over its
// vectors of 16 bytes with sums about a reference of its own, sum e^(x - r) and sum (x - r)
// e^(x - r), and keeps its largest logit and where that was. fp32 has the room to leave
// the reference behind: it moves only when a logit passes it by 40 binary orders. Sums
// of different references join as s e^(r - R) and e^(r - R) (b + s (r - R)).
//
// The alternatives cost the pass next to nothing: with the threads' largest logits known,
// the k-th largest of those is a bound that at least k logits reach, and only the k threads
// that reach it have to look again: at the one vector with their largest, or, where their
// second largest vector reaches the bound too, at all of theirs (a warp reads them in one
// gather; without the second, all k threads did, and half the row's bytes more came from
// DRAM). Logits and their indexes are compared as one number, so that equal logits count
// in the order of their indexes.
//
// Measured: 4096 x 131072 bf16 with the top 20, 201 us, 5.3 TB/s (79% of the copy rate): issue
// bounds it, ALU 56%, FMA 43%, exponentials 29% busy. 8 x 131072 9.1 us, 96 x 50257 fp32 12.4
// us: half of that is the join of the segments and the choice of the top ones.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "hc_window.cuh"

namespace hc {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kAhead = 4;                    // vectors of a thread on their way
constexpr int kList = 2048;                  // candidates that fit; more take the slow way
constexpr float kPass = 27.7f;               // 40 ln 2: by how much a logit may pass the reference
constexpr int kMaxSplits = 64;

// ---- logits

template <int kDtype>
struct Logits;
template <>
struct Logits<HC_DTYPE_FP32> {
    static constexpr int kN = 4;             // of a vector
    static constexpr float kFar = 1e6f;      // references up to which r - 200 is well below r
    using Two = float2;
    static __device__ __forceinline__ Two two(float x) { return make_float2(x, x); }
    static __device__ __forceinline__ float one(const void* p, int64_t i) { return static_cast<const float*>(p)[i]; }
    static __device__ __forceinline__ float at(const uint4& v, int i) {
        return __uint_as_float(i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w);
    }
};
template <>
struct Logits<HC_DTYPE_BF16> {
    static constexpr int kN = 8;
    static constexpr float kFar = 1024.f;    // references up to which fp32 holds x log2(e) - r log2(e) well
    static __device__ __forceinline__ float one(const void* p, int64_t i) { return bf16_lo(static_cast<const uint16_t*>(p)[i]); }
    static __device__ __forceinline__ float at(const uint4& v, int i) {
        const uint32_t w = (i >> 1) == 0 ? v.x : (i >> 1) == 1 ? v.y : (i >> 1) == 2 ? v.z : v.w;
        return (i & 1) ? bf16_hi(w) : bf16_lo(w);
    }
    using Two = __nv_bfloat162;
    // the larger of both, NaN where x is
    static __device__ __forceinline__ Two not_below(Two x, Two low) { return __hmax2_nan(x, low); }
    static __device__ __forceinline__ Two two(float x) { return __float2bfloat162_rn(x); }
    static __device__ __forceinline__ float2 widen(Two x) { return make_float2(__low2float(x), __high2float(x)); }
};
template <>
struct Logits<HC_DTYPE_FP16> {
    static constexpr int kN = 8;
    static constexpr float kFar = 1024.f;    // references up to which fp32 holds x log2(e) - r log2(e) well
    static __device__ __forceinline__ float one(const void* p, int64_t i) { return __half2float(static_cast<const __half*>(p)[i]); }
    static __device__ __forceinline__ float at(const uint4& v, int i) {
        const uint32_t w = (i >> 1) == 0 ? v.x : (i >> 1) == 1 ? v.y : (i >> 1) == 2 ? v.z : v.w;
        const __half2 h = *reinterpret_cast<const __half2*>(&w);
        return (i & 1) ? __high2float(h) : __low2float(h);
    }
    using Two = __half2;
    static __device__ __forceinline__ Two not_below(Two x, Two low) { return __hmax2_nan(x, low); }
    static __device__ __forceinline__ Two two(float x) { return __float2half2_rn(x); }
    static __device__ __forceinline__ float2 widen(Two x) { return __half22float2(x); }
};

// Value, then index, in one whole number that grows with the value and falls with the index
// (0 is below every entry; -0 and 0 are one value).
__device__ __forceinline__ uint64_t order_key(float x, int i) {
    uint32_t u = __float_as_uint(x + 0.0f);
    u = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
    return (static_cast<uint64_t>(u) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(i));
}
__device__ __forceinline__ float key_value(uint64_t k) {
    const uint32_t u = static_cast<uint32_t>(k >> 32);
    return __uint_as_float((u & 0x80000000u) ? (u & 0x7FFFFFFFu) : ~u);
}
__device__ __forceinline__ int key_index(uint64_t k) { return static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(k)); }

// ---- sums about a reference

struct Sums {
    float ref, s, b;
    __host__ __device__ Sums() : ref(-__builtin_huge_valf()), s(0.f), b(0.f) {}
    // to a reference that is at least as large; 0 e^(-inf) is 0
    __device__ __forceinline__ void move(float to) {
        if (ref == to || s == 0.f) {
            ref = to;
            return;
        }
        const float d = ref - to, f = exp2_fast(d * kLog2e);
        b = f == 0.f ? 0.f : f * fmaf(s, d, b);
        s = f * s;
        ref = to;
    }
    __device__ __forceinline__ void add(float x) {               // any logit
        const float d = x - ref;
        const float e = exp2_fast(d * kLog2e);
        s += e;
        if (e != 0.f) b = fmaf(e, d, b);
    }
    __device__ __forceinline__ bool passed(float x) const { return x > ref + kPass; }   // always, at first
};

// ---- the largest 32 of a list of keys

__device__ __forceinline__ uint64_t max64(uint64_t x, uint64_t y) { return x > y ? x : y; }
__device__ __forceinline__ uint64_t min64(uint64_t x, uint64_t y) { return x < y ? x : y; }

// A warp's 32 keys (one a lane), a bitonic sequence, in falling order; and any 32 keys.
__device__ __forceinline__ uint64_t bitonic_merge(uint64_t k, int lane) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const uint64_t o = __shfl_xor_sync(~0u, k, d);
        k = (lane & d) ? min64(k, o) : max64(k, o);
    }
    return k;
}
__device__ __forceinline__ uint64_t bitonic_sort(uint64_t k, int lane) {
#pragma unroll
    for (int n = 2; n < 32; n <<= 1)
#pragma unroll
        for (int d = n >> 1; d > 0; d >>= 1) {
            const uint64_t o = __shfl_xor_sync(~0u, k, d);
            k = (((lane & d) != 0) != ((lane & n) != 0)) ? min64(k, o) : max64(k, o);
        }
    return bitonic_merge(k, lane);
}

// The largest 32 of list[0..n) in falling order, in every warp, a key a lane (0: none). Every
// thread calls it; `list` and `buffer` [kWarps * 32] are shared memory. kFalling: each 32 of
// the list are in falling order already.
template <bool kFalling>
__device__ uint64_t top32(const uint64_t* list, int n, uint64_t* buffer) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint64_t best = 0;
    for (int c = warp * 32; c < n; c += kThreads) {
        uint64_t k = c + lane < n ? list[c + lane] : 0;
        if (!kFalling) k = bitonic_sort(k, lane);
        // the larger of each and its mirror image are the largest 32 of both, in bitonic order
        best = c == warp * 32 ? k : bitonic_merge(max64(best, __shfl_sync(~0u, k, 31 - lane)), lane);
    }
    buffer[threadIdx.x] = best;
    __syncthreads();
    const int lists = min(kWarps, (n + 31) / 32);
#pragma unroll 1
    for (int stride = 1; stride < lists; stride <<= 1) {
        if ((warp & (2 * stride - 1)) == 0 && warp + stride < lists) {
            best = bitonic_merge(max64(best, buffer[(warp + stride) * 32 + 31 - lane]), lane);
            buffer[threadIdx.x] = best;
        }
        __syncthreads();
    }
    best = buffer[lane];
    __syncthreads();
    return best;
}

// The sums of a warp's lanes, in every lane.
__device__ __forceinline__ Sums warp_sums(Sums x) {
    float ref = x.ref;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) ref = fmaxf(ref, __shfl_xor_sync(~0u, ref, d));
    x.move(ref);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        x.s += __shfl_xor_sync(~0u, x.s, d);
        x.b += __shfl_xor_sync(~0u, x.b, d);
    }
    return x;
}

// A segment's result in scratch.
struct alignas(16) Part {
    float ref, s, b;
    int above;
    uint64_t keys[32];
};

template <int kDtype>
__global__ void __launch_bounds__(kThreads, 5)
    score_kernel(const LogprobArgs a, int splits, unsigned char* scratch, unsigned* arrivals, int* status) {
    using L = Logits<kDtype>;
    constexpr int kN = L::kN;
    __shared__ uint64_t list[kList];
    __shared__ uint64_t buffer[kThreads];
    __shared__ float4 warps[kWarps];
    __shared__ int count, last_one;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row = blockIdx.x / splits, split = blockIdx.x % splits;
    constexpr int kItem = kDtype == HC_DTYPE_FP32 ? 4 : 2;
    const unsigned char* x = static_cast<const unsigned char*>(a.logits) + row * a.row * kItem;
    // the row: single logits up to 16-byte alignment, vectors, single logits
    const int head = min(a.vocab, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) / kItem);
    const int vectors = (a.vocab - head) / kN, tail = a.vocab - head - vectors * kN;
    const uint4* vec = reinterpret_cast<const uint4*>(x + head * kItem);
    const int v0 = static_cast<int>(static_cast<int64_t>(vectors) * split / splits);
    const int v1 = static_cast<int>(static_cast<int64_t>(vectors) * (split + 1) / splits);
    // the first logits on their way while the token's is found
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        if (v0 + tid + i * kThreads < v1 && (lane & 7) == 0) prefetch_l2(vec + v0 + tid + i * kThreads);
    // (without asking for the next kernel: its CTAs would lie unevenly over what the SMs have left,
    // 96 rows 14.2 us against 12.1)
    pdl_wait();
    if (!HC_IN_RANGE(row, 1, a.tokens, status)) return;
    const int id = a.ids[row];
    const bool known = id >= 0 && id < a.vocab;
    const float mine = known ? L::one(x, id) : CUDART_INF_F;

    // ---- the pass
    Sums sums;
    float best = -CUDART_INF_F, second = -CUDART_INF_F;
    int best_v = -1;                             // the vector with this thread's largest logit
    int above = 0;
    auto rank_in = [&](float top, int at) {
        second = fmaxf(second, fminf(best, top));
        if (top > best || best_v < 0) best = top, best_v = at;
    };
    // Two at a time, about the reference: 16-bit logits in powers of two (one fma), fp32 ones by
    // their difference (which keeps their last bits)
    float limit = CUDART_NAN_F;                  // what a logit may be without a look at the reference (NaN: none)
    uint64_t s2 = 0, z2 = 0, r2 = 0;             // sums of e and z e (d e), and the reference
    float floor_at = 0.f;       // logits below it count as it: e = 0, and z is finite
    auto fold = [&]() {
        const float2 s = unpair(s2), z = unpair(z2);
        sums.s += s.x + s.y, sums.b = fmaf(z.x + z.y, kDtype == HC_DTYPE_FP32 ? 1.f : kLn2, sums.b);
        s2 = z2 = 0;
    };
    auto vector = [&](const uint4& v, int at, auto& count) {
        if constexpr (kDtype == HC_DTYPE_FP32) {
            const float y[4] = {L::at(v, 0), L::at(v, 1), L::at(v, 2), L::at(v, 3)};
            const float top = fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3]));
            rank_in(top, at);
#pragma unroll
            for (int i = 0; i < 4; ++i) above += y[i] > mine;
            if (!(top <= limit)) {
                fold();
                if (sums.passed(top)) sums.move(top);
#pragma unroll 1
                for (int i = 0; i < 4; ++i)
                    if (sums.ref != -CUDART_INF_F || L::at(v, i) != L::at(v, i)) sums.add(L::at(v, i));
                limit = fabsf(sums.ref) <= L::kFar ? sums.ref + kPass : CUDART_NAN_F;
                floor_at = sums.ref - 200.f;
                r2 = pair(-sums.ref, -sums.ref);
            } else {
                const uint64_t l2 = pair(kLog2e, kLog2e);
#pragma unroll
                for (int i = 0; i < 4; i += 2) {
                    const uint64_t d = add2(pair(max_nan(y[i], floor_at), max_nan(y[i + 1], floor_at)), r2);
                    const float2 z = unpair(mul2(d, l2));
                    const uint64_t e = pair(exp2_fast(z.x), exp2_fast(z.y));
                    s2 = add2(s2, e);
                    z2 = fma2(e, d, z2);
                }
            }
        } else {
            using Two = typename L::Two;
            const Two w[4] = {*reinterpret_cast<const Two*>(&v.x), *reinterpret_cast<const Two*>(&v.y),
                              *reinterpret_cast<const Two*>(&v.z), *reinterpret_cast<const Two*>(&v.w)};
            const float2 hi = L::widen(__hmax2(__hmax2(w[0], w[1]), __hmax2(w[2], w[3])));
            const float top = fmaxf(hi.x, hi.y);
            rank_in(top, at);
            const Two m = L::two(mine);
            count = __hadd2(count, __hadd2(__hadd2(__hgt2(w[0], m), __hgt2(w[1], m)), __hadd2(__hgt2(w[2], m), __hgt2(w[3], m))));
            if (!(top <= limit)) {
                // the first logits, some that pass the reference, NaN, or a reference far from 0
                fold();
                if (sums.passed(top)) sums.move(top);
#pragma unroll 1
                for (int i = 0; i < 8; ++i) {
                    const float y = L::at(v, i);
                    if (sums.ref != -CUDART_INF_F || y != y) sums.add(y);
                }
                limit = fabsf(sums.ref) <= L::kFar ? sums.ref + kPass : CUDART_NAN_F;
                floor_at = sums.ref - 200.f;
                r2 = pair(-sums.ref * kLog2e, -sums.ref * kLog2e);
            } else {
                const uint64_t l2 = pair(kLog2e, kLog2e);
                const Two low = L::two(floor_at);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 y = L::widen(L::not_below(w[i], low));
                    const uint64_t z = fma2(pair(y.x, y.y), l2, r2);
                    const float2 zz = unpair(z);
                    const uint64_t e = pair(exp2_fast(zz.x), exp2_fast(zz.y));
                    s2 = add2(s2, e);
                    z2 = fma2(e, z, z2);
                }
            }
        }
    };
    // (a vector outside of the row counts as one of -inf)
    constexpr uint32_t kNothing = kDtype == HC_DTYPE_FP32 ? 0xFF800000u : kDtype == HC_DTYPE_BF16 ? 0xFF80FF80u : 0xFC00FC00u;
    auto bring = [&](int i) {
        return HC_IN_RANGE(head + static_cast<int64_t>(i) * kN, kN, a.vocab, status) ? ldg_stream_v4(vec + i)
                                                                                      : make_uint4(kNothing, kNothing, kNothing, kNothing);
    };
    using Count = typename L::Two;
    auto count_up = [&](Count& count) {
        if constexpr (kDtype != HC_DTYPE_FP32) {
            const float2 n = L::widen(count);
            above += static_cast<int>(n.x + n.y);
        }
    };
    int at = v0 + tid;
    for (; at + (kAhead - 1) * kThreads < v1; at += kAhead * kThreads) {
        uint4 v[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) v[i] = bring(at + i * kThreads);
        Count count = L::two(0.f);               // at most 4 kAhead: exact
#pragma unroll
        for (int i = 0; i < kAhead; ++i) vector(v[i], at + i * kThreads, count);
        count_up(count);
    }
    for (; at < v1; at += kThreads) {
        Count count = L::two(0.f);
        vector(bring(at), at, count);
        count_up(count);
    }
    fold();
    // the single logits, one a thread, by the first segment's CTA
    const int singles = split == 0 ? head + tail : 0;
    const int single = tid < head ? tid : a.vocab - tail + (tid - head);
    float y1 = -CUDART_INF_F;
    if (tid < singles && HC_IN_RANGE(single, 1, a.vocab, status)) {
        y1 = L::one(x, single);
        if (sums.passed(y1)) sums.move(y1);
        if (sums.ref != -CUDART_INF_F || y1 != y1) sums.add(y1);
        above += y1 > mine;
    }

    // ---- the CTA's sums: of each warp, then in every thread of the warps in order
    sums = warp_sums(sums);
    above = __reduce_add_sync(~0u, above);
    if (lane == 0) warps[warp] = make_float4(sums.ref, sums.s, sums.b, __int_as_float(above));
    // of this thread's largest logit, with the index of its vector's first: vectors of different
    // threads compare by that as their logits do by their own
    uint64_t key = 0;
    if (a.top > 0) {
        if (best_v >= 0) key = order_key(best, head + best_v * kN);
        list[tid] = key;
        if (tid < singles) list[kThreads + tid] = order_key(y1, single);
        if (tid == 0) count = 0;
    }
    __syncthreads();
    {
        Sums all;
        above = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) all.ref = fmaxf(all.ref, warps[w].x);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            Sums one;
            one.ref = warps[w].x, one.s = warps[w].y, one.b = warps[w].z;
            one.move(all.ref);
            all.s += one.s, all.b += one.b;
            above += __float_as_int(warps[w].w);
        }
        sums = all;
    }

    // ---- its largest logits
    uint64_t top = 0;                            // lane i: the i-th
    if (a.top > 0) {
        top = top32<false>(list, kThreads + singles, buffer);
        {
            // every logit that reaches the bound, of the threads and single logits that do
            const uint64_t bound = __shfl_sync(~0u, top, a.top - 1);
            const bool again = key != 0 && key >= bound;
            const uint64_t mine_too = tid < singles ? order_key(y1, single) : 0;
            auto look = [&](int i) {
                if (!HC_IN_RANGE(head + static_cast<int64_t>(i) * kN, kN, a.vocab, status)) return;
                const uint4 v = vec[i];
#pragma unroll
                for (int n = 0; n < kN; ++n) {
                    const float y = L::at(v, n);
                    if (order_key(y, head + i * kN) >= bound) {
                        const int to = atomicAdd(&count, 1);
                        if (to < kList) list[to] = order_key(y, head + i * kN + n);
                    }
                }
            };
            const bool all = again && !(second < key_value(bound));
            if (mine_too != 0 && mine_too >= bound) {
                const int to = atomicAdd(&count, 1);
                if (to < kList) list[to] = mine_too;
            }
            if (again && !all) look(best_v);
            for (uint32_t todo = __ballot_sync(~0u, all); todo != 0; todo &= todo - 1) {
                const int who = warp * 32 + __ffs(todo) - 1;
                for (int i = v0 + who + lane * kThreads; i < v1; i += 32 * kThreads) look(i);
            }
            __syncthreads();
            if (count <= kList) {
                top = top32<false>(list, count, buffer);
            } else {
                // so many only where a few threads have most of the largest logits: one by one
                uint64_t last = ~0ull;
                for (int n = 0; n < a.top; ++n) {
                    uint64_t next = mine_too < last ? mine_too : 0;
                    for (int i = v0 + tid; i < v1; i += kThreads) {
                        if (!HC_IN_RANGE(head + static_cast<int64_t>(i) * kN, kN, a.vocab, status)) continue;
                        const uint4 v = vec[i];
                        for (int m = 0; m < kN; ++m) {
                            const uint64_t k = order_key(L::at(v, m), head + i * kN + m);
                            if (k < last) next = max64(next, k);
                        }
                    }
                    buffer[tid] = next;
                    __syncthreads();
                    for (int d = kThreads / 2; d > 0; d >>= 1) {
                        if (tid < d) buffer[tid] = max64(buffer[tid], buffer[tid + d]);
                        __syncthreads();
                    }
                    last = buffer[0];
                    __syncthreads();
                    if (lane == n) top = last;
                }
            }
        }
    }

    // ---- segments joined by the last of them
    if (splits > 1) {
        Part* parts = reinterpret_cast<Part*>(scratch) + static_cast<int64_t>(row) * splits;
        if (warp == 0) {
            if (lane == 0) __stcg(reinterpret_cast<float4*>(&parts[split]), make_float4(sums.ref, sums.s, sums.b, __int_as_float(above)));
            if (lane < a.top)
                __stcg(reinterpret_cast<unsigned long long*>(&parts[split].keys[lane]), static_cast<unsigned long long>(top));
            __syncwarp();
            if (lane == 0) {
                last_one = arrive(&arrivals[row]) == static_cast<unsigned>(splits - 1);
                if (last_one) arrivals[row] = 0;                 // for the next launch
            }
        }
        __syncthreads();
        if (!last_one) return;
        // the segments' largest, on their way while their sums are joined
        for (int i = tid; a.top > 0 && i < splits * 32; i += kThreads)
            list[i] = (i & 31) < a.top ? __ldcg(reinterpret_cast<const unsigned long long*>(&parts[i >> 5].keys[i & 31])) : 0;
        // the segments' sums, two a lane at most, in a fixed order
        Sums mine_of[2];
        above = 0;
#pragma unroll
        for (int n = 0; n < kMaxSplits / 32; ++n) {
            if (lane + 32 * n >= splits) continue;
            const float4 x = __ldcg(reinterpret_cast<const float4*>(&parts[lane + 32 * n]));
            mine_of[n].ref = x.x, mine_of[n].s = x.y, mine_of[n].b = x.z;
            above += __float_as_int(x.w);
        }
        const float ref = fmaxf(mine_of[0].ref, mine_of[1].ref);
        mine_of[0].move(ref), mine_of[1].move(ref);
        mine_of[0].s += mine_of[1].s, mine_of[0].b += mine_of[1].b;
        sums = warp_sums(mine_of[0]);
        above = __reduce_add_sync(~0u, above);
        if (a.top > 0) {
            __syncthreads();
            top = top32<true>(list, splits * 32, buffer);
        }
    }

    // ---- results
    const bool empty = sums.ref == -CUDART_INF_F && sums.s == 0.f;         // -inf alone
    const float ln_s = logf(sums.s), lse = empty ? -CUDART_INF_F : sums.ref + ln_s;
    // y - lse, by the difference from the reference: beside a large one fp32 does not hold the logarithm
    // (a row of the type's lowest value alone is as likely everywhere, -ln vocab)
    auto logprob = [&](float y) {
        if (y == -CUDART_INF_F && lse == lse && lse != CUDART_INF_F) return y;
        return lse == CUDART_INF_F ? CUDART_NAN_F : (y - sums.ref) - ln_s;
    };
    if (tid == 0) {
        a.lse[row] = lse;
        a.logprob[row] = known ? logprob(mine) : lse == lse ? -CUDART_INF_F : lse;
        a.entropy[row] = empty ? 0.f : ln_s - sums.b / sums.s;
        a.rank[row] = known ? above : a.vocab;
    }
    if (warp == 0 && lane < a.top) {
        a.top_ids[static_cast<int64_t>(row) * a.top + lane] = key_index(top);
        a.top_logprobs[static_cast<int64_t>(row) * a.top + lane] = logprob(key_value(top));
    }
}

// The segments of a row, where there are too few rows to fill the GPU: twice as many CTAs as
// SMs, but no segment below the vectors that a CTA's threads have on their way at once (8 x
// 131072 bf16: 16 segments a row took 10.3 us, 38 took 15.3).
int row_splits(int sm_count, int rows, int vocab, int vector) {
    const int want = (2 * sm_count + rows - 1) / rows, most = vocab / (kThreads * kAhead * vector);
    int n = want < most ? want : most;
    if (n > kMaxSplits) n = kMaxSplits;
    return rows >= 2 * sm_count || n < 1 ? 1 : n;
}

}  // namespace

size_t score_scratch_bytes(int sm_count) { return static_cast<size_t>(4) * sm_count * sizeof(Part); }

cudaError_t launch_logprobs(const Ctx& ctx, const LogprobArgs& a, int dtype, cudaStream_t st) {
    const int splits = row_splits(ctx.sm_count, a.tokens, a.vocab, dtype == HC_DTYPE_FP32 ? 4 : 8);
    const unsigned grid = static_cast<unsigned>(a.tokens) * splits;
    switch (dtype) {
        case HC_DTYPE_BF16: return launch_early(score_kernel<HC_DTYPE_BF16>, dim3(grid), kThreads, 0, st, a, splits, ctx.score_parts, ctx.score_arrivals, ctx.s.status);
        case HC_DTYPE_FP16: return launch_early(score_kernel<HC_DTYPE_FP16>, dim3(grid), kThreads, 0, st, a, splits, ctx.score_parts, ctx.score_arrivals, ctx.s.status);
        default: return launch_early(score_kernel<HC_DTYPE_FP32>, dim3(grid), kThreads, 0, st, a, splits, ctx.score_parts, ctx.score_arrivals, ctx.s.status);
    }
}

}  // namespace hc
