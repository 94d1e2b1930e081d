// Tokens drawn from logits with temperature, top-k, top-p and min-p.
//
// Weights are whole numbers, multiples of 2^-45 of the largest, so that sums are exact and the
// same in any order: which token a uniform number falls on, and where a filter cuts, are decided
// by comparing whole numbers.
//
// exp((x - M) / T) = 2^z. 32 z = x c - M c, c = 32 log2(e) / T, is cut into a whole number m and a
// rest g by one fma that rounds x c to a whole number and a second that leaves what that lacks: 2^z =
// 2^(m / 32) (1 + p(g)), the first from a table of 32 bits (32 words: no two lanes that look up different ones
// meet on a bank), p by its series to the fourth power (2^-34), held to 2^-28. c and M c are two floats each. In
// all 2^-27 of a weight.
//
// A row belongs to a cluster of CTAs, which hold it in their shared memory: it is read once. What
// the filters leave is found in steps that look at less and less of it:
//
// * the largest logit; for a top-p without a top-k also the sum of all weights
// * an estimate, from an eighth of the logits, of a bound above which what stays must lie, and a list
//   of the logits above it; where they turn out too few, a deeper bound is taken, at last that of all
//   that have weight
// * counts and weights of the listed logits by value, in 256 bins; those of the bin in which the border
//   lies again, in bins 256 times as narrow, until one value is left. Of equal logits the first ones in
//   the order of their ids stay, so that a border is a value and how many of it stay.
// * the sum of what stays by CTA, warp and lane, in the order of the ids, down to the token.
//
// Each step ends in a barrier of the cluster, after which every CTA reads what the others found and
// comes to the same end. A short list is handed to the first CTA, which ends the row alone. Lists and
// rows are gone through in the order of the ids, by each warp its part.
//
// Measured: rows of 131072 bf16 logits, 8 and 512 of them: the largest 3.5 and 35 us, no filter 9.5 and 101, a top-50
// 8.1 and 79, a top-1000 16 and 136, a top-p of 0.5 18 and 177, of 0.95 24 and 271; 512 of mixed settings 126 to 146 us
// by the draw of these, 1.0 TB/s; 96 of 50257 in fp32 33 to 52, by the slowest row. The logits are read once (20 us of it at the copy rate). Few rows wait at barriers (a cluster's takes
// some 0.5 us, a filter has 6 to 10); many are bound by issue (38% of the slots, four CTAs an SM wait for one
// another) and by the weights, 64-bit arithmetic.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stddef.h>
#include <stdint.h>

#include <type_traits>

#include "hc_serve_internal.h"
#include "hc_window.cuh"

namespace cg = cooperative_groups;

namespace hc {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = kThreads;              // a thread a bin when they are summed
constexpr int kBinBits = 8;
constexpr int kShort = 1408;                 // logits of a list that one CTA takes
constexpr int kUnitBits = 45;
constexpr uint64_t kOne = 1ull << kUnitBits;
constexpr int kMaxCtas = 8;                  // of a cluster
constexpr int kSteps = 32;                   // of the table, an octave
constexpr float kRound = 12582912.f;         // 1.5 2^23
constexpr float kDeep = -46.5f;              // log2 of weights that are 0
constexpr float kTop = 3.402823466e38f;
// A temperature above kHot, and the logits with it, are weighed as 2^-64 of themselves: M - x and 46.5 T ln 2 pass fp32's
// range there, and c falls below its normal numbers. (The logits that 2^-64 makes subnormal are all 0 beside such a T.)
constexpr float kHot = 18446744073709551616.f, kCooled = 1.f / kHot;
static_assert(HC_SAMPLE_MAX_VOCAB <= kMaxCtas * 32768);

// 2^(j / 32) 2^31
__device__ const uint32_t kPowers[kSteps] = {
    0x80000000u, 0x82CD8699u, 0x85AAC368u, 0x88980E81u, 0x8B95C1E4u, 0x8EA4398Bu, 0x91C3D374u, 0x94F4EFA9u,
    0x9837F052u, 0x9B8D39BAu, 0x9EF53261u, 0xA2704303u, 0xA5FED6AAu, 0xA9A15AB5u, 0xAD583EEAu, 0xB123F582u,
    0xB504F334u, 0xB8FBAF47u, 0xBD08A39Fu, 0xC12C4CCAu, 0xC5672A11u, 0xC9B9BD86u, 0xCE248C15u, 0xD2A81D92u,
    0xD744FCCBu, 0xDBFBB798u, 0xE0CCDEECu, 0xE5B906E7u, 0xEAC0C6E8u, 0xEFE4B99Cu, 0xF5257D15u, 0xFA83B2DBu,
};

// Logits in shared memory.
template <int kDtype>
__device__ __forceinline__ float logit(const void* p, int i) {
    if (kDtype == HC_DTYPE_FP32) return static_cast<const float*>(p)[i];
    const uint16_t u = static_cast<const uint16_t*>(p)[i];
    return kDtype == HC_DTYPE_BF16 ? __uint_as_float(static_cast<uint32_t>(u) << 16) : __half2float(__ushort_as_half(u));
}

// A number that grows with x, without the bits that a 16-bit type's fp32 patterns do not use.
template <int kDtype>
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t u = __float_as_uint(x + 0.0f);
    const uint32_t k = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
    return kDtype == HC_DTYPE_BF16 ? k >> 16 : kDtype == HC_DTYPE_FP16 ? k >> 13 : k;
}

template <int kDtype>
__device__ __forceinline__ float value_of(uint32_t key) {
    // (a negative value's pattern is the complement of its key: its unused bits are zeros)
    constexpr int kUnused = kDtype == HC_DTYPE_BF16 ? 16 : kDtype == HC_DTYPE_FP16 ? 13 : 0;
    const uint32_t k = key << kUnused;
    return __uint_as_float((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k & ~((1u << kUnused) - 1u));
}

// A row's temperature and largest logit, as the weights need them.
struct Heat {
    float c, c_low, a, rest;                 // c in two floats; 1.5 2^23 - rint(M c); what makes g(M) 0
    float top, deep;                         // M; the logit below which weights are 0 (-kTop: of finite ones perhaps none)
    bool far;                                // M c is beyond what a rounds well, or T above kHot (c is not used then)
};
constexpr float kHi = 1.44269502f, kLo = 1.92596299e-8f;     // log2(e)
// (In fp32 alone: 64-bit operations took 15 us of a row's 40.)
__device__ __forceinline__ Heat heat_of(float t, float top) {
    Heat h;
    const float z = kHi / t, z_low = (fmaf(-z, t, kHi) + kLo) / t;
    h.c = z * kSteps, h.c_low = z_low * kSteps;
    // M's own weight is 2^45: its m is 0, and so is its g to 2^-25, whose p is held as 0
    const float at = h.c * top;
    float whole = rintf(at);
    whole += fmaf(top, h.c, kRound - whole) - kRound;
    h.a = kRound - whole;
    h.rest = fmaf(-h.c_low, top, -fmaf(top, h.c, -whole));
    h.top = top;
    h.deep = fmaxf(fmaf(t, kDeep * kLn2, top), -kTop);                   // never -inf
    // (a word of which the compiler knows nothing: what it made of the comparisons in all that follows took 5 us of the
    // 142 of 512 rows)
    unsigned far = !(fabsf(at) < 1000000.f && t <= kHot);
    asm volatile("" : "+r"(far));
    h.far = far != 0;
    return h;
}

// Whole numbers times an fp32 factor in [0, 1), rounded down or up, exactly.
__device__ __forceinline__ uint64_t part_of(uint64_t x, float by, bool up) {
    const uint32_t bits = __float_as_uint(by), e = bits >> 23;
    const uint64_t m = (bits & 0x7FFFFFu) | (e ? 0x800000u : 0u);
    const int down = e ? 150 - static_cast<int>(e) : 149;                // by = m 2^-down, 24 <= down
    const uint64_t lo = x * m, hi = __umul64hi(x, m);
    uint64_t r = 0, rest = lo | hi;
    if (down < 64) r = (hi << (64 - down)) | (lo >> down), rest = lo << (64 - down);
    else if (down < 128) r = down == 64 ? hi : hi >> (down - 64), rest = lo | (down == 64 ? 0 : hi << (128 - down));
    return r + (up && rest != 0);
}

// The least weight that a min-p leaves.
__device__ __forceinline__ uint64_t least_weight(float least) {
    return !(least > 0.f) ? 1 : least < 1.f ? max(part_of(kOne, least, true), static_cast<uint64_t>(1)) : kOne;
}

// 2^((m + g) / 32) in multiples of 2^-45, -47 32 <= m <= 1, of `bits` = m + the pattern of kRound and
// `part` = 2^27 p(g) + that pattern.
__device__ __forceinline__ uint64_t power(int bits, int part, const uint32_t* powers) {
    constexpr int kPattern = 0x4B400000, kStepBits = 5;
    static_assert(kSteps == 1 << kStepBits);
    const uint64_t w = static_cast<uint64_t>(powers[bits & (kSteps - 1)]) * static_cast<uint32_t>(part - kPattern + (1 << 27));     // 2^31 2^27
    return w >> (58 - kUnitBits + (kPattern >> kStepBits) - (bits >> kStepBits));
}
// p(g) = 2^(g / 32) - 1 in multiples of 2^-27, behind kRound: (g l) + (g l)^2 / 2 + ..., l = ln 2 / 32; |g| <= 1.2, |p| < 2^-5
constexpr float kP1 = 2.1660849392e-2f, kP2 = 2.3459619820e-4f, kP3 = 1.6938509724e-6f, kP4 = 9.1725627018e-9f, kPart = 134217728.f;
// The weights of two logits, 0 below h.deep. Two fp32 operations in one instruction.
__device__ __forceinline__ void weights(float x0, float x1, const Heat& h, const uint32_t* powers, uint64_t& w0, uint64_t& w1) {
    const uint64_t x = pair(fmaxf(x0, h.deep), fmaxf(x1, h.deep)), c = pair(h.c, h.c), a = pair(h.a, h.a);
    const uint64_t v = fma2(x, c, a);
    const uint64_t g = add2(fma2(x, c, fma2(v, pair(-1.f, -1.f), a)), fma2(x, pair(h.c_low, h.c_low), pair(h.rest, h.rest)));
    const uint64_t p = mul2(g, fma2(g, fma2(g, fma2(g, pair(kP4, kP4), pair(kP3, kP3)), pair(kP2, kP2)), pair(kP1, kP1)));
    const float2 bits = unpair(v), part = unpair(fma2(p, pair(kPart, kPart), pair(kRound, kRound)));
    w0 = power(__float_as_int(bits.x), __float_as_int(part.x), powers);
    w1 = power(__float_as_int(bits.y), __float_as_int(part.y), powers);
}
// Where M c or T is so large that this way loses bits: from the difference to M, in two floats. 0 of -inf. What it needs of
// the row lies in shared memory, since registers are short.
struct Far {
    float by, c, c_low;                      // 1, or 2^-64 of a hot row; log2(e) / (by T) in two floats
};
__device__ __noinline__ void far_of(float t, Far* to) {
    const float by = t > kHot ? kCooled : 1.f, cool = t * by, c = kHi / cool;
    to->by = by, to->c = c, to->c_low = (fmaf(-c, cool, kHi) + kLo) / cool;
}
__device__ __noinline__ uint64_t weight_far(float x, float top, const Far* far, const uint32_t* powers) {
    const float by = far->by, c = far->c, c_low = far->c_low;
    x *= by, top *= by;
    const float d = __fsub_rn(x, top), z = __fmul_rn(d, c);
    if (!(z > kDeep)) return 0;
    const float b = __fsub_rn(d, x);
    const float dl = __fsub_rn(__fsub_rn(x, __fsub_rn(d, b)), __fadd_rn(top, b));     // x - top = d + dl
    const float zl = fmaf(dl, c, fmaf(d, c_low, fmaf(d, c, -z)));
    const float v = fmaf(z, kSteps, kRound);
    const float g = fmaf(z, kSteps, kRound - v) + zl * kSteps;
    const float p = g * fmaf(g, fmaf(g, fmaf(g, kP4, kP3), kP2), kP1);
    return power(__float_as_int(v), __float_as_int(fmaf(p, kPart, kRound)), powers);
}

// ln of a weight, by halves: a difference of logits may pass fp32's range where that over T does not.
__device__ __forceinline__ float log_weight(float x, float top, float t) { return (0.5f * x - 0.5f * top) / t * 2.f; }

template <typename T>
__device__ __forceinline__ T warp_sum(T x) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(~0u, x, d);
    return x;
}
// Sums of the lanes up to and with this one.
template <typename T>
__device__ __forceinline__ T warp_scan(T x, int lane) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const T y = __shfl_up_sync(~0u, x, d);
        if (lane >= d) x += y;
    }
    return x;
}

template <int kDtype>
struct Shared {
    uint32_t powers[kSteps];
    // of a step's bins: their logits, and their weights as sums of each 16 bits of them (shared memory adds
    // 32 bits at a time by itself: three such sums take 8 cycles a warp, one of 64 bits 50 to 570)
    unsigned count[kBins];
    alignas(uint64_t) unsigned mass[3][kBins];           // (taken as 64-bit words by finish_alone)
    // what the warps tell the cluster
    alignas(16) uint64_t told_mass[kWarps];
    alignas(16) unsigned told_count[kWarps];
    alignas(16) float told_top[kWarps];
    Far far;                                 // of a row whose weights are found that way
    float u, p, t, least;                    // the row's settings, for where they are needed again (registers are short)
    // within the CTA
    uint64_t warp_mass[kWarps];
    unsigned warp_count[kWarps];
    uint64_t before_mass, in_mass;           // of the bin with the border
    unsigned before, in;
    int warp_first[kWarps], warp_begin[kWarps], warp_n[kWarps];
    // a short list: ids and values; before it, the bins of the estimate lie in the first
    int id[kShort];
    typename std::conditional<kDtype == HC_DTYPE_FP32, float, uint16_t>::type value[kShort];
};

// What the warps of a cluster have told, two warps a lane, in their order: CTA lane / 4, warps 2 (lane % 4) and the
// next. Lanes past the CTAs get `none`.
template <typename T>
struct Two {
    T x, y;
};
template <typename T, int kDtype>
__device__ __forceinline__ Two<T> of_warps(cg::cluster_group& cluster, int ctas, int lane, Shared<kDtype>& s, T (Shared<kDtype>::*told)[kWarps], T none) {
    static_assert(kWarps == 8, "four lanes a CTA");
    const bool there = lane < 4 * ctas;
    const Shared<kDtype>* o = ctas == 1 ? &s : cluster.map_shared_rank(&s, there ? lane >> 2 : 0);
    const T* p = (o->*told) + 2 * (lane & 3);
    return there ? Two<T>{p[0], p[1]} : Two<T>{none, none};
}

// The two halves of a cluster's barrier.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait;" ::: "memory"); }

// Logits above `at` stay, and of those equal to it the first `ties`.
struct Cut {
    float at;
    unsigned ties;
    uint64_t above;                          // weight of those above
};

// Packed maxima, NaN where one is.
template <int kDtype>
struct Most {
    float m = -__builtin_huge_valf();
    __device__ __forceinline__ void take(const uint4& v) {
        m = max_nan(m, max_nan(max_nan(__uint_as_float(v.x), __uint_as_float(v.y)), max_nan(__uint_as_float(v.z), __uint_as_float(v.w))));
    }
    __device__ __forceinline__ float get() const { return m; }
};
template <typename Two>
__device__ __forceinline__ Two two_of(uint32_t w) { return *reinterpret_cast<const Two*>(&w); }
template <>
struct Most<HC_DTYPE_BF16> {
    __nv_bfloat162 m = __float2bfloat162_rn(-__builtin_huge_valf());
    __device__ __forceinline__ void take(const uint4& v) {
        using Two = __nv_bfloat162;
        m = __hmax2_nan(m, __hmax2_nan(__hmax2_nan(two_of<Two>(v.x), two_of<Two>(v.y)), __hmax2_nan(two_of<Two>(v.z), two_of<Two>(v.w))));
    }
    __device__ __forceinline__ float get() const { return max_nan(__low2float(m), __high2float(m)); }
};
template <>
struct Most<HC_DTYPE_FP16> {
    __half2 m = __float2half2_rn(-__builtin_huge_valf());
    __device__ __forceinline__ void take(const uint4& v) {
        using Two = __half2;
        m = __hmax2_nan(m, __hmax2_nan(__hmax2_nan(two_of<Two>(v.x), two_of<Two>(v.y)), __hmax2_nan(two_of<Two>(v.z), two_of<Two>(v.w))));
    }
    __device__ __forceinline__ float get() const { return max_nan(__low2float(m), __high2float(m)); }
};
// The logits of a vector.
template <int kDtype>
__device__ __forceinline__ void unpack(const uint4& v, float (&y)[kDtype == HC_DTYPE_FP32 ? 4 : 8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if constexpr (kDtype == HC_DTYPE_FP32) {
            y[e] = __uint_as_float(w[e]);
        } else {
            const float2 f = widen2<kDtype>(w[e]);
            y[2 * e] = f.x, y[2 * e + 1] = f.y;
        }
    }
}

// The end of a row of which at most kThreads logits are left, in one CTA, a logit a thread: each counts and weighs
// those before it. `want`: the weight of a top-p alone (`whole`: it follows from the list's). (A row of a top-50 among
// 131072 13.4 us in bins, 9.1 so.)
template <int kDtype, typename Weigh>
__device__ __forceinline__ void finish_alone(Shared<kDtype>& s, const SampleArgs& a, int row, int n, int k, bool by_count, bool by_mass, bool whole,
                                             uint64_t want, float top, Weigh& weigh) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // the bins' room is free: values and weights of the list
    float* value = reinterpret_cast<float*>(s.count);
    uint64_t* mass = reinterpret_cast<uint64_t*>(s.mass);
    static_assert(sizeof(s.count) >= kThreads * sizeof(float) && sizeof(s.mass) >= kThreads * sizeof(uint64_t));
    static_assert(offsetof(Shared<kDtype>, mass) % alignof(uint64_t) == 0 && alignof(Shared<kDtype>) % alignof(uint64_t) == 0);
    const float y[4] = {tid < n ? logit<kDtype>(s.value, tid) : -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
    uint64_t w[4];
    weigh(y, w);
    value[tid] = y[0], mass[tid] = w[0];
    __syncthreads();
    // sums over the CTA: in every thread; up to and with this one
    auto sum_of = [&](uint64_t x) {
        x = warp_sum(x);
        if (lane == 0) s.warp_mass[warp] = x;
        __syncthreads();
        x = 0;
        for (int i = 0; i < kWarps; ++i) x += s.warp_mass[i];
        __syncthreads();
        return x;
    };
    const uint64_t low = least_weight(s.least);
    unsigned rank = 0;
    uint64_t before = 0;
    if (warp * 32 < n) {
#pragma unroll 4
        for (int j = 0; j < n; ++j) {
            const bool first = j < tid ? value[j] >= y[0] : value[j] > y[0];
            rank += first;
            if (by_mass) before += first ? mass[j] : 0;
        }
    }
    bool stays = tid < n && w[0] >= low && (!by_count || rank < static_cast<unsigned>(k));
    if (by_mass) {
        if (by_count) want = max(part_of(sum_of(tid < n && rank < static_cast<unsigned>(k) ? w[0] : 0), fmaxf(s.p, 0.f), true), static_cast<uint64_t>(1));
        else if (whole) want = max(part_of(sum_of(w[0]), fmaxf(s.p, 0.f), true), static_cast<uint64_t>(1));
        stays = stays && before < want;
    }
    const uint64_t kept = stays ? w[0] : 0;
    uint64_t upto = warp_scan(kept, lane);
    if (lane == 31) s.warp_mass[warp] = upto;
    __syncthreads();
    uint64_t total = 0;
    for (int i = 0; i < kWarps; ++i) {
        if (i == warp) upto += total;
        total += s.warp_mass[i];
    }
    const uint64_t goal = s.u < 1.f ? part_of(total, fmaxf(s.u, 0.f), false) : total - 1;
    if (upto > goal && upto - kept <= goal) {
        a.ids[row] = s.id[tid];
        a.logprob[row] = log_weight(y[0], top, s.t) - logf(static_cast<float>(total) * (1.f / kOne));
    }
}

template <int kDtype>
__global__ void __launch_bounds__(kThreads, kDtype == HC_DTYPE_FP32 ? 3 : 4) sample_kernel(const SampleArgs a, int ctas, int segment_bytes, int list_room, int* status) {
    constexpr int kItem = kDtype == HC_DTYPE_FP32 ? 4 : 2, kN = 16 / kItem;
    using S = Shared<kDtype>;
    __shared__ S s;
    extern __shared__ __align__(16) unsigned char smem[];
    unsigned char* segment = smem;
    uint16_t* list = reinterpret_cast<uint16_t*>(smem + segment_bytes);
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int log_ctas = 31 - __clz(ctas);       // (a power of two)
    const int row = blockIdx.x >> log_ctas, rank = blockIdx.x & (ctas - 1);
    begin_early();
    // (the whole cluster has one row, so that all of it leaves together)
    if (!HC_IN_RANGE(row, 1, a.tokens, status)) return;

    // on their way together with the row
    const float u = a.uniform[row], t = a.temperature ? a.temperature[row] : 1.f;
    const float p = a.top_p ? a.top_p[row] : 1.f, least = a.min_p ? a.min_p[row] : 0.f;
    const int k = a.top_k ? a.top_k[row] : 0;
    const uint32_t power_of = kPowers[lane];
    static_assert(kSteps == 32);

    // ---- the CTA's part of the row: whole vectors of 16 bytes, with -inf for what lies around the row
    const unsigned char* x = static_cast<const unsigned char*>(a.logits) + row * a.row * kItem;
    const int shift = static_cast<int>(reinterpret_cast<uintptr_t>(x) & 15) / kItem;
    const int vectors = (shift + a.vocab + kN - 1) / kN;
    const int v0 = (vectors * rank) >> log_ctas, v1 = (vectors * (rank + 1)) >> log_ctas;
    const int id0 = v0 * kN - shift;             // the id of local index 0
    uint4* const vec = reinterpret_cast<uint4*>(segment);
    // whole vectors by asynchronous copies, all on their way at once; the ends of the row by one thread each
    const int n_vec = v1 - v0, w0 = id0 < 0 ? 1 : 0, w1 = id0 + n_vec * kN > a.vocab ? n_vec - 1 : n_vec;
    {
        const uint4* from = reinterpret_cast<const uint4*>(x - shift * kItem) + v0;
#pragma unroll 4
        for (int i = w0 + tid; i < w1; i += kThreads)
            if (HC_IN_RANGE(id0 + i * kN, kN, a.vocab, status)) copy16(tc::smem_u32(vec + i), from + i);
        copy_commit();
    }
    bool bad = !(u == u && p == p && least == least) || !(fabsf(t) <= kTop);
    s.count[tid] = s.mass[0][tid] = s.mass[1][tid] = s.mass[2][tid] = 0, s.id[tid] = 0;
    Most<kDtype> largest;
    const int end = tid == 0 && w0 > 0 ? 0 : tid == 32 && w1 < n_vec && n_vec > w0 ? n_vec - 1 : -1;
    if (end >= 0) {
        for (int e = 0; e < kN; ++e) {
            const int id = id0 + end * kN + e;
            const bool in = id >= 0 && id < a.vocab;
            if (kItem == 4) reinterpret_cast<uint32_t*>(vec + end)[e] = in ? reinterpret_cast<const uint32_t*>(x)[id] : 0xFF800000u;
            else reinterpret_cast<uint16_t*>(vec + end)[e] = in ? reinterpret_cast<const uint16_t*>(x)[id] : static_cast<uint16_t>(kDtype == HC_DTYPE_BF16 ? 0xFF80u : 0xFC00u);
        }
        largest.take(vec[end]);
    }
    copy_wait<0>();
#pragma unroll 4
    for (int i = w0 + tid; i < w1; i += kThreads) largest.take(vec[i]);
    const float my_most = largest.get();         // of this thread's logits
    float most = my_most;

    // ---- the largest logit
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) most = max_nan(most, __shfl_xor_sync(~0u, most, d));
    if (lane == 0) s.told_top[warp] = most;
    if (tid < kSteps) s.powers[tid] = power_of;
    if (tid == 0) s.u = u, s.p = p, s.t = t, s.least = least;
    cluster.sync();
    const Two<float> tops = of_warps<float>(cluster, ctas, lane, s, &S::told_top, -CUDART_INF_F);
    float top = max_nan(tops.x, tops.y);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = max_nan(top, __shfl_xor_sync(~0u, top, d));
    bad = bad || !(fabsf(top) <= kTop);
    // each warp's part of the segment
    const int all = (v1 - v0) * kN, per = ((v1 - v0 + kWarps - 1) / kWarps) * kN;
    const int part_begin = min(warp * per, all), part_end = min(part_begin + per, all);
    if (bad || t < 5.421010862427522e-20f) {
        // nothing, or the first of the largest: the first CTA that has it finds it
        const unsigned with = __ballot_sync(~0u, tops.x == top || tops.y == top);
        cluster_arrive();                        // all have read what the others told: they wait for it in the end
        if (bad ? rank == 0 : rank == (__ffs(with) - 1) / 4) {
            int first = 0x7FFFFFFF;
            if (!bad)
                for (int i = part_begin / kN + lane; i < part_end / kN; i += 32) {
                    float y[kN];
                    unpack<kDtype>(vec[i], y);
#pragma unroll
                    for (int e = 0; e < kN; ++e)
                        if (y[e] == top) first = min(first, id0 + i * kN + e);
                }
            first = __reduce_min_sync(~0u, first);
            if (lane == 0) s.warp_first[warp] = first;
            __syncthreads();
            if (tid == 0) {
                for (int w = 1; w < kWarps; ++w) first = min(first, s.warp_first[w]);
                a.ids[row] = bad ? -1 : first;
                a.logprob[row] = bad ? CUDART_NAN_F : 0.f;
            }
        }
        cluster_wait();
        return;
    }
    const Heat heat = heat_of(t, top);
    if (heat.far) far_of(t, &s.far);             // (all threads the same)
    const bool by_count = k > 0 && k < a.vocab, by_mass = p < 1.f;
    // a warp's sum, told to the cluster
    auto tell_mass = [&](uint64_t mass) {
        mass = warp_sum(mass);
        if (lane == 0) s.told_mass[warp] = mass;
    };
    auto all_mass = [&]() {
        const Two<uint64_t> told = of_warps<uint64_t>(cluster, ctas, lane, s, &S::told_mass, 0);
        return warp_sum(told.x + told.y);
    };

    // The logits that this warp goes through, four a lane at a time: all of its part, those listed of it, or
    // its share of the short list.
    enum { kAll, kListed, kAlone } mode = kAll;
    int n = part_end - part_begin, begin = part_begin;
    uint16_t* mine = list + warp * list_room;
    auto value_at = [&](int i) {
        if (mode == kAlone) return logit<kDtype>(s.value, begin + i);
        return logit<kDtype>(segment, mode == kListed ? static_cast<int>(mine[i]) : begin + i);
    };
    auto each = [&](auto use) {
        for (int i = lane; i < n; i += 128) {
            float y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = i + 32 * e < n ? value_at(i + 32 * e) : -CUDART_INF_F;
            use(y);
        }
    };
    // (in no order)
    auto each_of_all = [&](auto use) {
        for (int i = part_begin / kN + lane; i < part_end / kN; i += 32) {
            float y[kN];
            unpack<kDtype>(vec[i], y);
#pragma unroll
            for (int e = 0; e < kN; e += 4) {
                const float z[4] = {y[e], y[e + 1], y[e + 2], y[e + 3]};
                use(z);
            }
        }
    };
    // and their weights, 0 for those at -inf
    auto weigh2 = [&](float y0, float y1, uint64_t& w0, uint64_t& w1) {
        if (heat.far) {
            w0 = weight_far(y0, top, &s.far, s.powers);
            w1 = weight_far(y1, top, &s.far, s.powers);
        } else {
            weights(y0, y1, heat, s.powers, w0, w1);
        }
    };
    auto weigh = [&](const float (&y)[4], uint64_t (&w)[4]) { weigh2(y[0], y[1], w[0], w[1]), weigh2(y[2], y[3], w[2], w[3]); };
    // the end of a step
    auto sync = [&]() {
        if (mode == kAlone) __syncthreads();
        else cluster.sync();
    };
    Cut cut = {-CUDART_INF_F, 0, 0};             // all stay
    if (by_count || by_mass) {
        const bool few = a.vocab <= kShort;                             // they go to one CTA without an estimate
        const float width = -kDeep / kBins * kLn2 * t;                  // of an estimate's bin, in logits
        uint64_t total = 0, want = k, mass = 0, upto = 0;
        float estimated = 0.f, estimated_upto = 0.f;
        unsigned number = 0;
        float bound;
        const bool by_largest = by_count && k <= kThreads / 2 * ctas;
        if (!few) {
            // ---- the threads' largest logits (at least as many logits lie above a bound), or an eighth of all, by how
            // far they lie below the largest, in bins of an octave / 5.5
            const float per_logit = 1.f / width;
            auto add_depth = [&](float y) {
                const float z = (top - y) * per_logit;
                if (z < static_cast<float>(kBins)) atomicAdd(&s.id[min(static_cast<int>(z), kBins - 1)], 1);
            };
            if (by_largest) add_depth(my_most);
            else
                for (int i = tid; i < all / 8; i += kThreads) add_depth(logit<kDtype>(segment, i * 8 + (i & 7)));
            auto add_up = [&](const float (&y)[4]) {
                uint64_t w[4];
                weigh(y, w);
                total += (w[0] + w[1]) + (w[2] + w[3]);
            };
            if (!by_count) {
                each_of_all(add_up);
                tell_mass(total);
            }
            cluster.sync();
            if (!by_count) total = all_mass();
            unsigned theirs[kMaxCtas];
#pragma unroll
            for (int r = 0; r < kMaxCtas; ++r) theirs[r] = r < ctas ? cluster.map_shared_rank(&s, r < ctas ? r : 0)->id[tid] : 0;
#pragma unroll
            for (int r = 0; r < kMaxCtas; ++r) number += theirs[r];
            // (every CTA adds up the same in the same order)
            const float share = static_cast<float>(number) * (by_largest ? 1.f : by_count ? 8.f : 8.f * exp2_fast((static_cast<float>(tid) + 0.5f) * (kDeep / kBins)));
            estimated_upto = warp_scan(share, lane);
            if (lane == 31) s.told_top[warp] = estimated_upto;
            __syncthreads();
            for (int w = 0; w < kWarps; ++w) {
                if (w == warp) estimated_upto += estimated;
                estimated += s.told_top[w];
            }
            if (!by_count) want = max(part_of(total, fmaxf(s.p, 0.f), true), static_cast<uint64_t>(1));
        }
        float lid = top;                         // above which the border does not lie, by the same estimate
        // The bound of an attempt. Counts, or the weight that may lie below (the whole less 'want', of which
        // an eighth of the logits give an idea), with room for what chance does to the estimate.
        auto bound_of = [&](int attempt) {
            lid = top;
            if (few || attempt == 2) return heat.deep;
            const float goal = static_cast<float>(want), rest = static_cast<float>(total - want) * (1.f / kOne);
            const float least_of = by_largest ? 0.f : by_count ? goal - goal * 0.25f - 64.f : estimated - 1.25f * rest;
            const float most_of = !by_count ? estimated - (attempt == 0 ? 0.75f : 0.25f) * rest : attempt > 0 ? 2.f * goal + 512.f : by_largest ? goal : goal * 1.25f + 64.f;
            const int bin = min(__syncthreads_count(estimated_upto < most_of), kBins - 1), lid_bin = min(__syncthreads_count(estimated_upto < least_of), bin);
            // (a top-p of a top-k may cut anywhere)
            if (attempt == 0 && !(by_count && by_mass)) lid = top - static_cast<float>(lid_bin) * width;
            return fmaxf(top - static_cast<float>(bin + 1) * width, heat.deep);
        };

        // ---- the step's bins summed over the cluster, a bin a thread: its own, those up to it
        unsigned upto_count = 0;
        auto sum_bins = [&]() {
            sync();
            mass = number = 0;
            auto take = [&](const S& o) {
                number += o.count[tid];
                if (by_mass) mass += o.mass[0][tid] + (static_cast<uint64_t>(o.mass[1][tid]) << 16) + (static_cast<uint64_t>(o.mass[2][tid]) << 32);
            };
            if (mode == kAlone) {
                take(s);
            } else {
#pragma unroll 4
                for (int r = 0; r < ctas; ++r) take(*cluster.map_shared_rank(&s, r));
                cluster.sync();                                 // all have read them
            }
            s.count[tid] = 0;
#pragma unroll
            for (int e = 0; e < 3; ++e) s.mass[e][tid] = 0;
            upto = warp_scan(mass, lane), upto_count = warp_scan(number, lane);
            if (lane == 31) s.warp_mass[warp] = upto, s.warp_count[warp] = upto_count;
            __syncthreads();
            for (int w = 0; w < warp; ++w) upto += s.warp_mass[w], upto_count += s.warp_count[w];
        };
        // the bin in which `goal` is reached: it, what lies before it and in it (false: none)
        int bin;
        uint64_t before_mass, in_mass;
        unsigned before, in;
        auto find_bin = [&](bool count, uint64_t goal) {
            bin = __syncthreads_count(count ? upto_count < goal : upto < goal);
            if (bin == tid) s.before_mass = upto - mass, s.in_mass = mass, s.before = upto_count - number, s.in = number;
            __syncthreads();
            before_mass = s.before_mass, in_mass = s.in_mass, before = s.before, in = s.in;
            return bin < kBins;
        };
        auto add = [&](int to, uint64_t w, unsigned n = 1) {
            atomicAdd(&s.count[to], n);
            if (!by_mass) return;
            atomicAdd(&s.mass[0][to], static_cast<unsigned>(w) & 0xFFFFu);
            atomicAdd(&s.mass[1][to], static_cast<unsigned>(w) >> 16);
            atomicAdd(&s.mass[2][to], static_cast<unsigned>(w >> 32));
        };

        // the listed logits by value: those above the lid in the first bin, which a warp adds up by itself
        float fine = 0.f;
        bool found = false;
        auto coarse = [&](float y) { return y > lid ? 0 : min(1 + static_cast<int>((lid - y) * fine), kBins - 1); };
        auto by_value = [&]() {
            fine = (kBins - 1.5f) / fmaxf(lid - bound, 1e-30f);
            unsigned over = 0;
            uint64_t over_mass = 0;
            each([&](const float (&y)[4]) {
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    uint64_t w[2] = {};
                    if (by_mass) weigh2(y[e], y[e + 1], w[0], w[1]);
#pragma unroll
                    for (int f = 0; f < 2; ++f) {
                        if (y[e + f] > lid) ++over, over_mass += w[f];
                        else if (y[e + f] >= bound) add(coarse(y[e + f]), w[f]);
                    }
                }
            });
            over = __reduce_add_sync(~0u, over), over_mass = warp_sum(over_mass);
            if (lane == 0 && over > 0) add(0, over_mass, over);
            sum_bins();
        };
        // ---- the list of the logits at the bound and above
        for (int attempt = 0;; ++attempt) {
            bound = bound_of(attempt);
            int m = 0;
            for (int i0 = part_begin / kN; i0 < part_end / kN; i0 += 128) {
                // 128 vectors, four a lane: a bit a logit
                unsigned set[4] = {};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = i0 + 32 * e + lane;
                    if (i >= part_end / kN) continue;
                    const uint4 v = vec[i];
                    Most<kDtype> most_of;
                    most_of.take(v);
                    if (!(most_of.get() >= bound)) continue;
                    float y[kN];
                    unpack<kDtype>(v, y);
#pragma unroll
                    for (int n = 0; n < kN; ++n) set[e] |= (y[n] >= bound ? 1u : 0u) << n;
                }
                if (!__any_sync(~0u, (set[0] | set[1] | set[2] | set[3]) != 0)) continue;
                // the counts of all four in one scan (at most 256 each)
                const uint64_t count = static_cast<uint64_t>(__popc(set[0])) | static_cast<uint64_t>(__popc(set[1])) << 16 |
                                       static_cast<uint64_t>(__popc(set[2])) << 32 | static_cast<uint64_t>(__popc(set[3])) << 48;
                const uint64_t upto = warp_scan(count, lane), sums = __shfl_sync(~0u, upto, 31), before = upto - count;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    int to = m + static_cast<int>((before >> (16 * e)) & 0xFFFF);
                    for (; set[e] != 0; set[e] &= set[e] - 1, ++to)
                        if (to < list_room) mine[to] = static_cast<uint16_t>((i0 + 32 * e + lane) * kN + __ffs(set[e]) - 1);
                    m += static_cast<int>((sums >> (16 * e)) & 0xFFFF);
                }
            }
            if (lane == 0) s.told_count[warp] = m;
            cluster.sync();
            const Two<unsigned> lists = of_warps<unsigned>(cluster, ctas, lane, s, &S::told_count, 0);
            const unsigned lists_upto = warp_scan(lists.x + lists.y, lane), listed = __shfl_sync(~0u, lists_upto, 31);
            // all of the CTA's warps go through their lists, or all through everything
            const bool fits = !__any_sync(~0u, lane / 4 == rank && (lists.x > list_room || lists.y > list_room));
            mode = fits ? kListed : kAll;
            n = fits ? m : part_end - part_begin;
            const bool last = bound == heat.deep;
            // (of a long list of a top-p alone it is seen by value)
            bool enough = last || (by_count ? listed >= want : listed > kShort);
            if (!enough && !by_count) {
                uint64_t have = 0;
                each([&](const float (&y)[4]) {
                    uint64_t w[4];
                    weigh(y, w);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (y[e] >= bound) have += w[e];
                });
                tell_mass(have);
                cluster.sync();
                enough = all_mass() >= want;
            }
            if (!enough) {
                cluster.sync();                  // all have read what is told anew
                continue;
            }
            if (listed <= kShort) {
                // to the first CTA, in the order of the ids
                S* first = cluster.map_shared_rank(&s, 0);
                auto put = [&](int to, int at) {
                    if constexpr (kDtype == HC_DTYPE_FP32) first->value[to] = reinterpret_cast<const float*>(segment)[at];
                    else first->value[to] = reinterpret_cast<const uint16_t*>(segment)[at];
                    first->id[to] = id0 + at;
                };
                const unsigned first_of_two = lists_upto - lists.x - lists.y;
                int to = __shfl_sync(~0u, (warp & 1) ? first_of_two + lists.x : first_of_two, 4 * rank + warp / 2);
                if (fits) {
                    for (int i = lane; i < m; i += 32) put(to + i, mine[i]);
                } else {                                        // (found again)
                    for (int i = part_begin; i < part_end; i += 32) {
                        const float y = i + lane < part_end ? logit<kDtype>(segment, i + lane) : -CUDART_INF_F;
                        const unsigned votes = __ballot_sync(~0u, y >= bound);
                        if (y >= bound) put(to + __popc(votes & ((1u << lane) - 1u)), i + lane);
                        to += __popc(votes);
                    }
                }
                cluster.sync();
                if (rank != 0) return;
                if (listed <= kThreads) {
                    finish_alone(s, a, row, static_cast<int>(listed), k, by_count, by_mass, few && !by_count, want, top, weigh);
                    return;
                }
                mode = kAlone, ctas = 1;
                const int share = (static_cast<int>(listed) + kWarps - 1) / kWarps;
                begin = min(warp * share, static_cast<int>(listed));
                n = min(share, static_cast<int>(listed) - begin);
            }
            // by value, and the bin with the border that `want` makes
            while (true) {
                by_value();
                if (few && by_mass && !by_count) {              // (the whole is known from the bins)
                    __syncthreads();
                    if (tid == kBins - 1) s.before_mass = upto;
                    __syncthreads();
                    total = s.before_mass;
                    want = max(part_of(total, fmaxf(s.p, 0.f), true), static_cast<uint64_t>(1));
                }
                found = find_bin(by_count, want);
                if (bin > 0 || lid >= top) break;
                lid = top;                       // the estimate was wrong
            }
            if (found || last || mode == kAlone) break;         // (else fewer have weight: all of them stay)
        }
        // ---- borders: the value at which `goal` is reached, in the bin that has been found
        auto border = [&](bool count, uint64_t goal) {
            // the values of that bin, and what rounding may add to them
            const int first = bin;
            const float high = lid - static_cast<float>(first - 1) / fine, least_of = lid - static_cast<float>(first) / fine;
            const float slack = 1e-5f * (fabsf(top) + fabsf(bound));
            uint32_t hi = key_of<kDtype>(fminf(high + slack, top));
            uint32_t lo = key_of<kDtype>(fmaxf((first == kBins - 1 ? bound : least_of) - slack, -kTop));
            if (hi - lo < 32) {
                // where one value falls into that bin, it is the border
                const unsigned fall = __ballot_sync(~0u, lo + lane <= hi && value_of<kDtype>(lo + lane) >= bound && coarse(value_of<kDtype>(lo + lane)) == first);
                if (__popc(fall) == 1) lo += __ffs(fall) - 1, hi = lo;
            }
            uint64_t mass_above = before_mass;
            unsigned above = before;
            while (hi > lo) {
                const int down = max(32 - __clz(hi - lo) - kBinBits, 0);
                __syncthreads();                                // the bins are free
                each([&](const float (&y)[4]) {
                    bool in_it[4];
                    uint32_t key[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        key[e] = key_of<kDtype>(y[e]);
                        in_it[e] = y[e] >= bound && key[e] >= lo && key[e] <= hi && coarse(y[e]) == first;
                    }
#pragma unroll
                    for (int e = 0; e < 4; e += 2) {
                        if (!__any_sync(__activemask(), in_it[e] | in_it[e + 1])) continue;
                        uint64_t w[2] = {};
                        if (by_mass) weigh2(y[e], y[e + 1], w[0], w[1]);
#pragma unroll
                        for (int f = 0; f < 2; ++f)
                            if (in_it[e + f]) add((hi - key[e + f]) >> down, w[f]);
                    }
                });
                sum_bins();
                if (!find_bin(count, goal - (count ? above : mass_above))) break;   // (cannot be: what was summed is summed again)
                above += before, mass_above += before_mass;
                hi -= static_cast<uint32_t>(bin) << down;
                lo = max(lo, hi - ((1u << down) - 1u));
            }
            Cut c;
            c.at = value_of<kDtype>(hi);
            c.above = mass_above;
            const uint64_t one = in > 0 ? in_mass / in : 1;
            c.ties = static_cast<unsigned>(count ? goal - above : (goal - mass_above + one - 1) / one);
            return c;
        };
        // what a thread found of the first bins, for a second border
        const uint64_t first_upto = upto, first_mass = mass;
        const unsigned first_count = upto_count, first_number = number;
        bool count = by_count;
        if (by_count && by_mass && !found) {
            __syncthreads();
            if (tid == kBins - 1) s.before_mass = upto;                         // all that are listed
            __syncthreads();
            want = max(part_of(s.before_mass, fmaxf(s.p, 0.f), true), static_cast<uint64_t>(1));
            count = false, found = find_bin(false, want);
        }
        while (found) {
            cut = border(count, want);
            if (!(count && by_mass)) break;
            // the top-p of what the top-k leaves
            uint64_t tie, none;
            weigh2(cut.at, -CUDART_INF_F, tie, none);
            want = max(part_of(cut.above + cut.ties * tie, fmaxf(s.p, 0.f), true), static_cast<uint64_t>(1));
            if (want > cut.above) {
                if (tie > 0) cut.ties = min(cut.ties, static_cast<unsigned>((want - cut.above + tie - 1) / tie));
                break;
            }
            upto = first_upto, mass = first_mass, upto_count = first_count, number = first_number;
            count = false, found = find_bin(false, want);
        }
    }

    // ---- the sums of what stays, and the token
    const uint64_t low = least_weight(s.least);
    uint64_t mass = 0;
    unsigned ties = 0;
    auto keep = [&](const float (&y)[4]) {
        uint64_t w[4];
        weigh(y, w);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (w[e] < low) continue;
            if (y[e] > cut.at) mass += w[e];
            if (y[e] == cut.at) ++ties;
        }
    };
    if (mode == kAll && cut.at == -CUDART_INF_F && low == 1) each_of_all([&](const float (&y)[4]) {
        uint64_t w[4];
        weigh(y, w);
        mass += (w[0] + w[1]) + (w[2] + w[3]);
    });
    else if (mode == kAll) each_of_all(keep);
    else each(keep);
    tell_mass(mass);
    ties = __reduce_add_sync(~0u, ties);
    if (lane == 0) s.told_count[warp] = ties, s.warp_begin[warp] = begin, s.warp_n[warp] = n;
    sync();
    // two warps a lane: how many of their equal ones stay, and the sums up to them
    const Two<uint64_t> masses = of_warps<uint64_t>(cluster, ctas, lane, s, &S::told_mass, 0);
    const Two<unsigned> all_ties = of_warps<unsigned>(cluster, ctas, lane, s, &S::told_count, 0);
    uint64_t tie = 0;
    if (cut.ties > 0) {
        uint64_t none;
        weigh2(cut.at, -CUDART_INF_F, tie, none);
    }
    const unsigned ties_before = warp_scan(all_ties.x + all_ties.y, lane) - all_ties.x - all_ties.y;
    const unsigned take_x = min(cut.ties - min(cut.ties, ties_before), all_ties.x);
    const unsigned take_y = min(cut.ties - min(cut.ties, ties_before + all_ties.x), all_ties.y);
    const uint64_t sum_x = masses.x + take_x * tie, sum_y = masses.y + take_y * tie, upto = warp_scan(sum_x + sum_y, lane);
    const uint64_t total = __shfl_sync(~0u, upto, 31);
    const uint64_t goal = s.u < 1.f ? part_of(total, fmaxf(s.u, 0.f), false) : total - 1;
    // the warp whose sum passes the goal, what lies before it, and how many equal ones of it stay
    const unsigned past = __ballot_sync(~0u, upto > goal);
    const int at_lane = __ffs(past) - 1;
    const bool in_y = __shfl_sync(~0u, goal >= upto - sum_y, at_lane);
    uint64_t from = __shfl_sync(~0u, in_y ? upto - sum_y : upto - sum_y - sum_x, at_lane);
    unsigned allow = __shfl_sync(~0u, in_y ? take_y : take_x, at_lane);
    // no CTA leaves while another reads its memory: the one with the token waits behind the rest of its work
    const bool joined = mode != kAlone;
    if (joined) cluster_arrive();
    if (at_lane / 4 == rank) {
        // the warp's logits, a run of them a thread: how many equal ones stay, and the sum, of those before
        const int owner = 2 * (at_lane % 4) + in_y, its_n = s.warp_n[owner];
        begin = s.warp_begin[owner], mine = list + owner * list_room;
        const int share = (its_n + kThreads - 1) / kThreads, i0 = min(tid * share, its_n), i1 = min(i0 + share, its_n);
        auto bring = [&](int i, float (&y)[4], uint64_t (&w)[4]) {
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = i + e < i1 ? value_at(i + e) : -CUDART_INF_F;
            weigh(y, w);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (w[e] < low || y[e] < cut.at) w[e] = 0;
        };
        mass = ties = 0;
        for (int i = i0; i < i1; i += 4) {
            float y[4];
            uint64_t w[4];
            bring(i, y, w);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (y[e] != cut.at) mass += w[e];
                else ties += w[e] > 0;
            }
        }
        unsigned ties_upto = warp_scan(ties, lane);
        if (lane == 31) s.warp_count[warp] = ties_upto;
        __syncthreads();
        for (int w = 0; w < warp; ++w) ties_upto += s.warp_count[w];
        unsigned take = min(allow - min(allow, ties_upto - ties), ties);
        const uint64_t sum = mass + take * tie;
        uint64_t at = warp_scan(sum, lane);
        if (lane == 31) s.warp_mass[warp] = at;
        __syncthreads();
        for (int w = 0; w < warp; ++w) at += s.warp_mass[w];
        at += from - sum;
        // the thread whose sum passes the goal goes through its own
        if (goal >= at && goal - at < sum) {
            for (int i = i0; i < i1 && at <= goal; i += 4) {
                float y[4];
                uint64_t w[4];
                bring(i, y, w);
                int j = -1;
                float drawn = 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (w[e] > 0 && y[e] == cut.at) {
                        if (take == 0) w[e] = 0;
                        else --take;
                    }
                    at += w[e];
                    if (j < 0 && at > goal) j = i + e, drawn = y[e];
                }
                if (j < 0) continue;
                a.ids[row] = mode == kAlone ? s.id[begin + j] : id0 + (mode == kListed ? static_cast<int>(mine[j]) : begin + j);
                a.logprob[row] = log_weight(drawn, top, s.t) - logf(static_cast<float>(total) * (1.f / kOne));
            }
        }
    }
    if (joined) cluster_wait();
}

// CTAs of a row: as many as keep a part within 16384 logits, and twice, four times as many where there
// are too few rows to fill the GPU and a part stays above 2048.
int row_ctas(int sm_count, int rows, int vocab) {
    int n = 1;
    while (n < kMaxCtas && vocab > n * 16384) n *= 2;
    while (n < kMaxCtas && static_cast<int64_t>(rows) * n * 2 <= sm_count && vocab > n * 2 * 2048) n *= 2;
    return n;
}

template <int kDtype>
cudaError_t call(const Ctx& ctx, const SampleArgs& a, cudaStream_t st) {
    constexpr int kItem = kDtype == HC_DTYPE_FP32 ? 4 : 2, kN = 16 / kItem;
    const int ctas = row_ctas(ctx.sm_count, a.tokens, a.vocab);
    // a row may begin anywhere in its first vector
    const int vectors = ((a.vocab + 2 * kN - 2) / kN + ctas - 1) / ctas;
    // a list of all that a warp goes through, 16 bits each; of three tenths where CTAs share the SMs, so that four
    // CTAs do
    const bool alone = static_cast<int64_t>(a.tokens) * ctas <= 2 * ctx.sm_count;
    const int most = (vectors + kWarps - 1) / kWarps * kN, room = alone ? most : most * 3 / 10;
    const size_t smem = static_cast<size_t>(vectors) * 16 + sizeof(uint16_t) * kWarps * room;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.tokens) * ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas, attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, sample_kernel<kDtype>, a, ctas, vectors * 16, room, ctx.s.status);
}

// A launch has at most 2^31 - 1 CTAs.
template <int kDtype>
cudaError_t call_in_parts(const Ctx& ctx, const SampleArgs& a, cudaStream_t st) {
    constexpr int kRows = 1 << 27, kItem = kDtype == HC_DTYPE_FP32 ? 4 : 2;
    for (int64_t at = 0; at < a.tokens; at += kRows) {
        SampleArgs b = a;
        b.tokens = static_cast<int>(a.tokens - at < kRows ? a.tokens - at : kRows);
        b.logits = static_cast<const unsigned char*>(a.logits) + at * a.row * kItem;
        b.uniform += at, b.ids += at, b.logprob += at;
        if (a.temperature) b.temperature += at;
        if (a.top_k) b.top_k += at;
        if (a.top_p) b.top_p += at;
        if (a.min_p) b.min_p += at;
        const cudaError_t e = call<kDtype>(ctx, b, st);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <int kDtype>
cudaError_t allow_smem() {
    constexpr int kItem = kDtype == HC_DTYPE_FP32 ? 4 : 2, kN = 16 / kItem;
    const int vectors = ((HC_SAMPLE_MAX_VOCAB + 2 * kN - 2) / kN + kMaxCtas - 1) / kMaxCtas;
    const int room = (vectors + kWarps - 1) / kWarps * kN;
    return cudaFuncSetAttribute(sample_kernel<kDtype>, cudaFuncAttributeMaxDynamicSharedMemorySize, vectors * 16 + static_cast<int>(sizeof(uint16_t)) * kWarps * room);
}

}  // namespace

cudaError_t sample_setup() {
    cudaError_t e = allow_smem<HC_DTYPE_BF16>();
    if (e == cudaSuccess) e = allow_smem<HC_DTYPE_FP16>();
    if (e == cudaSuccess) e = allow_smem<HC_DTYPE_FP32>();
    return e;
}

cudaError_t launch_sample_tokens(const Ctx& ctx, const SampleArgs& a, int dtype, cudaStream_t st) {
    switch (dtype) {
        case HC_DTYPE_BF16: return call_in_parts<HC_DTYPE_BF16>(ctx, a, st);
        case HC_DTYPE_FP16: return call_in_parts<HC_DTYPE_FP16>(ctx, a, st);
        default: return call_in_parts<HC_DTYPE_FP32>(ctx, a, st);
    }
}

}  // namespace hc
