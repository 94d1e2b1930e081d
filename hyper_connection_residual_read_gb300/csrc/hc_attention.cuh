// Attention over the cache held in 4 bits, for windows of few rows: the new tokens times
// the query heads of one kv head, at most 16.
//
// With few rows the cache's bytes bound the operator: head_dim / 2 + 4 bytes a token for
// the key and as much for the value, read once. Everything else has to keep out of their
// way:
//
// * Codes go from their words straight into matrix fragments. The keys are the left
//   operand (16 tokens x 16 dimensions) and the queries the right one, so that 8 rows fill
//   an mma.m16n8k16 and each further 8 rows reuse the decoded keys; the values,
//   transposed, are the left operand of the second product. (tcgen05 would take its
//   operands from shared or tensor memory: a second trip for every decoded value, four
//   times its bytes in the cache, and 128 rows where 8 are wanted.)
// * S_j = s_j (q . c_j) + m_j sum(q): the codes enter as whole numbers, exactly (as fp16
//   subnormals, one logical operation for two), and step and minimum are applied to the
//   product in fp32, once a token and row instead of once a value. Likewise o = sum w_j
//   (c_j - 8) + sum p_j (m_j + 8 s_j) with w_j = p_j s_j. w_j is rounded to fp16 (11 bits:
//   the one rounding of the product), after division by a power of two near the largest
//   w_j that its row has seen (so that neither a step of a key that the row does not see nor
//   one of next to no weight costs the others their bits); p_j itself is summed in fp32. 8 sum
//   w_j comes from the same rounded weights, by one more product with a constant, so that
//   their errors meet c_j - 8 and not c_j, which is three times as large.
// * The order of dimensions within a product is free as long as both operands agree, and
//   so is that of the tokens: both follow from which words a lane loads (16 bytes of a
//   key row, 8 of a value row), so that no value moves between lanes. Only the weights
//   do: an 8 x 8 transpose (movmatrix) turns the first product's result into the second
//   one's operand.
// * The running maximum is raised only when a logit passes it by 2^8 (weights stay
//   within fp16, sums in fp32): one vote a step instead of a reduction over lanes.
//
// Work is cut evenly, whatever the lengths: the units (256 tokens of one request and kv
// head) are numbered through, and each CTA takes an equal run of them (with four
// more counted for each request and head, for its start and merge). A CTA's eight
// warps take 32 tokens of each unit each and merge at the end of a (request, head). One
// that is split between CTAs is joined by the last of them to finish, in the order of
// the CTAs, from fp32 sums in scratch of a fixed size (a CTA can have at most two such
// pieces).
//
// Measured: 64 requests of one token over up to 16K tokens, 32/8 heads of 128, 116 us, 5.1
// TB/s of cache (75% of the copy rate): issue bounds it, the ALU pipe at 58%, 509
// instructions a warp for 32 tokens of 4 rows; 12 bytes a thread are spilled. One request over 4K
// tokens 9.6 us, over 200 6.0. 64 windows of 16 rows over 2K tokens, 4 heads of 128, 48 us, 1.5 TB/s:
// the 236 registers of 16 rows leave 8 warps an SM (12.5% of what it holds), which wait for
// instructions, barriers and one another's results; no pipe is a quarter busy but ALU (24%).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "hc_window.cuh"

namespace hc {
namespace {

#ifndef HC_WINDOW_WARPS
#define HC_WINDOW_WARPS 8
#endif
constexpr int kWarps = HC_WINDOW_WARPS;          // of a CTA; fewer where the requests behind a prefix are short (hc_attention_short.cu)
constexpr bool kShort = kWarps < 8;              // and then each (request, head) is one CTA's
constexpr int kCtasPerSm = kAttnCtasPerSm * 8 / kWarps;
constexpr int kThreads = kWarps * 32;
constexpr int kStep = 32;                        // tokens of a warp's step
constexpr int kUnit = kWarps * kStep;            // tokens of a unit
constexpr float kRaise = 8.f;                    // log2 by which a logit may pass the maximum
constexpr float kRoom = 32768.f;                 // by how much a weight times its step may pass their reference: fp16's range

constexpr int kStages = 3;                       // steps of a warp's ring
constexpr int kPieceCost = 4;                    // what a piece costs beside its units, in units (64 ragged requests:
                                                 // 129 us with 2, 116 with 4, 115 with 7)

// A step's slot in a warp's ring: key codes, value codes, key scales, value scales.
template <int kD>
struct Slot {
    static constexpr int kCodes = kStep * kD / 2;
    static constexpr int kScales = kStep * 4;
    static constexpr int kBytes = 2 * kCodes + 2 * kScales;
};

template <int kD, int kNT>
struct Smem {
    static constexpr int kMerge = kWarps * kStages * Slot<kD>::kBytes;  // 2 [kWarps][32] float4
    static constexpr int kQueries = kMerge + 2 * kWarps * 32 * 16;
    static constexpr int kQueryBytes = kNT > 1 ? kWarps * kNT * 8 * kD * 2 : 0;   // fragments, a copy a warp
    static constexpr int kStats = kQueries + kQueryBytes;              // max, sum [kWarps][8 kNT]
    static constexpr int kBytes = kStats + 2 * kWarps * 8 * kNT * 4;
};

// Fixed scratch: per CTA two pieces, and a counter of arrivals.
// Rows of this kernel; more go to the chunk kernel. (Requests x tokens, 4 kv heads of 128: 64 x
// 2K with 16 rows take 48 us here and 24 rows 79 us there, where 24 to 32 rows took 110 to 120
// us in a form of this kernel; one x 16K 20 us here with 16 rows, 44 us there with 30.)
constexpr int kMaxRows = 16;
constexpr int kPieceRows = kMaxRows;
constexpr int kPieceFloats = kPieceRows * (128 + 2);

// The walk of a CTA through its run. Runs are cut in slots: a (request, head) has its
// units, and before them kPieceCost slots that stand for the work of starting and merging.
struct Walk {
    int b, h, u0, u1, units;     // the units [u0, u1) of (b, h), of `units`
    int64_t left, base;          // slots left, and the number of (b, h)'s first slot; or kWhole and (b, h)'s number
    int cost;                    // slots before its units
    Window w;
};

__device__ __forceinline__ int window_units(const Window& w) {
    return w.n > 0 ? max((w.kv - 1) / kUnit + 1, 1) : 0;     // (kv may be 2^31 - 1)
}
__device__ __forceinline__ int64_t window_slots(const AttentionArgs& a, const Window& w, int cost) {
    const int units = window_units(w);
    return units ? static_cast<int64_t>(units + cost) * a.c.kv_heads : 0;
}

// Takes the slots of (b, h) from `from` on; false if none of them is a unit.
__device__ __forceinline__ bool walk_piece(Walk& k, int from) {
    const int64_t to = min(static_cast<int64_t>(k.units + k.cost), from + k.left);
    k.left -= to - from;
    k.u0 = max(from - k.cost, 0);
    k.u1 = static_cast<int>(to) - k.cost;
    return k.u1 > k.u0;
}

// Where the requests behind a prefix are many and short, a CTA takes each gridDim.x-th of all (request, head)s
// as a whole instead of a run: the joins of cut ones cost more than they even out (64 requests of up to 1K tokens
// of their own, 8 heads: 31 us in runs, 28.5 whole, 20 with CTAs of four warps).
constexpr int64_t kWhole = -1;
constexpr int kWholeUnits = 8;                   // of the longest request
constexpr int kWholeHeads = 128;                 // fewer leave most SMs without one

__device__ __forceinline__ bool walk_whole(const SharedArgs& a, Walk& k, int64_t number, int* status) {
    const int64_t all = static_cast<int64_t>(a.requests) * a.c.kv_heads;
    for (; number < all; number += gridDim.x) {
        k.b = static_cast<int>(number / a.c.kv_heads), k.h = static_cast<int>(number % a.c.kv_heads);
        k.w = load_window<kJoined>(a, k.b, status);
        k.units = window_units(k.w);
        if (k.units == 0) continue;
        k.u0 = 0, k.u1 = k.units;
        k.left = kWhole, k.base = number;
        return true;
    }
    return false;
}

// To the next piece; false at the end of the run.
template <Side kSide>
__device__ __forceinline__ bool walk_next(const Args<kSide>& a, Walk& k, int* status) {
    if constexpr (kSide == kJoined)
        if (k.left == kWhole) return walk_whole(a, k, k.base + gridDim.x, status);
    if (k.left == 0) return false;
    k.base += k.units + k.cost;
    if (++k.h == a.c.kv_heads) {
        k.h = 0;
        do {
            ++k.b;
            if (k.b >= a.requests) return false;
            k.w = load_window<kSide>(a, k.b, nullptr);
            k.units = window_units(k.w);
        } while (k.units == 0);
    }
    return walk_piece(k, 0);     // a run that ends within the leading slots has no unit there
}

struct Run {
    int b;
    int64_t offset, begin, end, total, ctas;
    int cost;
    bool whole;
    Window w;                    // of request b
};

__device__ __forceinline__ void cut_run(Run& run, int64_t total) {
    // CTAs beyond the number of slots have none, so that no run before them is empty
    run.total = total;
    run.ctas = min(static_cast<int64_t>(gridDim.x), total);
    const int64_t i = blockIdx.x;
    run.begin = i < run.ctas ? total * i / run.ctas : total;
    run.end = i < run.ctas ? total * (i + 1) / run.ctas : total;
}

// The CTA's run: every CTA sums the slots of all requests, and the thread whose share of
// the requests holds the run's first slot says where it lies. Up to 32 requests each warp
// does so for itself, a request a lane, without a barrier.
template <Side kSide>
__device__ Run find_run(const Args<kSide>& a, Run* shared, int64_t* sums, int* status) {
    const int tid = threadIdx.x, lane = tid & 31;
    if (kShort) {                                // (what does not fit is reported as it is loaded)
        Run run = {};
        run.whole = true;
        return run;
    }
    const int64_t heads = static_cast<int64_t>(a.requests) * a.c.kv_heads;
    const bool many = kSide == kJoined && heads >= kWholeHeads && 2 * heads >= gridDim.x;
    if (a.requests <= 32) {
        Window w = {};
        if (lane < a.requests) w = load_window<kSide>(a, lane, blockIdx.x == 0 ? status : nullptr);
        // no more units than CTAs: one each (a piece's cost would leave CTAs without one, and others
        // with two: one request of 8K tokens 14.7 us against 13.6)
        const int units = __reduce_add_sync(~0u, lane < a.requests ? window_units(w) : 0);
        const int cost = static_cast<int64_t>(units) * a.c.kv_heads <= gridDim.x ? 0 : kPieceCost;
        const int64_t mine = lane < a.requests ? window_slots(a, w, cost) : 0;
        int64_t upto = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t t = __shfl_up_sync(~0u, upto, d);
            if (lane >= d) upto += t;
        }
        Run run;
        run.cost = cost;
        run.whole = many && !__any_sync(~0u, lane < a.requests && window_units(w) > kWholeUnits);
        cut_run(run, __shfl_sync(~0u, upto, 31));
        run.b = min(__popc(__ballot_sync(~0u, upto <= run.begin)), 31);
        run.offset = run.begin - __shfl_sync(~0u, upto - mine, run.b);
        run.w.begin = __shfl_sync(~0u, w.begin, run.b);
        run.w.n = __shfl_sync(~0u, w.n, run.b);
        run.w.rows = __shfl_sync(~0u, w.rows, run.b);
        run.w.kv = __shfl_sync(~0u, w.kv, run.b);
        run.w.first = __shfl_sync(~0u, w.first, run.b);
        return run;
    }
    const int per = (a.requests - 1) / kThreads + 1;             // (of up to 2^31 - 1)
    const int b0 = static_cast<int>(min(static_cast<int64_t>(tid) * per, static_cast<int64_t>(a.requests))), b1 = b0 + min(per, a.requests - b0);
    int64_t mine = 0;
    bool long_one = false;
    for (int b = b0; b < b1; ++b) {
        const Window w = load_window<kSide>(a, b, blockIdx.x == 0 ? status : nullptr);
        mine += window_slots(a, w, kPieceCost);
        if (kSide == kJoined) long_one = long_one || window_units(w) > kWholeUnits;
    }
    const bool whole = kSide == kJoined && !__syncthreads_or(long_one) && many;
    int64_t upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t t = __shfl_up_sync(~0u, upto, d);
        if (lane >= d) upto += t;
    }
    if (lane == 31) sums[tid >> 5] = upto;
    __syncthreads();
    int64_t total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w == (tid >> 5)) upto += total;
        total += sums[w];
    }
    Run run;
    run.cost = kPieceCost;
    run.whole = whole;
    cut_run(run, total);
    if (run.begin < run.end && run.begin < upto && run.begin >= upto - mine) {
        int64_t at = upto - mine;
        for (int b = b0; b < b1; ++b) {
            const Window w = load_window<kSide>(a, b, nullptr);
            const int64_t n = window_slots(a, w, kPieceCost);
            if (run.begin < at + n) {
                run.b = b;
                run.offset = run.begin - at;
                run.w = w;
                *shared = run;
                break;
            }
            at += n;
        }
    }
    __syncthreads();
    return run.begin < run.end ? *shared : run;
}

// The first piece of the run; false if it has none.
template <Side kSide>
__device__ __forceinline__ bool walk_start(const Args<kSide>& a, const Run& run, Walk& k, int* status) {
    if constexpr (kSide == kJoined)
        if (run.whole) return walk_whole(a, k, blockIdx.x, status);
    if (run.begin >= run.end) return false;
    k.b = run.b;
    k.w = run.w;
    k.units = window_units(k.w);
    k.cost = run.cost;
    const int slots = k.units + k.cost;
    k.h = static_cast<int>(run.offset / slots);
    const int from = static_cast<int>(run.offset - static_cast<int64_t>(k.h) * slots);
    k.left = run.end - run.begin;
    k.base = run.begin - from;
    return walk_piece(k, from) || walk_next<kSide>(a, k, status);
}

// D += A (16 x 16, row-major fragments) B (16 x 8), fp16 with fp32 sums.
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                    uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ uint32_t permute(uint32_t x, uint32_t y, uint32_t how) {
    return __byte_perm(x, y, how);
}

// The token of a 16-token tile that row m of the first product stands for. Any order
// would do; this one keeps the lanes that load together on different banks.
__device__ __forceinline__ int tile_token(int m) { return m ^ ((m >> 1) & 1); }

template <int kD, int kDtype, int kNT, Side kSide>
__global__ void __launch_bounds__(kThreads, kNT == 1 ? kCtasPerSm : kCtasPerSm / 2)
    window_kernel(const Args<kSide> a, float* scratch, unsigned* arrivals, int* status) {
    constexpr int kW = kD / 32;              // words of a key row that a lane loads
    constexpr int kVW = kD / 64;             // words of a value row that a lane loads
    constexpr int kRows = 8 * kNT;
    using S = Smem<kD, kNT>;
    using L = Slot<kD>;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ Run shared_run;
    __shared__ int64_t sums[kThreads / 32];
    __shared__ unsigned last_one;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tq = lane & 3;
    const int group = a.q_heads / a.c.kv_heads;

    // The own part behind a prefix runs beside the kernel that ends the prefix, which began after all that
    // this one reads was written; it waits for it where it first touches what the two have in common.
    if (kSide != kJoined) begin_early();
    const Run run = find_run<kSide>(a, &shared_run, sums, status);
    // The walk, a copy a warp, kept here and not in registers, which the loop over the steps has
    // none to spare of.
    __shared__ Walk walks[kWarps];
    Walk& k = walks[warp];
    auto keep = [&](const Walk& next) {
        __syncwarp();
        if (lane == 0) k = next;
        __syncwarp();
    };
    {
        Walk first;
        if (!walk_start<kSide>(a, run, first, kShort ? status : nullptr)) {
            if (kSide == kJoined) begin_early();             // (who waits for this kernel waits for the one before)
            return;
        }
        keep(first);
    }

    uint32_t* my_q = reinterpret_cast<uint32_t*>(smem + S::kQueries) + warp * (kNT * 8 * kD / 2);
    float* s_max = reinterpret_cast<float*>(smem + S::kStats);
    float* s_sum = s_max + kWarps * kRows;
    const int sh = 31 - __clz(a.c.block_size);
    const uint32_t to_values = static_cast<uint32_t>(a.c.kv_heads) * a.c.block_size;   // groups from keys to values
    const unsigned char* ring = smem + warp * (kStages * L::kBytes);
    // Copies: lanes 0-15 bring the first 16 tokens of the warp's step, lanes 16-31 the others, 16
    // bytes a lane and copy; four lanes of each half the keys' scales and four the values'.
    const int half = lane >> 4, l16 = lane & 15;
    const uint32_t block_bytes = 2 * to_values * (kD / 2);
    const uint32_t put = tc::smem_u32(ring) + half * (L::kCodes / 2) + l16 * 16;
    const uint32_t put_scales = tc::smem_u32(ring) + 2 * L::kCodes + (l16 >> 2) * L::kScales + half * (L::kScales / 2) + (l16 & 3) * 16;
    int id = 0;                              // the block of this lane's half of the step to be copied next
    int u1, kv;                              // of the piece whose steps are copied
    const int32_t* pages;
    const unsigned char* head_codes;
    const unsigned char* head_scales;
    auto look_up = [&](int u) {
        const unsigned t = static_cast<unsigned>(u) * kUnit + warp * kStep + half * 16;
        if (u < u1 && t < static_cast<unsigned>(kv) && HC_IN_RANGE(pages + (t >> sh) - a.table, 1, table_extent(a), status))
            id = pages[t >> sh];
    };
    // brings the step of unit u to a slot of the ring (a group of copies, if an empty one)
    auto fetch = [&](int u, int slot) {
        const unsigned t = static_cast<unsigned>(u) * kUnit + warp * kStep + half * 16;
        if (u < u1 && t < static_cast<unsigned>(kv)) {
            if (static_cast<unsigned>(id) >= static_cast<unsigned>(a.c.blocks)) {
                atomicOr(status, kStatusBounds);
                id = 0;                      // wrong values, from the cache's own memory
            }
            const uint64_t at = static_cast<uint64_t>(static_cast<uint32_t>(id)) * block_bytes + (t & (a.c.block_size - 1)) * (kD / 2);
            const unsigned char* keys = head_codes + at;
            const unsigned char* values = keys + to_values * (kD / 2);
            const uint32_t to = put + slot * L::kBytes;
#pragma unroll
            for (int i = 0; i < kD / 32; ++i) {
                if (HC_IN_RANGE(keys + i * 256 - a.c.codes, 16, group_count(a.c) * (kD / 2), status)) copy16(to + i * 256, keys + i * 256);
                if (HC_IN_RANGE(values + i * 256 - a.c.codes, 16, group_count(a.c) * (kD / 2), status))
                    copy16(to + L::kCodes + i * 256, values + i * 256);
            }
            const unsigned char* from = head_scales + at / (kD / 8);
            if (l16 < 8 && HC_IN_RANGE(from - reinterpret_cast<const unsigned char*>(a.c.scales), 16, group_count(a.c) * 4, status))
                copy16(put_scales + slot * L::kBytes, from);
        }
        copy_commit();
    };
    // a piece's first steps, on their way before the piece before it is merged
    auto begin = [&]() {
        u1 = k.u1, kv = k.w.kv;
        pages = a.table + static_cast<int64_t>(table_row(a, k.b)) * a.width;
        head_codes = a.c.codes + l16 * 16 + static_cast<int64_t>(k.h) * a.c.block_size * (kD / 2);
        head_scales = reinterpret_cast<const unsigned char*>(a.c.scales) + static_cast<int64_t>((l16 >> 2) * to_values + k.h * a.c.block_size) * 4 + (l16 & 3) * 16;
        const int u0 = k.u0;
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) {
            look_up(u0 + i);
            fetch(u0 + i, i);
        }
        look_up(u0 + kStages - 1);
    };
    begin();
    bool more = true;
    while (more) {
        int slot = 0;
        // queries: row g of each 8, the dimensions that go with this lane's key words
        const int rows = k.w.rows * group;
        uint32_t q[kNT == 1 ? 4 * kW : 1];
        float qsum[kNT][2], factor[kNT][2];      // of rows 2 tq and 2 tq + 1: sum(q) 2^-24, and what makes logits of S 2^-24
        {
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt) {
                uint4 raw[kW];
                float top = 0.f;
                const int r = nt * 8 + g;
                const int64_t from = static_cast<int64_t>(k.w.begin + r / group) * a.q_token +
                                     static_cast<int64_t>(k.h * group + r % group) * a.q_head + tq * (8 * kW);
#pragma unroll
                for (int i = 0; i < kW; ++i) {
                    raw[i] = make_uint4(0, 0, 0, 0);
                    if (r < rows && HC_IN_RANGE(from + 8 * i, 8, row_extent(a.tokens, a.q_heads, kD, a.q_token, a.q_head), status))
                        raw[i] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + from + 8 * i);
                    const uint32_t x[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 f = widen2<kDtype>(x[e]);
                        top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
                    }
                }
                // the row's largest: its scale is its own, so that no row has fewer bits for another's size
                top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
                top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
                const int e = query_exponent(top);
                const float down = power_of_two(-e), up = a.scale * kLog2e * power_of_two(e) * kCodeUp;
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < kW; ++i) {
                    const uint32_t x[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
                    float f[8];
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        const float2 y = widen2<kDtype>(x[p]);
                        f[2 * p] = y.x * down, f[2 * p + 1] = y.y * (down * kOdd);
                    }
                    uint32_t o[4];
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        o[p] = pack_half2(f[p], f[p + 4]);
                        const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&o[p]));
                        sum += (p & 1) ? (y.x + y.y) * (1.f / kOdd) : y.x + y.y;
                    }
                    if (kNT == 1) {
#pragma unroll
                        for (int p = 0; p < 4; ++p) q[(4 * i + p) % (kNT == 1 ? 4 * kW : 1)] = o[p];
                    } else {
                        *reinterpret_cast<uint4*>(my_q + ((nt * kW + i) * 32 + lane) * 4) = make_uint4(o[0], o[1], o[2], o[3]);
                    }
                }
                sum += __shfl_xor_sync(~0u, sum, 1);
                sum += __shfl_xor_sync(~0u, sum, 2);
                sum *= 1.f / kCodeUp;
                qsum[nt][0] = __shfl_sync(~0u, sum, 8 * tq);
                qsum[nt][1] = __shfl_sync(~0u, sum, 8 * tq + 4);
                factor[nt][0] = __shfl_sync(~0u, up, 8 * tq);
                factor[nt][1] = __shfl_sync(~0u, up, 8 * tq + 4);
            }
            __syncwarp();
        }

        float o[kVW * 4][kNT][4] = {}, eight[kNT][4] = {};   // and 8 times the sum of the weights
        float base[kNT][2], sum[kNT][2], flat[kNT][2];     // maximum, sum of p, sum of p (m + 8 s)
        float down[kNT][2];                                 // 2^-E of a row's largest weight times step; E is -126 at first
        uint32_t fresh = (1u << (2 * kNT)) - 1;            // rows of this lane without a maximum (base is 0)
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                base[nt][e] = 0.f, sum[nt][e] = 0.f, flat[nt][e] = 0.f, down[nt][e] = power_of_two(126);
        const int clear = kSide == kPrefix ? k.w.kv : min(k.w.kv, a.mask ? k.w.first : k.w.first + 1);   // every row sees what lies before

        // One step. kTail: some of its tokens are hidden from some rows, or lie behind the end.
        auto step = [&](auto tail, int u) {
            constexpr bool kTail = decltype(tail)::value;
            const int t0 = u * kUnit + warp * kStep;
            const unsigned char* in = ring + slot * L::kBytes;
            const uint32_t* scales = reinterpret_cast<const uint32_t*>(in + 2 * L::kCodes);
            // first product
            float s[2][kNT][4] = {};
            uint32_t kw[4][kW];                              // tokens g, g + 8 of both tiles
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const unsigned char* from = in + (x * 8 + tile_token(g)) * (kD / 2) + tq * (kD / 8);
                if (kW == 4) {
                    const uint4 y = *reinterpret_cast<const uint4*>(from);
                    kw[x][0] = y.x, kw[x][1] = y.y, kw[x][kW - 2] = y.z, kw[x][kW - 1] = y.w;
                } else {
                    const uint2 y = *reinterpret_cast<const uint2*>(from);
                    kw[x][0] = y.x, kw[x][1] = y.y;
                }
            }
#pragma unroll
            for (int i = 0; i < kW; ++i) {
                uint32_t bq[kNT][4];
#pragma unroll
                for (int nt = 0; nt < kNT; ++nt) {
                    if (kNT == 1) {
#pragma unroll
                        for (int p = 0; p < 4; ++p) bq[nt][p] = q[(4 * i + p) % (kNT == 1 ? 4 * kW : 1)];
                    } else {
                        const uint4 x = *reinterpret_cast<const uint4*>(my_q + ((nt * kW + i) * 32 + lane) * 4);
                        bq[nt][0] = x.x, bq[nt][1] = x.y, bq[nt][2] = x.z, bq[nt][3] = x.w;
                    }
                }
#pragma unroll
                for (int mt = 0; mt < 2; ++mt) {
                    uint32_t lo[4], hi[4];
                    decode_word(kw[2 * mt][i], lo);
                    decode_word(kw[2 * mt + 1][i], hi);
#pragma unroll
                    for (int nt = 0; nt < kNT; ++nt) {
                        mma(s[mt][nt], lo[0], hi[0], lo[1], hi[1], bq[nt][0], bq[nt][1]);
                        mma(s[mt][nt], lo[2], hi[2], lo[3], hi[3], bq[nt][2], bq[nt][3]);
                    }
                }
            }
            // logits in powers of two, less the maximum so far
            float vs[4], vm[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {                    // tokens g, g + 8 of both tiles
                const int j = x * 8 + tile_token(g);
                uint32_t kk = scales[j], vv = scales[kStep + j];
                if (kTail && t0 + j >= k.w.kv) kk = vv = 0;
                const float sj = bf16_lo(kk), mj = bf16_hi(kk);
                vs[x] = bf16_lo(vv);
                vm[x] = fmaf(8.f, vs[x], bf16_hi(vv));
#pragma unroll
                for (int nt = 0; nt < kNT; ++nt) {
                    float& z0 = s[x >> 1][nt][(x & 1) * 2];
                    float& z1 = s[x >> 1][nt][(x & 1) * 2 + 1];
                    const uint64_t t = fma2(pair(sj, sj), pair(z0, z1), mul2(pair(mj, mj), pair(qsum[nt][0], qsum[nt][1])));
                    const float2 z = unpair(fma2(t, pair(factor[nt][0], factor[nt][1]), pair(-base[nt][0], -base[nt][1])));
                    z0 = z.x, z1 = z.y;
                }
            }
            if (kTail) {
#pragma unroll
                for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int r = nt * 8 + 2 * tq + e, i = r / group;
                        uint64_t bits = 0;
                        if (kSide != kPrefix && a.mask && r < rows && HC_IN_RANGE(k.w.begin + i, 1, a.tokens, status)) bits = a.mask[k.w.begin + i];
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const int j = t0 + x * 8 + tile_token(g), back = j - k.w.first;
                            const bool sees = j < k.w.kv && (kSide == kPrefix || (a.mask ? back < 0 || (back < 64 && ((bits >> back) & 1)) : back <= i));
                            if (!sees) s[x >> 1][nt][(x & 1) * 2 + e] = -CUDART_INF_F;
                        }
                    }
            }
            // weights p, and p times step in fp16
            float p[4][kNT][2];
            uint32_t w[4][kNT];
            auto weigh = [&]() {
#pragma unroll
                for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const float z0 = s[x >> 1][nt][(x & 1) * 2], z1 = s[x >> 1][nt][(x & 1) * 2 + 1];
                        const float p0 = p[x][nt][0] = exp2_fast(z0), p1 = p[x][nt][1] = exp2_fast(z1);
                        // (in this order: a step may be as far above the reference as its weight is small)
                        float2 y = unpair(mul2(mul2(pair(p0, p1), pair(vs[x], vs[x])), pair(down[nt][0], down[nt][1])));
                        if (kTail) {                         // a hidden value may be NaN
                            if (z0 == -CUDART_INF_F) y.x = 0.f;
                            if (z1 == -CUDART_INF_F) y.y = 0.f;
                        }
                        w[x][nt] = pack_half2(y.x, y.y);
                    }
            };
            weigh();
            // raise the maximum, or the reference of weights times steps, where they are passed
            bool raise = fresh != 0;
            float peak[kNT][2];
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt) {
                const __half2* y = reinterpret_cast<const __half2*>(w[0]) + nt;
                const __half2 most = __hmax2(__hmax2(y[0], y[kNT]), __hmax2(y[2 * kNT], y[3 * kNT]));
                raise |= !__hble2(most, __float2half2_rn(kRoom));
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    peak[nt][e] = fmaxf(fmaxf(s[0][nt][e], s[0][nt][2 + e]), fmaxf(s[1][nt][e], s[1][nt][2 + e]));
                    raise |= peak[nt][e] > kRaise;
                }
            }
            if (__any_sync(~0u, raise)) {
#pragma unroll
                for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float top = peak[nt][e];
                        top = fmaxf(top, __shfl_xor_sync(~0u, top, 4));
                        top = fmaxf(top, __shfl_xor_sync(~0u, top, 8));
                        top = fmaxf(top, __shfl_xor_sync(~0u, top, 16));
                        // by how much the maximum rises (of a fresh row: to the first logit seen)
                        const uint32_t bit = 1u << (2 * nt + e);
                        const bool first = (fresh & bit) != 0;
                        const float up = first ? (top == -CUDART_INF_F ? 0.f : top) : fmaxf(top, 0.f);
                        if (first && top != -CUDART_INF_F) fresh &= ~bit;
                        const float fix = first ? 1.f : exp2_fast(-up);
                        base[nt][e] += up;
#pragma unroll
                        for (int x = 0; x < 4; ++x) s[x >> 1][nt][(x & 1) * 2 + e] -= up;
                        sum[nt][e] *= fix;
                        flat[nt][e] *= fix;
                        // the largest weight times step: of this step's (hidden ones are 0 or NaN), and
                        // of those before, which the maximum has made smaller
                        float most = 0.f;
#pragma unroll
                        for (int x = 0; x < 4; ++x) most = fmaxf(most, exp2_fast(s[x >> 1][nt][(x & 1) * 2 + e]) * vs[x]);
                        most = fmaxf(most, __shfl_xor_sync(~0u, most, 4));
                        most = fmaxf(most, __shfl_xor_sync(~0u, most, 8));
                        most = fmaxf(most, __shfl_xor_sync(~0u, most, 16));
                        const int was = 127 - static_cast<int>(__float_as_uint(down[nt][e]) >> 23);
                        most = fmaxf(most, fix * power_of_two(was));
                        const int now = max(static_cast<int>(__float_as_uint(most) >> 23) - 127, -126);
                        down[nt][e] = power_of_two(-now);
                        // (in two factors: each alone is within fp32 where their product is)
                        const int half = (was - now) / 2;
                        const float by = fix * power_of_two(half) * power_of_two(was - now - half);
                        eight[nt][e] *= by;
#pragma unroll
                        for (int m = 0; m < kVW * 4; ++m) {
                            o[m][nt][e] *= by;
                            o[m][nt][2 + e] *= by;
                        }
                    }
                weigh();
            }
            uint32_t pw[2][kNT][2];
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    float m0 = vm[x], m1 = vm[x];
                    if (kTail) {
                        if (s[x >> 1][nt][(x & 1) * 2] == -CUDART_INF_F) m0 = 0.f;
                        if (s[x >> 1][nt][(x & 1) * 2 + 1] == -CUDART_INF_F) m1 = 0.f;
                    }
                    const uint64_t p2 = pair(p[x][nt][0], p[x][nt][1]);
                    const float2 s2 = unpair(add2(pair(sum[nt][0], sum[nt][1]), p2));
                    const float2 f2 = unpair(fma2(p2, pair(m0, m1), pair(flat[nt][0], flat[nt][1])));
                    sum[nt][0] = s2.x, sum[nt][1] = s2.y, flat[nt][0] = f2.x, flat[nt][1] = f2.y;
                    pw[x >> 1][nt][x & 1] = transpose8x8(w[x][nt]);
                }
            // second product
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
                for (int nt = 0; nt < kNT; ++nt)
                    mma(eight[nt], 0x00080008u, 0x00080008u, 0x00080008u, 0x00080008u, pw[mt][nt][0], pw[mt][nt][1]);
                uint32_t vw[4][kVW];                         // tokens 2 tq, 2 tq + 1, 2 tq + 8, 2 tq + 9
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const unsigned char* from = in + L::kCodes + (mt * 16 + tile_token(2 * tq + (x & 1)) + (x >> 1) * 8) * (kD / 2) + g * (kD / 16);
                    if (kVW == 2) {
                        const uint2 y = *reinterpret_cast<const uint2*>(from);
                        vw[x][0] = y.x, vw[x][kVW - 1] = y.y;
                    } else {
                        vw[x][0] = *reinterpret_cast<const uint32_t*>(from);
                    }
                }
#pragma unroll
                for (int i = 0; i < kVW; ++i)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint32_t ab[4], cd[4];
                        decode_word(permute(vw[0][i], vw[1][i], half ? 0x7632 : 0x5410), ab);
                        decode_word(permute(vw[2][i], vw[3][i], half ? 0x7632 : 0x5410), cd);
#pragma unroll
                        for (int y = 0; y < 2; ++y)
#pragma unroll
                            for (int nt = 0; nt < kNT; ++nt)
                                mma(o[i * 4 + half * 2 + y][nt], ab[2 * y], ab[2 * y + 1], cd[2 * y], cd[2 * y + 1],
                                    pw[mt][nt][0], pw[mt][nt][1]);
                    }
            }
        };
        for (int u = k.u0; u < u1; ++u) {
            const int t = u * kUnit + warp * kStep;
            if (t >= kv) break;
            copy_wait<kStages - 2>();
            __syncwarp();                                    // every lane's copies, and its reads of the slot before
            fetch(u + kStages - 1, slot == 0 ? kStages - 1 : slot - 1);
            look_up(u + kStages);
            if (t <= clear - kStep) step(std::false_type(), u);
            else step(std::true_type(), u);
            if (++slot == kStages) slot = 0;
        }
        copy_wait<0>();
        __syncwarp();
        const Walk done = k;
        {
            Walk next = done;
            more = walk_next<kSide>(a, next, kShort ? status : nullptr);
            if (more) {
                keep(next);
                begin();
            }
        }

        if (kSide == kJoined) begin_early();     // the workspace, scratch and counters are free, the prefix's part is there

        // ---- merge the warps: their fragments lie alike, so that unit m of 4 values a lane
        // is exchanged through [warp][lane] and summed by warp m % 8: one after the other through
        // two buffers, or, after the last piece, all at once through the ring (2 us
        // less: a request of 200 tokens 8.9 -> 6.9 us)
        static_assert(S::kMerge >= kNT * kVW * 4 * kWarps * 32 * 16, "the ring holds every unit");
        float4* merge = reinterpret_cast<float4*>(smem + (more ? S::kMerge : 0));
        asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");   // the last piece's statistics are read
        // rows 2 tq and 2 tq + 1 of each 8
        float top[kNT][2];
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) {
                    sum[nt][e] += __shfl_xor_sync(~0u, sum[nt][e], d);
                    flat[nt][e] += __shfl_xor_sync(~0u, flat[nt][e], d);
                }
                // a row that has seen nothing but NaN has no maximum, but its sum has to be told
                top[nt][e] = ((fresh >> (2 * nt + e)) & 1) && sum[nt][e] == sum[nt][e] ? -CUDART_INF_F : base[nt][e];
                if (g == 0) {
                    s_max[warp * kRows + nt * 8 + 2 * tq + e] = top[nt][e];
                    s_sum[warp * kRows + nt * 8 + 2 * tq + e] = sum[nt][e];
                }
            }
        asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");
        const bool whole = done.u0 == 0 && done.u1 == done.units;
        float* piece = scratch + (static_cast<int64_t>(blockIdx.x) * 2 + (done.u0 == 0 ? 1 : 0)) * kPieceFloats;
        constexpr int kParts = kVW * 4;                      // units of one nt
        // what the prefix left of rows 2 tq and 2 tq + 1 of each 8 in the parts that this warp ends: asked for
        // before the merge, whose steps would wait for it one after the other
        struct Prior {
            float2 stats, value;
        };
        constexpr int kMine = kSide == kJoined ? (kNT * kParts + kWarps - 1) / kWarps : 1;
        Prior prior[kMine][2] = {};
        auto ask = [&](int nt, int m, Prior (&p)[2]) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = nt * 8 + 2 * tq + e;
                const int64_t at = static_cast<int64_t>(done.w.begin + r / group) * a.q_heads + done.h * group + r % group;
                if (r >= rows || !HC_IN_RANGE(at, 1, static_cast<size_t>(a.tokens) * a.q_heads, status)) continue;
                if constexpr (kSide == kJoined) {
                    p[e].stats = __ldcg(partial_stats(a, kD) + at);
                    p[e].value = __ldcg(reinterpret_cast<const float2*>(a.partial + at * kD + g * (kD / 8) + 2 * m));
                }
            }
        };
        if (kSide == kJoined && whole) {
#pragma unroll
            for (int i = 0; i < kMine; ++i) {
                const int turn = i * kWarps + warp;
                if (turn < kNT * kParts) ask(turn / kParts, turn % kParts, prior[i]);
            }
        }
        auto write_rows = [&](int nt, int m, const float4& x, const float (&peak)[2], const float (&total)[2], const Prior (&p)[2]) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = nt * 8 + 2 * tq + e;
                if (r >= rows) continue;
                float inv = total[e] == 0.f ? 0.f : 1.f / total[e];
                const int64_t at = static_cast<int64_t>(done.w.begin + r / group) * a.q_heads + done.h * group + r % group;
                const int d = g * (kD / 8) + 2 * m;
                if (!HC_IN_RANGE(at * kD + d, 2, static_cast<size_t>(a.tokens) * a.q_heads * kD, status)) continue;
                if constexpr (kSide == kPrefix) {
                    *reinterpret_cast<float2*>(a.partial + at * kD + d) = e ? make_float2(x.y * inv, x.w * inv) : make_float2(x.x * inv, x.z * inv);
                    if (d == 0) partial_stats(a, kD)[at] = make_float2(peak[e], total[e]);
                    continue;
                }
                float lse = total[e] == 0.f ? -CUDART_INF_F : (peak[e] + log2f(total[e])) * kLn2;
                float2 y = make_float2(0.f, 0.f);
                if constexpr (kSide == kJoined) {
                    const Join j = join_parts_of_row(peak[e], total[e], p[e].stats);
                    inv = j.by_own, lse = j.lse;
                    y = make_float2(j.by_prefix * p[e].value.x, j.by_prefix * p[e].value.y);
                }
                // (with a prefix's part: one more fma; without, the product alone)
                auto scaled = [&](float v, float more) { return kSide == kJoined ? fmaf(v, inv, more) : v * inv; };
                *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + at * kD + d) =
                    e ? narrow2<kDtype>(scaled(x.y, y.x), scaled(x.w, y.y)) : narrow2<kDtype>(scaled(x.x, y.x), scaled(x.z, y.y));
                if (a.lse && d == 0) a.lse[at] = lse;
            }
        };
        auto finish = [&](int nt, int m, const float4* buffer, const float (&peak)[2], const float (&total)[2], const Prior (&p)[2]) {
            float4 x = buffer[lane];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) {
                const float4 y = buffer[w * 32 + lane];
                x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
            }
            if (whole) {
                write_rows(nt, m, x, peak, total, p);
            } else {
                __stcg(reinterpret_cast<float4*>(piece) + (nt * kParts + m) * 32 + lane, x);
                if (m == 0 && g == 0) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        __stcg(piece + kPieceRows * kD + nt * 8 + 2 * tq + e, peak[e]);
                        __stcg(piece + kPieceRows * kD + kPieceRows + nt * 8 + 2 * tq + e, total[e]);
                    }
                }
            }
        };
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
            float peak[2], total[2], fix[2], vup[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = nt * 8 + 2 * tq + e;
                peak[e] = -CUDART_INF_F, total[e] = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) peak[e] = fmaxf(peak[e], s_max[w * kRows + r]);
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float m = s_max[w * kRows + r];
                    if (m != -CUDART_INF_F) total[e] += s_sum[w * kRows + r] * exp2_fast(m - peak[e]);
                }
                fix[e] = top[nt][e] == -CUDART_INF_F ? 0.f : exp2_fast(top[nt][e] - peak[e]);
                vup[e] = 1.f / down[nt][e];
            }
#pragma unroll
            for (int m = 0; m < kParts; ++m) {
                const int turn_m = nt * kParts + m;
                float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                if (fix[0] != 0.f) {
                    x.x = fmaf((o[m][nt][0] - eight[nt][0]) * kCodeUp, vup[0], flat[nt][0]) * fix[0];
                    x.z = fmaf(fmaf(o[m][nt][2], kOdd, -eight[nt][0]) * kCodeUp, vup[0], flat[nt][0]) * fix[0];
                }
                if (fix[1] != 0.f) {
                    x.y = fmaf((o[m][nt][1] - eight[nt][1]) * kCodeUp, vup[1], flat[nt][1]) * fix[1];
                    x.w = fmaf(fmaf(o[m][nt][3], kOdd, -eight[nt][1]) * kCodeUp, vup[1], flat[nt][1]) * fix[1];
                }
                float4* buffer = merge + (more ? turn_m & 1 : turn_m) * kWarps * 32;
                buffer[warp * 32 + lane] = x;
                if (more) {
                    asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");
                    if (warp == turn_m % kWarps) finish(nt, m, buffer, peak, total, prior[kSide == kJoined ? turn_m / kWarps : 0]);
                }
            }
            if (!more) {
                asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");
                if constexpr (kSide == kJoined) {            // (unrolled: what was asked for lies in registers)
#pragma unroll
                    for (int i = 0; i < kMine; ++i) {
                        const int turn = i * kWarps + warp;
                        if (turn / kParts == nt) finish(nt, turn % kParts, merge + turn * kWarps * 32, peak, total, prior[i]);
                    }
                } else {
#pragma unroll 1
                    for (int m = 0; m < kParts; ++m)
                        if (warp == (nt * kParts + m) % kWarps) finish(nt, m, merge + (nt * kParts + m) * kWarps * 32, peak, total, prior[0]);
                }
            }
        }
        if (!whole) {
            // the CTAs that share this (request, head): from the one with its first unit on
            const int64_t total = run.total, n = run.ctas;
            const int c0 = static_cast<int>(((done.base + done.cost + 1) * n - 1) / total);
            const int c1 = static_cast<int>(((done.base + done.cost + done.units) * n - 1) / total);
            if (!HC_IN_RANGE(c0, c1 - c0 + 1, gridDim.x, status)) break;      // scratch and counters go by CTA
            asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");
            if (threadIdx.x == 0) {
                const unsigned before = arrive(&arrivals[c0]);
                last_one = before == static_cast<unsigned>(c1 - c0);
                if (last_one) arrivals[c0] = 0;              // for the next launch
            }
            asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");
            if (last_one) {
                for (int u = warp; u < kNT * kParts; u += kWarps) {
                    const int nt = u / kParts, m = u % kParts;
                    float peak[2] = {-CUDART_INF_F, -CUDART_INF_F}, sums_all[2] = {};
                    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
                    for (int c = c0; c <= c1; ++c) {
                        const float* from = scratch + (static_cast<int64_t>(c) * 2 + (c == c0 ? 1 : 0)) * kPieceFloats;
                        const float2 top2 = __ldcg(reinterpret_cast<const float2*>(from + kPieceRows * kD + nt * 8 + 2 * tq));
                        const float2 sum2 = __ldcg(reinterpret_cast<const float2*>(from + kPieceRows * kD + kPieceRows + nt * 8 + 2 * tq));
                        const float4 y = __ldcg(reinterpret_cast<const float4*>(from) + u * 32 + lane);
                        float fx[2], fy[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float mine = e ? top2.y : top2.x, to = fmaxf(peak[e], mine);
                            fx[e] = peak[e] == -CUDART_INF_F ? 0.f : exp2_fast(peak[e] - to);
                            fy[e] = mine == -CUDART_INF_F ? 0.f : exp2_fast(mine - to);
                            peak[e] = to;
                            sums_all[e] = sums_all[e] * fx[e] + (e ? sum2.y : sum2.x) * fy[e];
                        }
                        x.x = x.x * fx[0] + y.x * fy[0], x.z = x.z * fx[0] + y.z * fy[0];
                        x.y = x.y * fx[1] + y.y * fy[1], x.w = x.w * fx[1] + y.w * fy[1];
                    }
                    Prior p[2] = {};
                    if (kSide == kJoined) ask(nt, m, p);
                    write_rows(nt, m, x, peak, sums_all, p);
                }
            }
        }
    }
}

template <int kD, int kDtype, int kNT, Side kSide>
cudaError_t launch_window(const Ctx& ctx, const Args<kSide>& a, cudaStream_t st) {
    // as many CTAs as are resident at once, and no more than there can be units
    const int64_t most = static_cast<int64_t>(a.requests) * a.c.kv_heads *
                         (kShort ? 1 : (static_cast<int64_t>(a.width) * a.c.block_size + kUnit - 1) / kUnit);
    const int64_t resident = static_cast<int64_t>(ctx.sm_count) * (kNT == 1 ? kCtasPerSm : kCtasPerSm / 2);
    const int grid = static_cast<int>(most < resident ? most : resident);
    return launch_early(window_kernel<kD, kDtype, kNT, kSide>, dim3(grid), kThreads, Smem<kD, kNT>::kBytes, st, a, ctx.attn_pieces,
                        ctx.attn_arrivals, ctx.s.status);
}

template <int kD, int kDtype, Side kSide>
cudaError_t launch_rows(const Ctx& ctx, const Args<kSide>& a, cudaStream_t st) {
    const int64_t rows = static_cast<int64_t>(a.max_new) * (a.q_heads / a.c.kv_heads);
    if (rows <= 8) return launch_window<kD, kDtype, 1, kSide>(ctx, a, st);
    return launch_window<kD, kDtype, 2, kSide>(ctx, a, st);
}

template <int kD, int kDtype, int kNT, Side kSide>
cudaError_t allow_smem() {
    return cudaFuncSetAttribute(window_kernel<kD, kDtype, kNT, kSide>, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<kD, kNT>::kBytes);
}
template <int kD, int kDtype, Side kSide>
cudaError_t allow_rows() {
    const cudaError_t e = allow_smem<kD, kDtype, 1, kSide>();
    return e != cudaSuccess ? e : allow_smem<kD, kDtype, 2, kSide>();
}

}  // namespace

template <Side kSide>
cudaError_t attention_window_setup() {
    cudaError_t e = allow_rows<64, HC_DTYPE_BF16, kSide>();
    if (e == cudaSuccess) e = allow_rows<64, HC_DTYPE_FP16, kSide>();
    if (e == cudaSuccess) e = allow_rows<128, HC_DTYPE_BF16, kSide>();
    if (e == cudaSuccess) e = allow_rows<128, HC_DTYPE_FP16, kSide>();
    return e;
}

template <Side kSide>
cudaError_t launch_attention(const Ctx& ctx, const Args<kSide>& a, int dtype, cudaStream_t st) {
    if (static_cast<int64_t>(a.max_new) * (a.q_heads / a.c.kv_heads) > kMaxRows)
        return launch_attention_chunk<kSide>(ctx, a, dtype, st);
    if (a.c.head_dim == 64)
        return dtype == HC_DTYPE_BF16 ? launch_rows<64, HC_DTYPE_BF16, kSide>(ctx, a, st) : launch_rows<64, HC_DTYPE_FP16, kSide>(ctx, a, st);
    return dtype == HC_DTYPE_BF16 ? launch_rows<128, HC_DTYPE_BF16, kSide>(ctx, a, st) : launch_rows<128, HC_DTYPE_FP16, kSide>(ctx, a, st);
}

}  // namespace hc
