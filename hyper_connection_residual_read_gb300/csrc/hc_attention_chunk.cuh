// Attention over the cache held in 4 bits, for chunks: more than 16 rows (new tokens times
// the query heads of a kv head), on tcgen05.
//
// Both products run on the tensor cores in fp16 with fp32 sums, 128 rows x 128 keys at a
// time: S = Q K'^T from shared memory, O += P V' with P in tensor memory. A CTA has two
// warpgroups of softmax (a thread a row), each of which also issues its row tile's products,
// one warpgroup that decodes keys and one that decodes values.
//
// * The decoded values are exact. A step has 8 significant bits (bf16) and |code - 8| <= 8
//   at most 3, so s (code - 8) has 11 at most, which is what fp16 holds: K' = 2^-E s_j
//   (c_j - 8), with E from the largest step of a tile, is exact for steps down to 2^-8 of
//   that one, whose last bit is then fp16's least (a group whose m + 8 s is beyond 2^15 s counts
//   as that over 2^15, beside which its rounding is nothing). So is V', whose E stays from tile
//   to tile while all steps lie within that range of it. One logical and one fp16 operation
//   decode two codes: a code's bits alone are the subnormal code * 2^-24, and fma with S = 2^24
//   2^-E s gives S code 2^-24 - S 8 2^-24.
// * A tile with steps further apart than 2^8 (it is "wide") has an E for each key, exact again.
//   The softmax then multiplies a logit by 2^E of its key, and a weight by 2^E of its value over a
//   power of two of the row's own, near the largest of these products: neither the size of
//   a key that the row does not see nor that of one of no weight costs the others their bits, and
//   weights that fp16 does not hold count where their values are as large. (So a tile is taken
//   whose values are all far larger than those before.)
// * What is left of a key, m_j + 8 s_j, is the same for all its dimensions and meets
//   sum(q): a further step of the first product, with both in two fp16 terms (22 bits),
//   adds it to S; the keys' second terms are held 2^11 up, so that they are not below fp16's
//   range for keys far smaller than the tile's largest. (As an fma a logit in the softmax, with
//   the keys' terms read from shared memory, it took 2.08 ms where this took 1.83, the 8K chunk
//   behind 8K tokens.) Likewise sum p_j (m_j + 8 s_j) is summed in fp32 beside O. So the one
//   rounding of the product is that of p to fp16.
// * Rows are the new tokens times the query heads of one kv head, so that a key is
//   decoded once for all the heads that read it.
// * Two row tiles (256 rows) share each decoded key tile; their products alternate, so
//   that one softmax runs while the other's products do. Windows of up to 128 rows use
//   both warpgroups on the same rows, each on every other key tile.
// * Work is cut as in the window kernel: runs of equal cost over the CTAs, in key tiles.
//
// Measured: 8192 tokens behind 8192, 32/8 heads of 128, 1.65 ms, 1000 TFLOP/s of the causal
// products (52% of the library's rate): softmax, key and value warps each need 4500 to 5000
// cycles for a step of 256 rows x 128 keys, the products 2300. 16 windows of 8 tokens over up
// to 32K tokens, 20/4 heads of 128, 107 us, 1.2 TB/s of cache: the key warps are busy all of
// the time (some 4000 cycles a tile), the others wait for them. 6 ragged chunks of up to 1001
// tokens, 16 heads of 64, 92 us.
// Behind shared prefixes (kPrefix without a causal order, its pieces joined by a kernel of its own; kJoined the own
// parts, beside and behind that): 64 requests of a token behind 16384 tokens, 32/8 heads of 128, prefix some 30 us, join 8,
// with the window kernel's own parts 53 in all. 16 windows of up to 8 tokens behind 83K tokens in three prefixes, 20/4
// heads, prefix 57 us, 92 in all. 6 chunks of up to 501 tokens behind two prefixes of 5K, 16 heads of 64, fp16, prefix 97
// us, 148 in all.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "hc_window.cuh"

namespace hc {
namespace {

constexpr int kThreads = 512;
constexpr int kTile = 128;                 // keys of a tile, rows of a row tile
constexpr int kStages = 2;                 // key tiles and value tiles in shared memory
constexpr int kCols = 4;                   // column data of tiles (see Column)
constexpr int kPieceCost = 5;              // what a piece costs beside its tiles, in tiles (ragged chunks:
                                           // 104 us with 1, 99 with 2, 96 with 5)
constexpr float kRaise = 8.f;              // log2 by which a logit may pass the maximum before it is raised
constexpr float kMost = 15.f;              // and the most that a weight may have as fp16
constexpr int kPieceFloats = 256 * 128 + 512;

// What softmax needs of a tile's keys beside S and P. Four of them: a tile's data is
// rewritten for the tile four later, whose keys are decoded only after the products of the
// tile two later, which follow the softmax of this one.
struct alignas(16) Column {
    float v[kTile];                        // m + 8 s of the values
    float up[2];                           // 2^E of K', in two factors
    int ev;                                // E of V'
    int wide[2];                           // whether keys, values have an E of their own each
    int16_t e[2][kTile];                   // E of each key and value
};
static_assert(sizeof(Column) % 16 == 0, "Column::v is read 16 bytes at a time");
constexpr int kSpan = 8;                   // log2 of how far apart the steps of a tile with one E may lie
constexpr int kRise = 10;                  // by how much E of V' may pass a row's unit: a weight far below 1 may matter then
constexpr int kLower = 64;                 // and by how much E of V' may fall below the largest so far: O stays within fp32

template <int kD>
struct Smem {
    static constexpr int kOne = kTile * kD * 2;                        // a decoded tile, a row tile
    static constexpr int kQ = 0;
    static constexpr int kK = 2 * kOne;
    static constexpr int kV = kK + kStages * kOne;
    static constexpr int kColumn = kV + kStages * kOne;
    static constexpr int kSteps = kColumn + kCols * static_cast<int>(sizeof(Column));   // fp16 S [values?][tile parity]
    // the further step of the first product: [rows][16], of a row tile and of a key tile
    static constexpr int kMore = kTile * 32;
    static constexpr int kQMore = (kSteps + 4 * kTile * 2 + 255) / 256 * 256;
    static constexpr int kKMore = kQMore + 2 * kMore;
    static constexpr int kBytes = kKMore + kStages * kMore + 1024;     // and room to align
};

struct Bars {
    uint64_t s_full[2], o_done[2];
    uint64_t k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages], col_full[kCols];
};

// The walk through a CTA's run: as in the window kernel, with row tiles.
struct Walk {
    int b, h, row0;              // request, kv head, first row of the row tile
    int rows;                    // rows of the tile that exist
    int t0, t1, tiles;           // key tiles [t0, t1) of `tiles`
    int64_t left, base;
    Window w;
};

// Row tiles of a window, and the key tiles that row tile i sees.
__device__ __forceinline__ int row_tiles(const Window& w, int group, int step) {
    return (w.rows * group + step - 1) / step;
}
template <Side kSide>
__device__ __forceinline__ int key_tiles(const Args<kSide>& a, const Window& w, int group, int step, int i) {
    const int last = min(((i + 1) * step - 1) / group, w.rows - 1);
    const int seen = kSide == kPrefix || a.mask ? w.kv : min(w.kv, w.first + last + 1);
    return max((seen - 1) / kTile + 1, 1);     // (seen may be 2^31 - 1)
}
template <Side kSide>
__device__ __forceinline__ int64_t head_slots(const Args<kSide>& a, const Window& w, int group, int step) {
    int64_t n = 0;
    for (int i = row_tiles(w, group, step) - 1; i >= 0; --i) n += key_tiles<kSide>(a, w, group, step, i) + kPieceCost;
    return n;
}

__device__ __forceinline__ bool walk_piece(Walk& k, int from) {
    const int64_t to = min(static_cast<int64_t>(k.tiles + kPieceCost), from + k.left);
    k.left -= to - from;
    k.t0 = max(from - kPieceCost, 0);
    k.t1 = static_cast<int>(to) - kPieceCost;
    return k.t1 > k.t0;
}

template <Side kSide>
__device__ __forceinline__ void walk_row_tile(const Args<kSide>& a, Walk& k, int group, int step, int i) {
    k.row0 = i * step;
    k.rows = min(k.w.rows * group - k.row0, step);
    k.tiles = key_tiles<kSide>(a, k.w, group, step, i);
}

template <Side kSide>
__device__ __forceinline__ bool walk_next(const Args<kSide>& a, Walk& k, int group, int step) {
    if (k.left == 0) return false;
    k.base += k.tiles + kPieceCost;
    int i = k.row0 / step + 1;
    if (i == row_tiles(k.w, group, step)) {
        i = 0;
        if (++k.h == a.c.kv_heads) {
            k.h = 0;
            do {
                ++k.b;
                if (k.b >= a.requests) return false;
                k.w = load_window<kSide>(a, k.b, nullptr);
            } while (row_tiles(k.w, group, step) == 0);
        }
    }
    walk_row_tile<kSide>(a, k, group, step, i);
    return walk_piece(k, 0);
}

struct Run {
    int b;
    int64_t offset, head, begin, end, total, ctas;
    Window w;                    // of request b
};

template <Side kSide>
__device__ void find_run(const Args<kSide>& a, int group, int step, Run* run, int64_t* sums, int* status) {
    const int tid = threadIdx.x;
    const int per = (a.requests - 1) / kThreads + 1;             // (of up to 2^31 - 1)
    const int b0 = static_cast<int>(min(static_cast<int64_t>(tid) * per, static_cast<int64_t>(a.requests))), b1 = b0 + min(per, a.requests - b0);
    int64_t mine = 0;
    Window w = {};                               // the last of them, which is the only one up to kThreads requests
    for (int b = b0; b < b1; ++b) {
        w = load_window<kSide>(a, b, blockIdx.x == 0 ? status : nullptr);
        mine += head_slots<kSide>(a, w, group, step) * a.c.kv_heads;
    }
    int64_t upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t t = __shfl_up_sync(~0u, upto, d);
        if ((tid & 31) >= d) upto += t;
    }
    if ((tid & 31) == 31) sums[tid >> 5] = upto;
    __syncthreads();
    int64_t total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w == (tid >> 5)) upto += total;
        total += sums[w];
    }
    const int64_t ctas = min(static_cast<int64_t>(gridDim.x), total), i = blockIdx.x;
    const int64_t begin = i < ctas ? quotient(total * i, ctas) : total, end = i < ctas ? quotient(total * (i + 1), ctas) : total;
    if (tid == 0) {
        run->begin = begin;
        run->end = end;
        run->total = total;
        run->ctas = ctas;
    }
    if (begin < end && begin < upto && begin >= upto - mine) {
        int64_t at = upto - mine;
        for (int b = b0; b < b1; ++b) {
            if (b1 - b0 > 1) w = load_window<kSide>(a, b, nullptr);
            const int64_t head = head_slots<kSide>(a, w, group, step), n = head * a.c.kv_heads;
            if (begin < at + n) {
                run->b = b;
                run->w = w;
                run->offset = begin - at;
                run->head = head;
                break;
            }
            at += n;
        }
    }
    __syncthreads();
}

template <Side kSide>
__device__ __forceinline__ bool walk_start(const Args<kSide>& a, const Run& run, int group, int step, Walk& k) {
    if (run.begin >= run.end) return false;
    k.b = run.b;
    k.w = run.w;
    k.h = static_cast<int>(quotient(run.offset, run.head));
    int64_t from = run.offset - k.h * run.head;
    int i = 0;
    while (true) {
        walk_row_tile<kSide>(a, k, group, step, i);
        if (from < k.tiles + kPieceCost) break;
        from -= k.tiles + kPieceCost;
        ++i;
    }
    k.left = run.end - run.begin;
    k.base = run.begin - from;
    return walk_piece(k, static_cast<int>(from)) || walk_next<kSide>(a, k, group, step);
}

// ---- tensor memory

__device__ __forceinline__ void tmem_load32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_store32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_store16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
        : "memory");
}
// Eight floats of shared memory as pairs.
__device__ __forceinline__ void load_pairs(const float* p, uint64_t (&v)[4]) {
    asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(v[0]), "=l"(v[1]) : "r"(tc::smem_u32(p)));
    asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(v[2]), "=l"(v[3]) : "r"(tc::smem_u32(p) + 16));
}
__device__ __forceinline__ void tmem_load16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_load() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Descriptor of a K-major tile of 16 16-bit elements a row stored with the 32-byte swizzle (8-row
// atoms of 256 bytes), and the byte offset of 16-byte chunk c of row r in it.
__device__ __forceinline__ uint64_t desc_sw32(uint32_t saddr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>(1) << 16;
    d |= static_cast<uint64_t>(256 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(6) << 61;
    return d;
}
__device__ __forceinline__ uint32_t sw32_offset(int r, int c) { return r * 32 + ((c ^ ((r >> 2) & 1)) << 4); }

// x in two fp16 terms.
__device__ __forceinline__ void split2(float x, float low_up, __half& hi, __half& lo) {
    hi = __float2half_rn(x);
    lo = __float2half_rn((x - __half2float(hi)) * low_up);
}
constexpr float kMoreUp = 256.f;             // 2^8: the keys' terms up, the queries' down
constexpr float kLowUp = 2048.f;             // 2^11: the keys' second term up once more, and the queries' terms for it down

// True in one thread of a converged warp.
__device__ __forceinline__ bool elected() {
    uint32_t p;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(p));
    return p != 0;
}

// D[tmem] (+)= A[tmem] * B[smem]^T, issued by one thread.
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{ .reg .pred p; setp.ne.b32 p, %4, 0; "
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate ? 1u : 0u));
}

// A decoded word scaled: pairs 0 and 2 hold c 2^-24, pairs 1 and 3 c 2^-20; s = (S, S'), the
// steps of the two codes of a pair, and s16 = s / 16, low = -8 2^-24 s.
__device__ __forceinline__ void scale_word(uint32_t (&h)[4], __half2 s, __half2 s16, __half2 low) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 r = __hfma2(*reinterpret_cast<__half2*>(&h[i]), (i & 1) ? s16 : s, low);
        h[i] = *reinterpret_cast<const uint32_t*>(&r);
    }
}

// kSame: both warpgroups have the same rows.
template <int kD, int kDtype, bool kSame, Side kSide>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_kernel(const Args<kSide> a, float* scratch, unsigned* arrivals, int* status) {
    // also before tensor memory is taken, which the kernel before may hold. (Not so the own part behind a prefix:
    // the kernel before it, which ends the prefix and has none, began after all that this one reads was written
    // and after tensor memory was given back. It waits where it first touches what the two have in common.)
    if (kSide != kJoined) pdl_wait();
    if (kSide == kPrefix) pdl_launch_dependents();
    using S = Smem<kD>;
    constexpr bool same = kSame;
    // registers of a softmax thread and of a decoding one, 512 in all for two of each
    constexpr int kMany = kSame ? 152 : 168, kFew = 256 - kMany;
    static_assert(2 * (kMany + kFew) * 128 <= 65536);
    extern __shared__ unsigned char smem_raw[];
    __shared__ Bars bars;
    __shared__ Run run;
    __shared__ int64_t sums[kThreads / 32];
    __shared__ uint32_t tmem_slot;
    __shared__ unsigned last_one[2];
    __shared__ uint2 step_ends[2][2][4];       // largest and smallest, [keys or values][tile parity][warp]
    __shared__ volatile int abort_flag;
    // Each warpgroup's walk, kept here and not in registers: a spilled register of the loops
    // below is a trip to L2, since shared memory leaves L1 no room.
    __shared__ Walk walks[4];
    __shared__ int walking[4];
    unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    Column* columns = reinterpret_cast<Column*>(smem + S::kColumn);
    const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;   // uniform
    const int group = a.q_heads / a.c.kv_heads;
    const int step = same ? kTile : 2 * kTile;         // rows of a piece

    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&bars.s_full[i], 1);
            tc::mbar_init(&bars.o_done[i], 1);
        }
        for (int i = 0; i < kStages; ++i) {
            tc::mbar_init(&bars.k_full[i], 128);
            tc::mbar_init(&bars.k_empty[i], 2);     // one for each row tile
            tc::mbar_init(&bars.v_full[i], 128);
            tc::mbar_init(&bars.v_empty[i], 2);
        }
        for (int i = 0; i < kCols; ++i) tc::mbar_init(&bars.col_full[i], 256);
        tc::fence_barrier_init();
    }
    if (warp == 0) tc::tmem_alloc(&tmem_slot, 512);
    tc::tc_fence_before();
    find_run<kSide>(a, group, step, &run, sums, status);      // synchronises
    tc::tc_fence_after();
    const uint32_t tmem = tmem_slot;
    Walk& k = walks[warp >> 2];
    int& on = walking[warp >> 2];
    const bool leads = (threadIdx.x & 127) == 0;
    if (leads) on = walk_start<kSide>(a, run, group, step, k);
    __syncthreads();
    // to the next piece, by all threads of a warpgroup (named barrier `bar`) that are done with this one
    auto advance = [&](int bar) {
        asm volatile("bar.sync %0, 128;" ::"r"(bar) : "memory");
        if (leads) on = walk_next<kSide>(a, k, group, step);
        asm volatile("bar.sync %0, 128;" ::"r"(bar) : "memory");
    };

    // Every wait is bounded (tc::mbar_wait); one that gives up raises the abort flag, after
    // which the others return at once: the roles then run to their ends on whatever is there.
    auto wait = [&](uint64_t& bar, uint32_t phase) { tc::mbar_wait(&bar, phase & 1, &abort_flag, status); };

    if (warp < 8) {
        // ------------------------------------------------------------------ softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kMany));
        const int wg = warp >> 2, row = threadIdx.x & 127;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t s_mem = tmem + lanes + wg * kTile, o_mem = tmem + lanes + 2 * kTile + wg * kTile;
        unsigned char* q_tile = smem + S::kQ + wg * S::kOne;
        uint32_t s_phase = 0, o_phase = 0;
        uint32_t column = 0;                           // tiles before this one, over all pieces
        constexpr uint32_t kS = tc::idesc_f16_f32(kTile, kTile), kO = tc::idesc_f16_f32(kTile, kD);
        const uint64_t q_desc = tc::desc_sw128(tc::smem_u32(q_tile));
        unsigned char* q_more = smem + S::kQMore + wg * S::kMore;
        const uint64_t qm_desc = desc_sw32(tc::smem_u32(q_more)), km_desc = desc_sw32(tc::smem_u32(smem + S::kKMore));
        const uint64_t k_desc = tc::desc_sw128(tc::smem_u32(smem + S::kK)), v_desc = tc::desc_sw128(tc::smem_u32(smem + S::kV));
        constexpr uint32_t kStageStep = S::kOne / 16, kAtom = kTile * 128 / 16, kAtomV = kD * 128 / 16;   // in the descriptors' 16 bytes
        // The products of this row tile, issued by one thread of its first warp (the warp stays
        // together, so that descriptors are uniform). S of the tile that is number c of all:
        auto issue_s = [&](uint32_t c, bool alone) {
            const uint32_t stage = c % kStages;
            wait(bars.k_full[stage], c / kStages);
            tc::tc_fence_after();
            const uint64_t kb = k_desc + stage * kStageStep;
            if (elected()) {
#pragma unroll
                for (int x = 0; x < kD / 16; ++x) {
                    const uint32_t off = (x >> 2) * kAtom + (x & 3) * 2;
                    tc::mma_f16(tmem + wg * kTile, q_desc + off, kb + off, kS, x > 0);
                }
                tc::mma_f16(tmem + wg * kTile, qm_desc, km_desc + stage * (S::kMore / 16), kS, true);
                tc::mma_commit(&bars.s_full[wg]);
                tc::mma_commit(&bars.k_empty[stage]);
                if (alone) tc::mma_commit(&bars.k_empty[stage]);
            }
            __syncwarp();
        };
        // and P V', which follows S's reader and comes before S's next writer in issue order
        auto issue_o = [&](uint32_t c, bool alone, bool more) {
            const uint32_t stage = c % kStages;
            wait(bars.v_full[stage], c / kStages);
            tc::tc_fence_after();
            const uint64_t vb = v_desc + stage * kStageStep;
            if (elected()) {
#pragma unroll
                for (int n = 0; n < kTile / 16; ++n)
                    mma_ts(tmem + 2 * kTile + wg * kTile, tmem + wg * kTile + n * 8, vb + (n >> 2) * kAtomV + (n & 3) * 2, kO, n > 0 || more);
                tc::mma_commit(&bars.o_done[wg]);
                tc::mma_commit(&bars.v_empty[stage]);
                if (alone) tc::mma_commit(&bars.v_empty[stage]);
            }
            __syncwarp();
        };
        while (on) {
            const bool active = same || wg == 0 || k.rows > kTile;    // this warpgroup has rows
            // This thread's row, worked out anew for each use: what it would cost to keep is
            // registers of the loop over the tiles.
            struct Row {
                bool here;
                int i, hq;                             // token of the window, query head
            };
            auto my_row = [&]() {
                int x = row;
                asm volatile("" : "+r"(x));            // not the values of an earlier use
                const int r = k.row0 + (same ? 0 : wg * kTile) + x;
                return Row{r < k.row0 + k.rows, r / group, k.h * group + r % group};
            };
            float factor = 0.f, qsum = 0.f;
            if (active) {
                // ---- this warp's rows of Q: scaled to fp16, in the order of the decoded keys. A row is brought by
                // neighbouring lanes, 16 bytes each. (A row a thread touches 32 lines with each load: the start of
                // 256 rows took 12000 cycles of an L1 that looks up a line a cycle, where this takes 7000.)
                const Row m = my_row();
                const int64_t own = static_cast<int64_t>(k.w.begin + m.i) * a.q_token + static_cast<int64_t>(m.hq) * a.q_head;
                const int64_t from = m.here && HC_IN_RANGE(own, kD, row_extent(a.tokens, a.q_heads, kD, a.q_token, a.q_head), status) ? own : -1;
                constexpr int kOfRow = kD / 8, kRowsAt = 32 / kOfRow;  // lanes of a row, rows at a time
                const int c = lane % kOfRow;
                uint4 ahead[4];
                auto fetch = [&](int turn) {
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        const int64_t at = __shfl_sync(~0u, from, (turn + n) * kRowsAt + lane / kOfRow);
                        ahead[n] = at >= 0 ? *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + at + 8 * c) : make_uint4(0, 0, 0, 0);
                    }
                };
                fetch(0);
                float my_top = 0.f;
#pragma unroll 1
                for (int turn0 = 0; turn0 < 32 / kRowsAt; turn0 += 4) {
                    const uint4 four[4] = {ahead[0], ahead[1], ahead[2], ahead[3]};
                    if (turn0 + 4 < 32 / kRowsAt) fetch(turn0 + 4);
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        const uint32_t x[4] = {four[n].x, four[n].y, four[n].z, four[n].w};
                        float top = 0.f;
#pragma unroll
                        for (int p = 0; p < 4; ++p) {
                            const float2 y = widen2<kDtype>(x[p]);
                            top = fmaxf(top, fmaxf(fabsf(y.x), fabsf(y.y)));
                        }
#pragma unroll
                        for (int d = 1; d < kOfRow; d <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
                        const float down = power_of_two(-query_exponent(top));
                        float f[8];
#pragma unroll
                        for (int p = 0; p < 4; ++p) {
                            const float2 y = widen2<kDtype>(x[p]);
                            f[2 * p] = y.x * down, f[2 * p + 1] = y.y * down;
                        }
                        const int to = (warp & 3) * 32 + (turn0 + n) * kRowsAt + lane / kOfRow;
                        *reinterpret_cast<uint4*>(q_tile + (c >> 3) * (kTile * 128) + tc::sw128_offset(to, (c & 7) * 8)) =
                            make_uint4(pack_half2(f[0], f[4]), pack_half2(f[1], f[5]), pack_half2(f[2], f[6]), pack_half2(f[3], f[7]));
                        const float theirs = __shfl_sync(~0u, top, (lane % kRowsAt) * kOfRow);
                        if (lane / kRowsAt == turn0 + n) my_top = theirs;
                    }
                }
                factor = a.scale * kLog2e * power_of_two(query_exponent(my_top));
                __syncwarp();
#pragma unroll 4
                for (int x = 0; x < kD / 8; ++x) {
                    const uint4 o4 = *reinterpret_cast<const uint4*>(q_tile + (x >> 3) * (kTile * 128) + tc::sw128_offset(row, (x & 7) * 8));
                    const uint32_t o[4] = {o4.x, o4.y, o4.z, o4.w};
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&o[p]));
                        qsum += y.x + y.y;
                    }
                }
                // sum(q), met by the keys' m + 8 s
                __half hi, lo;
                split2(qsum * (1.f / kMoreUp), 1.f, hi, lo);
                const __half2 both = __halves2half2(hi, lo), less = __hmul2(both, __float2half2_rn(1.f / kLowUp));
                *reinterpret_cast<uint4*>(q_more + sw32_offset(row, 0)) =
                    make_uint4(*reinterpret_cast<const uint32_t*>(&both), *reinterpret_cast<const uint32_t*>(&less), 0, 0);
                *reinterpret_cast<uint4*>(q_more + sw32_offset(row, 1)) = make_uint4(0, 0, 0, 0);
                tc::fence_proxy_async_smem();
            }
            // this row tile's key tiles: all, or every other one, which then no other row tile uses
            const int stride = same ? 2 : 1, j0 = k.t0 + (same ? wg : 0);
            const bool alone = same || k.rows <= kTile;
            if (active) {
                asm volatile("bar.sync %0, 128;" ::"r"(2 + wg) : "memory");
                if ((warp & 3) == 0 && j0 < k.t1) issue_s(column + (j0 - k.t0), alone);
            }

            float base = 0.f, sum = 0.f, flat = 0.f;
            bool fresh = true;
            float later = 1.f;                         // what O is to be multiplied by before its next product
            int ev = 1000, done_tiles = 0;             // (above any E, until the first tile)
            const int t1 = k.t1;
            const int clear = kSide == kPrefix ? k.w.kv : min(k.w.kv, a.mask ? k.w.first : k.w.first + 1 + k.row0 / group);   // every row sees what lies before
            for (int j = k.t0; j < t1; ++j, ++column) {
                if (!active || (same && ((j - j0) & 1))) continue;
                const Column& col = columns[column % kCols];
                wait(bars.col_full[column % kCols], column / kCols);
                wait(bars.s_full[wg], s_phase++);
                __syncwarp();
                tc::tc_fence_after();
                // (all ask the same of shared memory: the vote tells the compiler that they branch together)
                const bool wide = __any_sync(~0u, (col.wide[0] | col.wide[1] | max(col.ev - ev - kRise, 0)) != 0);
                const float f = wide ? 1.f : factor * col.up[0] * col.up[1];
                int to = col.ev;                             // 2^to: the unit of O with this tile
                // hidden keys: behind the end, or behind this row's token, or out of its mask
                const int t = j * kTile;
                const bool tail = t > clear - kTile;
                float fix = 1.f, peak = -CUDART_INF_F;
                const uint64_t f2 = pair(f, f);
                // of this tile alone: sums of millions of keys would not notice one key's weight
                uint64_t sum2 = 0, flat2 = 0;
                bool quick = !tail && !wide && __ballot_sync(~0u, fresh) == 0;
                if (quick) {
                    // Weights against the maximum so far, 32 keys at a time, two to an instruction,
                    // held as P until all are known to be within fp16; and their products with what is
                    // common to a value's dimensions.
                    const uint64_t b2 = pair(-base, -base);
                    uint32_t pw[4][16], ahead[2][16];
                    uint64_t vo[4];                              // of 8 keys
                    load_pairs(&col.v[0], vo);
                    tmem_load16(s_mem, ahead[0]);
#pragma unroll
                    for (int part = 0; part < 8; ++part) {
                        tmem_wait_load();
                        uint32_t(&raw)[16] = ahead[part & 1];
                        if (part < 7) tmem_load16(s_mem + (part + 1) * 16, ahead[(part + 1) & 1]);
#pragma unroll
                        for (int c = 0; c < 16; c += 8) {
                            uint64_t vn[4] = {};                 // the next eight keys'
                            if (part * 16 + c + 8 < kTile) load_pairs(&col.v[part * 16 + c + 8], vn);
                            float e[8];
#pragma unroll
                            for (int n = 0; n < 4; ++n) {
                                const float2 x = unpair(fma2(pair(__uint_as_float(raw[c + 2 * n]), __uint_as_float(raw[c + 2 * n + 1])), f2, b2));
                                peak = max3(peak, x.x, x.y);
                                e[2 * n] = exp2_fast(x.x), e[2 * n + 1] = exp2_fast(x.y);
                                const uint64_t w = pair(e[2 * n], e[2 * n + 1]);
                                sum2 = add2(sum2, w);
                                flat2 = fma2(w, vo[n], flat2);
                            }
#pragma unroll
                            for (int n = 0; n < 4; ++n) vo[n] = vn[n];
                            // P: column x * 8 + n of each 32 is token n * 4 + x, the order of the decoded values
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                pw[part >> 1][4 * x + 2 * (part & 1) + c / 8] = pack_half2(e[x], e[4 + x]);
                        }
                    }
                    quick = !__any_sync(~0u, peak > kMost);
                    if (quick) {
#pragma unroll
                        for (int n = 0; n < 4; ++n) tmem_store16(s_mem + n * 16, pw[n]);
                    }
                }
                if (!quick) {
                    // In two passes, the maximum first: tiles with hidden keys, a row's first tile, wide
                    // tiles, and those whose logits pass the maximum by so much that the weights overflow.
                    // Rolled: what every tile runs has to stay in the instruction cache.
                    const Row m = my_row();
                    const int limit = (kSide == kPrefix || a.mask ? k.w.kv : min(k.w.kv, k.w.first + m.i + 1)) - t;
                    uint32_t seen[4];                            // one bit a key
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        const int left = limit - 32 * n;
                        seen[n] = left >= 32 ? ~0u : left <= 0 ? 0u : (1u << left) - 1u;
                    }
                    if (kSide != kPrefix && a.mask) {
                        // bit 0 of `bits` is the key at `at`; keys before it are seen
                        const uint64_t bits = m.here && HC_IN_RANGE(k.w.begin + m.i, 1, a.tokens, status) ? a.mask[k.w.begin + m.i] : 0;
                        const int at = k.w.first - t;
#pragma unroll
                        for (int n = 0; n < 4; ++n) {
                            const int from = 32 * n - at;        // bit of this word's first key
                            uint32_t word;
                            if (from <= -32) word = ~0u;
                            else if (from < 0) word = (static_cast<uint32_t>(bits) << -from) | ((1u << -from) - 1u);
                            else word = from < 64 ? static_cast<uint32_t>(bits >> from) : 0u;
                            seen[n] &= word;
                        }
                    }
                    float most = -CUDART_INF_F;                  // of a wide tile, the largest logit + E of its value
                    if (wide) {
                        // S becomes the logits: each key has an exponent of its own
#pragma unroll 1
                        for (int n = 0; n < 8; ++n) {
                            uint32_t raw[16];
                            tmem_load16(s_mem + n * 16, raw);
                            tmem_wait_load();
                            const uint32_t visible = (n < 4 ? n < 2 ? seen[0] : seen[1] : n < 6 ? seen[2] : seen[3]) >> (n & 1) * 16;
#pragma unroll
                            for (int c = 0; c < 16; ++c) {
                                const int e = col.e[0][n * 16 + c];
                                const float x = __uint_as_float(raw[c]) * (factor * power_of_two(e >> 1)) * power_of_two(e - (e >> 1));
                                raw[c] = __float_as_uint(x);
                                if ((visible >> c) & 1) most = fmaxf(most, x + static_cast<float>(col.e[1][n * 16 + c]));
                            }
                            tmem_store16(s_mem + n * 16, raw);
                        }
                        tmem_wait_store();
                    }
                    peak = -CUDART_INF_F;
#pragma unroll 1
                    for (int n = 0; n < 4; ++n) {
                        uint32_t raw[32];
                        tmem_load32(s_mem + n * 32, raw);
                        tmem_wait_load();
                        const uint32_t visible = n == 0 ? seen[0] : n == 1 ? seen[1] : n == 2 ? seen[2] : seen[3];
#pragma unroll
                        for (int c = 0; c < 32; ++c) {
                            const float x = fmaf(__uint_as_float(raw[c]), f, -base);
                            if ((visible >> c) & 1) peak = fmaxf(peak, x);
                        }
                    }
                    if (fresh ? peak != -CUDART_INF_F : peak > kRaise) {
                        fix = fresh ? 1.f : exp2_fast(-peak);
                        base += peak, sum *= fix, flat *= fix;
                        fresh = false;
                    }
                    peak = 0.f;
                    if (wide) {
                        // the largest weight times 2^E of its value, or what is in O already, is the unit
                        // (a row that sees nothing here keeps its own; the bounds are those of any E)
                        const float kept = fix * later;
                        to = static_cast<int>(ceilf(fminf(fmaxf(most - base, -250.f), 250.f)));
                        if (done_tiles > 0 && kept > 0.f) to = max(to, ev + static_cast<int>(__float_as_uint(kept) >> 23) - 127);
                    }
                    const uint64_t b2 = pair(-base, -base);
                    sum2 = flat2 = 0;
                    // (A loop each, so that what a wide tile does more does not lie between what every tile
                    // does: ragged chunks 97.8 -> 96.3 us. With shared rows two of them spill.)
                    auto weigh = [&](auto scaled) {
#pragma unroll 1
                        for (int n = 0; n < 4; ++n) {
                            uint32_t raw[32];
                            tmem_load32(s_mem + n * 32, raw);
                            tmem_wait_load();
                            const uint32_t visible = n == 0 ? seen[0] : n == 1 ? seen[1] : n == 2 ? seen[2] : seen[3];
                            float e[32];
#pragma unroll
                            for (int c = 0; c < 32; c += 8) {
                                uint64_t vo[4];
                                load_pairs(&col.v[n * 32 + c], vo);
#pragma unroll
                                for (int m = 0; m < 4; ++m) {
                                    const int c2 = c + 2 * m;
                                    const float2 x = unpair(fma2(pair(__uint_as_float(raw[c2]), __uint_as_float(raw[c2 + 1])), f2, b2));
                                    float2 v = unpair(vo[m]);        // a hidden value may be NaN
                                    if ((visible >> c2) & 1) e[c2] = exp2_fast(x.x);
                                    else e[c2] = 0.f, v.x = 0.f;
                                    if ((visible >> (c2 + 1)) & 1) e[c2 + 1] = exp2_fast(x.y);
                                    else e[c2 + 1] = 0.f, v.y = 0.f;
                                    const uint64_t w = pair(e[c2], e[c2 + 1]);
                                    sum2 = add2(sum2, w);
                                    flat2 = fma2(w, pair(v.x, v.y), flat2);
                                }
                            }
                            if (scaled) {
                                // (a weight that 2^126 would not bring up is 0)
#pragma unroll
                                for (int c = 0; c < 32; ++c) {
                                    const int up = col.e[1][n * 32 + c] - to;
                                    e[c] *= power_of_two(min(max(up, -126), 126));
                                }
                            }
                            uint32_t p[16];
#pragma unroll
                            for (int c = 0; c < 4; ++c)
#pragma unroll
                                for (int m = 0; m < 4; ++m) p[4 * c + m] = pack_half2(e[8 * m + c], e[8 * m + 4 + c]);
                            tmem_store16(s_mem + n * 16, p);         // over keys that have been read
                        }
                    };
                    if constexpr (kSame) weigh(wide);
                    else if (wide) weigh(std::true_type());
                    else weigh(std::false_type());
                }
                {
                    const float2 s2 = unpair(sum2), l2 = unpair(flat2);
                    sum += s2.x + s2.y, flat += l2.x + l2.y;
                }
                fix *= later, later = 1.f;
                if (done_tiles == 0) {
                    ev = to;
                } else {
                    const bool other = to != ev;
                    if (__any_sync(~0u, fix != 1.f || other)) {
                        // O of the tiles before is complete, and this warp's lanes of it are rescaled
                        wait(bars.o_done[wg], o_phase + done_tiles - 1);
                        __syncwarp();
                        tc::tc_fence_after();
                        const float by = other ? ldexpf(fix, ev - to) : fix;
                        ev = to;
#pragma unroll 1
                        for (int c = 0; c < kD / 32; ++c) {
                            uint32_t v[32];
                            tmem_load32(o_mem + c * 32, v);
                            tmem_wait_load();
#pragma unroll
                            for (int n = 0; n < 32; ++n) v[n] = __float_as_uint(__uint_as_float(v[n]) * by);
                            tmem_store32(o_mem + c * 32, v);
                        }
                    }
                }
                tmem_wait_store();
                tc::tc_fence_before();
                asm volatile("bar.sync %0, 128;" ::"r"(2 + wg) : "memory");
                if ((warp & 3) == 0) {
                    issue_o(column, alone, done_tiles > 0);
                    if (j + stride < t1) issue_s(column + stride, alone);
                }
                ++done_tiles;
                // a maximum that was passed is raised for the tiles to come
                if (peak > kRaise) {
                    later = exp2_fast(-peak);
                    sum *= later, flat *= later, base += peak;
                }
            }
            // ---- the end of the piece
            if (done_tiles > 0) {
                wait(bars.o_done[wg], o_phase + done_tiles - 1);
                __syncwarp();
                tc::tc_fence_after();
            }
            o_phase += done_tiles;
            if (fresh && sum == sum) base = -CUDART_INF_F;     // (a sum of NaN alone has to be told, about 0)
            if (kSide == kJoined) pdl_wait();                  // scratch and counters are free, the prefix's part is there
            const bool whole = k.t0 == 0 && k.t1 == k.tiles;
            float other_base = -CUDART_INF_F, other_sum = 0.f;
            float* exchange = reinterpret_cast<float*>(smem + S::kQ);          // [kD][128], both row tiles' room
            __shared__ float2 stats[kTile], joined[2][kTile];
            __shared__ float by_prefix[kSide == kJoined ? 2 : 1][kSide == kJoined ? kTile : 1];
            if (same) {
                // the two warpgroups' sums over the same rows
                asm volatile("bar.sync 1, 256;" ::: "memory");         // no product reads Q any more
                if (wg == 1) {
                    stats[row] = make_float2(base, sum);
#pragma unroll 1
                    for (int c = 0; c < kD / 32; ++c) {
                        uint32_t v[32];
                        if (done_tiles > 0) tmem_load32(o_mem + c * 32, v);
                        tmem_wait_load();
                        const float up = done_tiles > 0 ? ldexpf(later, ev) : 0.f;
#pragma unroll
                        for (int n = 0; n < 32; ++n)
                            exchange[(c * 32 + n) * kTile + row] = done_tiles > 0 ? fmaf(__uint_as_float(v[n]), up, flat) : 0.f;
                    }
                }
                asm volatile("bar.sync 1, 256;" ::: "memory");
                if (wg == 0) other_base = stats[row].x, other_sum = stats[row].y;
            }
            const bool writes = active && !(same && wg == 1);
            float peak = base, total = sum, mine = base == -CUDART_INF_F ? 0.f : 1.f, other = 0.f;
            const float up = done_tiles > 0 ? ldexpf(later, ev) : 0.f;
            if (same && wg == 0) {
                peak = fmaxf(base, other_base);
                mine = base == -CUDART_INF_F ? 0.f : exp2_fast(base - peak);
                other = other_base == -CUDART_INF_F ? 0.f : exp2_fast(other_base - peak);
                total = sum * mine + other_sum * other;
            }
            const Row mine_row = my_row();
            const int64_t at = static_cast<int64_t>(k.w.begin + mine_row.i) * a.q_heads + mine_row.hq;
            const bool here = mine_row.here && HC_IN_RANGE(at, 1, static_cast<size_t>(a.tokens) * a.q_heads, status);
            float* piece = scratch + (static_cast<int64_t>(blockIdx.x) * 2 + (k.t0 == 0 ? 1 : 0)) * kPieceFloats;
            const int prow = (same ? 0 : wg * kTile) + row;
            auto write = [&](int c, const float (&v)[32], float inv) {
                if constexpr (kSide == kPrefix) {
                    float4* to = reinterpret_cast<float4*>(a.partial + at * kD + c * 32);
#pragma unroll
                    for (int n = 0; n < 8; ++n) to[n] = make_float4(v[4 * n] * inv, v[4 * n + 1] * inv, v[4 * n + 2] * inv, v[4 * n + 3] * inv);
                    return;
                }
                uint4* to = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + at * kD + c * 32);
#pragma unroll
                for (int n = 0; n < 4; ++n)
                    to[n] = make_uint4(narrow2<kDtype>(v[8 * n] * inv, v[8 * n + 1] * inv), narrow2<kDtype>(v[8 * n + 2] * inv, v[8 * n + 3] * inv),
                                       narrow2<kDtype>(v[8 * n + 4] * inv, v[8 * n + 5] * inv), narrow2<kDtype>(v[8 * n + 6] * inv, v[8 * n + 7] * inv));
            };
            if (writes) {
                float inv = total == 0.f ? 0.f : 1.f / total, by_prefix = 0.f, lse = 0.f;
                if constexpr (kSide == kJoined) {
                    if (whole && here) {
                        const Join j = join_parts_of_row(peak, total, __ldcg(partial_stats(a, kD) + at));
                        inv = j.by_own, by_prefix = j.by_prefix, lse = j.lse;
                    }
                }
#pragma unroll 1
                for (int c = 0; c < kD / 32; ++c) {
                    uint32_t v[32];
                    tmem_load32(o_mem + c * 32, v);
                    tmem_wait_load();
                    float o[32];
#pragma unroll
                    for (int n = 0; n < 32; ++n) {
                        o[n] = mine == 0.f ? 0.f : fmaf(__uint_as_float(v[n]), up, flat) * mine;
                        if (same && other != 0.f) o[n] = fmaf(exchange[(c * 32 + n) * kTile + row], other, o[n]);
                    }
                    if (here && whole) {
                        if constexpr (kSide == kJoined) {
                            const float4* prefix = reinterpret_cast<const float4*>(a.partial + at * kD + c * 32);
#pragma unroll
                            for (int n = 0; n < 8; ++n) {
                                const float4 y = __ldcg(prefix + n);
                                o[4 * n] = fmaf(o[4 * n], inv, y.x * by_prefix), o[4 * n + 1] = fmaf(o[4 * n + 1], inv, y.y * by_prefix);
                                o[4 * n + 2] = fmaf(o[4 * n + 2], inv, y.z * by_prefix), o[4 * n + 3] = fmaf(o[4 * n + 3], inv, y.w * by_prefix);
                            }
                            write(c, o, 1.f);
                        } else {
                            write(c, o, inv);
                        }
                    } else if (here) {
#pragma unroll
                        for (int n = 0; n < 8; ++n)
                            __stcg(reinterpret_cast<float4*>(piece) + (c * 8 + n) * 256 + prow,
                                   make_float4(o[4 * n], o[4 * n + 1], o[4 * n + 2], o[4 * n + 3]));
                    }
                    __syncwarp();
                }
                if (whole) {
                    if constexpr (kSide == kPrefix) {
                        if (here) partial_stats(a, kD)[at] = make_float2(peak, total);
                    } else if (here && a.lse) {
                        a.lse[at] = kSide == kJoined ? lse : total == 0.f ? -CUDART_INF_F : (peak + log2f(total)) * kLn2;
                    }
                } else if (here) {
                    __stcg(reinterpret_cast<float2*>(piece + 256 * kD) + prow, make_float2(peak, total));
                }
            }
            tc::tc_fence_before();
            // Both together to the next piece: the exchange is read; and a warpgroup without rows
            // must not run ahead, since a wait tells only whether a phase of its parity is over.
            if (alone) asm volatile("bar.sync 1, 256;" ::: "memory");
            // (pieces of a prefix stay in scratch: a kernel of its own joins them, since they are many: 64
            // requests behind 16384 tokens took 73 us where the last CTA of each head joined them)
            if (kSide != kPrefix && !whole && writes) {
                // each row tile is joined by the last CTA that has part of it
                const int64_t n = run.ctas;
                const int c0 = static_cast<int>(((k.base + kPieceCost + 1) * n - 1) / run.total);
                const int c1 = static_cast<int>(((k.base + kPieceCost + k.tiles) * n - 1) / run.total);
                const bool known = HC_IN_RANGE(c0, c1 - c0 + 1, gridDim.x, status);     // scratch and counters go by CTA
                asm volatile("bar.sync %0, 128;" ::"r"(2 + wg) : "memory");
                if (row == 0) {
                    const unsigned before = known ? arrive(&arrivals[2 * c0 + wg]) : 0u;
                    last_one[wg] = known && before == static_cast<unsigned>(c1 - c0);
                    if (last_one[wg]) arrivals[2 * c0 + wg] = 0;
                }
                asm volatile("bar.sync %0, 128;" ::"r"(2 + wg) : "memory");
                if (last_one[wg]) {
                    auto from = [&](int c) { return scratch + (static_cast<int64_t>(c) * 2 + (c == c0 ? 1 : 0)) * kPieceFloats; };
                    if (here) {
                        float top = -CUDART_INF_F, all = 0.f;
#pragma unroll 8
                        for (int c = c0; c <= c1; ++c) top = fmaxf(top, __ldcg(reinterpret_cast<const float2*>(from(c) + 256 * kD) + prow).x);
#pragma unroll 8
                        for (int c = c0; c <= c1; ++c) {
                            const float2 st = __ldcg(reinterpret_cast<const float2*>(from(c) + 256 * kD) + prow);
                            if (st.x != -CUDART_INF_F) all += st.y * exp2_fast(st.x - top);
                        }
                        joined[wg][row] = make_float2(top, all == 0.f ? 0.f : 1.f / all);
                        float lse = all == 0.f ? -CUDART_INF_F : (top + log2f(all)) * kLn2;
                        if constexpr (kSide == kJoined) {
                            const Join j = join_parts_of_row(top, all, __ldcg(partial_stats(a, kD) + at));
                            joined[wg][row].y = j.by_own, lse = j.lse;
                            by_prefix[wg][row] = j.by_prefix;
                        }
                        if (a.lse) a.lse[at] = lse;
                    }
                    asm volatile("bar.sync %0, 128;" ::"r"(2 + wg) : "memory");
                    // Four dimensions of each half or quarter of a row a thread, of kAhead parts at
                    // a time: their latency is what a join waits for. (A row a thread and part after
                    // part, 30 rows of one request of 16384 tokens took 94 us where this takes 45;
                    // quarters, which suit few parts, make the kernel of shared rows spill: 16
                    // verify windows 115 us with halves, 143 with quarters.)
                    constexpr int kOf = kSame ? 2 : 4, kAhead = kSame ? 6 : 4, kQuads = kD / 4 / kOf;
                    const int rows = same ? k.rows : min(k.rows - wg * kTile, kTile), at_row = prow - row;
                    for (int n = row; n < rows * kQuads; n += 128) {
                        const int r = n % rows, q = n / rows;
                        const float2 join = joined[wg][r];
                        float4 o[kOf] = {};
                        auto join_parts = [&](int c, auto count) {
                            constexpr int kCount = decltype(count)::value;
                            float2 st[kCount];
                            float4 y[kCount][kOf];
#pragma unroll
                            for (int m = 0; m < kCount; ++m) {
                                const float* part = from(c + m);
                                st[m] = __ldcg(reinterpret_cast<const float2*>(part + 256 * kD) + at_row + r);
#pragma unroll
                                for (int x = 0; x < kOf; ++x)
                                    y[m][x] = __ldcg(reinterpret_cast<const float4*>(part) + (x * kQuads + q) * 256 + at_row + r);
                            }
#pragma unroll
                            for (int m = 0; m < kCount; ++m) {
                                if (st[m].x == -CUDART_INF_F) continue;
                                const float by = exp2_fast(st[m].x - join.x);
#pragma unroll
                                for (int x = 0; x < kOf; ++x) {
                                    o[x].x = fmaf(y[m][x].x, by, o[x].x), o[x].y = fmaf(y[m][x].y, by, o[x].y);
                                    o[x].z = fmaf(y[m][x].z, by, o[x].z), o[x].w = fmaf(y[m][x].w, by, o[x].w);
                                }
                            }
                        };
                        int c = c0;
                        for (; c + kAhead <= c1 + 1; c += kAhead) join_parts(c, std::integral_constant<int, kAhead>{});
                        for (; c + 2 <= c1 + 1; c += 2) join_parts(c, std::integral_constant<int, 2>{});
                        if (c <= c1) join_parts(c, std::integral_constant<int, 1>{});
                        const int of = k.row0 + (same ? 0 : wg * kTile) + r;
                        const int64_t to = (static_cast<int64_t>(k.w.begin + of / group) * a.q_heads + k.h * group + of % group) * kD;
                        if (!HC_IN_RANGE(to, kD, static_cast<size_t>(a.tokens) * a.q_heads * kD, status)) continue;
#pragma unroll
                        for (int x = 0; x < kOf; ++x) {
                            const int64_t put = to + (x * kQuads + q) * 4;
                            float4 y = make_float4(o[x].x * join.y, o[x].y * join.y, o[x].z * join.y, o[x].w * join.y);
                            if constexpr (kSide == kJoined) {
                                const float4 prefix = __ldcg(reinterpret_cast<const float4*>(a.partial + put));
                                const float by = by_prefix[wg][r];
                                y.x = fmaf(prefix.x, by, y.x), y.y = fmaf(prefix.y, by, y.y);
                                y.z = fmaf(prefix.z, by, y.z), y.w = fmaf(prefix.w, by, y.w);
                            }
                            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + put) = make_uint2(narrow2<kDtype>(y.x, y.y), narrow2<kDtype>(y.z, y.w));
                        }
                    }
                }
            }
            advance(2 + wg);
        }
    } else {
        // ------------------------------------------------------------------ keys, values
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFew));
        const bool is_v = warp >= 12;
        const int p = threadIdx.x & 127, w = warp & 3;
        const int sh = 31 - __clz(a.c.block_size), in_block = a.c.block_size - 1;
        const int64_t to_values = static_cast<int64_t>(a.c.kv_heads) * a.c.block_size;
        const uint32_t block_bytes = static_cast<uint32_t>(2 * to_values * (kD / 2));
        const __half2 sixteenth = __float2half2_rn(0.0625f), eighth = __float2half2_rn(-4.76837158203125e-7f);   // -8 2^-24
        // Keys: piece u of a thread is 16 bytes, `seg`, of token key_token(u). Values: tokens n * 4
        // + vt (n = 0..7) of the 64-token half vh, kVW words from dimension vd on.
        constexpr int kUnits = kD / 32, kSegs = kD / 32, kVW = kD / 64;
        const int seg = (lane >> 3) % kSegs;
        auto key_token = [&](int u) { return u * (128 / kUnits) + w * (32 / kUnits) + (lane >> 3) / kSegs * 8 + (lane & 7); };
        const int vc = lane & 7, vt = (vc >> 2) * 32 + (vc & 3), vh = w >> 1, vd = ((w & 1) * 4 + (lane >> 3)) * (8 * kVW);
        uint32_t column = 0;
        while (on) {
            // Lanes 0-7 hold the blocks of a tile's eight 16-token parts, looked up a tile ahead. Loads
            // have no conditions: tokens behind the end are read from the last block or one known
            // before, and count for nothing once their scale is taken as 0. (A condition makes the
            // loaded register one of two, joined, and so waited for, long before its use.)
            int ids = 0;
            const int64_t first = (static_cast<int64_t>(k.h) + (is_v ? a.c.kv_heads : 0)) * a.c.block_size;   // group in a block
            const unsigned char* codes = a.c.codes + first * (kD / 2) + (is_v ? vd / 2 : seg * 16);
            const uint32_t* scales = reinterpret_cast<const uint32_t*>(a.c.scales) + first;
            auto look_up = [&](int j) {
                const unsigned t = min(static_cast<unsigned>(j) * kTile + lane * 16, static_cast<unsigned>(max(k.w.kv - 1, 0)));
                const int64_t at = static_cast<int64_t>(k.b) * a.width + (t >> sh);
                if (HC_IN_RANGE(at, 1, table_extent(a), status)) ids = a.table[at];
            };
            uint64_t parts, parts_next = 0;                     // bytes from `codes` to those of lane's part
            auto check = [&](int j) -> uint64_t {
                if (static_cast<unsigned>(ids) >= static_cast<unsigned>(a.c.blocks)) {
                    if (k.w.kv > 0) atomicOr(status, kStatusBounds);
                    ids = 0;                                    // wrong values, from the cache's own memory
                }
                return static_cast<uint64_t>(static_cast<uint32_t>(ids)) * block_bytes +
                       ((static_cast<unsigned>(j) * kTile + lane * 16) & in_block) * (kD / 2);
            };
            // bytes from `codes` to those of token `x` of that tile
            auto place = [&](uint64_t parts, int x) -> uint64_t {
                return __shfl_sync(~0u, parts, x >> 4) + static_cast<uint32_t>((x & 15) * (kD / 2));
            };
            uint32_t raw[16];                                   // keys [kUnits][4], or values [8][kVW]
            uint32_t scale = 0, scale_next = 0;                 // of token p of this tile and the next
            auto load_scale = [&](uint64_t parts) -> uint32_t {
                const uint64_t at = place(parts, p);
                if (!HC_IN_RANGE(first + at / (kD / 2), 1, group_count(a.c), status)) return 0;
                prefetch_l2(a.c.codes + first * (kD / 2) + at);  // its codes are loaded a tile later
                return scales[at / (kD / 2)];
            };
            // (a piece of keys, loaded again as soon as it is decoded; or the values' tokens)
            auto load_keys = [&](int u, uint64_t at) {
                if (!HC_IN_RANGE(codes + at - a.c.codes, 16, group_count(a.c) * (kD / 2), status)) return;
                const uint4 y = *reinterpret_cast<const uint4*>(codes + at);
                raw[4 * u] = y.x, raw[4 * u + 1] = y.y, raw[4 * u + 2] = y.z, raw[4 * u + 3] = y.w;
            };
            auto load_values = [&]() {
#pragma unroll
                for (int n = 0; n < 8; ++n) {
                    const int x = vh * 64 + n * 4 + vt;
                    const uint64_t at = place(parts, x);
                    if (!HC_IN_RANGE(codes + at - a.c.codes, 4 * kVW, group_count(a.c) * (kD / 2), status)) continue;
                    if (kVW == 2) {
                        const uint2 y = *reinterpret_cast<const uint2*>(codes + at);
                        raw[n * kVW] = y.x, raw[n * kVW + kVW - 1] = y.y;
                    } else {
                        raw[n] = *reinterpret_cast<const uint32_t*>(codes + at);
                    }
                }
            };
            // what a group asks of E: its step; of a NaN, 0; of a key whose common part would leave
            // fp16, as much as that does
            auto need = [&](uint32_t scale) {
                const float own = bf16_lo(scale), rest = fabsf(fmaf(8.f, own, bf16_hi(scale)));
                return __float_as_uint(fmaxf(fmaxf(own, 0.f), is_v ? 0.f : rest * (1.f / 32768.f)));
            };
            auto exponent = [&](uint32_t need) { return static_cast<int>(need >> 23) - 127 + 9; };   // a step in [2^-9, 2^-8)
            // the largest and the smallest of a tile, exchanged between the warps a tile ahead
            uint32_t mine = 0;                                  // of token p of the tile told last
            auto tell = [&](uint32_t scale, uint32_t parity) {
                mine = need(scale);
                const uint32_t most = __reduce_max_sync(~0u, mine), least = __reduce_min_sync(~0u, mine - 1u);   // not of 0
                if (lane == 0) step_ends[is_v][parity][w] = make_uint2(most, least);
            };
            look_up(k.t0 + 1);
            const int second = ids;                             // (asked for together with the first)
            look_up(k.t0);
            parts = check(k.t0);
            scale = load_scale(parts);
            auto seen = [&](int j, uint32_t scale) { return static_cast<unsigned>(j) * kTile + p < static_cast<unsigned>(k.w.kv) ? scale : 0u; };
            if (is_v) {
                load_values();
            } else {
#pragma unroll
                for (int u = 0; u < kUnits; ++u) load_keys(u, place(parts, key_token(u)));
            }
            ids = second;
            parts = check(k.t0 + 1);
            scale_next = load_scale(parts);
            look_up(k.t0 + 2);
            scale = seen(k.t0, scale);
            tell(scale, column & 1);
            asm volatile("bar.sync %0, 128;" ::"r"(4 + is_v) : "memory");
            int e = 0, e_most = -1000;
            for (int j = k.t0; j < k.t1; ++j, ++column) {
                const int stage = column % kStages, turn = column / kStages;
                // E: the largest step of K' in [2^-9, 2^-8); of V', kept while the steps are in its range
                const uint2* ends = step_ends[is_v][column & 1];
                const uint32_t top = max(max(ends[0].x, ends[1].x), max(ends[2].x, ends[3].x));
                const uint32_t low = min(min(ends[0].y, ends[1].y), min(ends[2].y, ends[3].y)) + 1u;
                const int e_top = exponent(top), e_low = exponent(low);
                bool wide = false;
                if (top) {
                    if (!is_v) {
                        e = e_top;
                    } else if (e_top > e || e_low < e - kSpan || e_most < -999) {
                        e_most = max(e_most, e_top);
                        e = max(e_top, e_most - kLower);
                    }
                    wide = e_low < e - kSpan;
                }
                int e_mine = e;
                if (wide && mine) e_mine = exponent(mine);
                // the softmax of the tile four before has been through with its column: see Column
                if (turn > 0) wait(is_v ? bars.v_empty[stage] : bars.k_empty[stage], turn - 1);
                Column& col = columns[column % kCols];
                // two of them: other threads may still be decoding the tile before
                __half* steps = reinterpret_cast<__half*>(smem + S::kSteps) + (is_v * 2 + (column & 1)) * kTile;
                // 2^24 2^-E s, for E of any step
                const float up0 = power_of_two((24 - e_mine) / 2), up1 = power_of_two(24 - e_mine - (24 - e_mine) / 2);
                // a group held as NaN keeps the NaN in its common part alone
                const float own = bf16_lo(scale);
                const float rest = fmaf(8.f, own, bf16_hi(scale));
                if (is_v) {
                    col.v[p] = rest;
                } else {
                    __half hi, lo;
                    split2(rest * (up0 * (1.f / 65536.f)) * up1, kLowUp, hi, lo);  // 2^8 2^-E
                    const __half2 h2 = __half2half2(hi), l2 = __half2half2(lo);
                    unsigned char* more = smem + S::kKMore + stage * S::kMore;
                    *reinterpret_cast<uint4*>(more + sw32_offset(p, 0)) =
                        make_uint4(*reinterpret_cast<const uint32_t*>(&h2), *reinterpret_cast<const uint32_t*>(&l2), 0, 0);
                    *reinterpret_cast<uint4*>(more + sw32_offset(p, 1)) = make_uint4(0, 0, 0, 0);
                }
                steps[p] = __float2half_rn(own <= 3.0e38f ? own * up0 * up1 : 0.f);
                col.e[is_v][p] = static_cast<int16_t>(e_mine);
                if (p == 0) {
                    col.wide[is_v] = wide;
                    if (is_v) col.ev = e;
                    else col.up[0] = power_of_two(e / 2), col.up[1] = power_of_two(e - e / 2);
                }
                tc::mbar_arrive(&bars.col_full[column % kCols]);
                scale = seen(j + 1, scale_next);
                tell(scale, (column + 1) & 1);
                asm volatile("bar.sync %0, 128;" ::"r"(4 + is_v) : "memory");
                const bool more = j + 1 < k.t1;
                if (more) {
                    parts_next = check(j + 2);
                    scale_next = load_scale(parts_next);
                }
                if (!is_v) {
                    unsigned char* to = smem + S::kK + stage * S::kOne;
                    uint64_t next_at[kUnits];
#pragma unroll
                    for (int u = 0; u < kUnits; ++u) next_at[u] = place(parts, key_token(u));
                    __half2 step[kUnits];
#pragma unroll
                    for (int u = 0; u < kUnits; ++u) step[u] = __half2half2(steps[key_token(u)]);
#pragma unroll
                    for (int u = 0; u < kUnits; ++u) {
                        const int t = key_token(u);
                        const __half2 s = step[u], s16 = __hmul2(s, sixteenth), low = __hmul2(s, eighth);
#pragma unroll
                        for (int n = 0; n < 4; ++n) {
                            uint32_t h[4];
                            decode_word(raw[4 * u + n], h);
                            scale_word(h, s, s16, low);
                            const int c = seg * 4 + n;           // 8 dimensions
                            *reinterpret_cast<uint4*>(to + (c >> 3) * (kTile * 128) + tc::sw128_offset(t, (c & 7) * 8)) =
                                make_uint4(h[0], h[1], h[2], h[3]);
                        }
                        if (more) load_keys(u, next_at[u]);
                    }
                    tc::fence_proxy_async_smem();
                    tc::mbar_arrive(&bars.k_full[stage]);
                } else {
                    // transposed: a row of V' is a dimension
                    unsigned char* to = smem + S::kV + stage * S::kOne + vh * (kD * 128);
                    __half2 s[4], s16[4], low[4];
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        s[n] = __halves2half2(steps[vh * 64 + 8 * n + vt], steps[vh * 64 + 8 * n + 4 + vt]);
                        s16[n] = __hmul2(s[n], sixteenth), low[n] = __hmul2(s[n], eighth);
                    }
#pragma unroll
                    for (int x = 0; x < kVW; ++x)
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            uint32_t h[4][4], two[4];            // [token pair][dimension]
#pragma unroll
                            for (int n = 0; n < 4; ++n)
                                two[n] = __byte_perm(raw[2 * n * kVW + x], raw[(2 * n + 1) * kVW + x], half ? 0x7632 : 0x5410);
#pragma unroll
                            for (int n = 0; n < 4; ++n) {
                                decode_word(two[n], h[n]);
                                scale_word(h[n], s[n], s16[n], low[n]);
                            }
#pragma unroll
                            for (int d = 0; d < 4; ++d)
                                *reinterpret_cast<uint4*>(to + tc::sw128_offset(vd + x * 8 + half * 4 + d, vc * 8)) =
                                    make_uint4(h[0][d], h[1][d], h[2][d], h[3][d]);
                        }
                    tc::fence_proxy_async_smem();
                    tc::mbar_arrive(&bars.v_full[stage]);
                    if (more) load_values();
                }
                parts = parts_next;
                look_up(j + 3);
            }
            advance(4 + is_v);
        }
    }
    if (kSide == kJoined) pdl_wait();          // (who waits for this kernel waits for the one before)
    __syncthreads();
    if (warp == 0) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, 512);
    }
}

// Joins the pieces of a prefix's row tiles that several CTAs share: a CTA takes 8 rows at a time, a thread four dimensions
// of one of them, of all pieces. The rows of a request and head are numbered through, 8 to a number; a CTA has one number, or
// (kMany) each gridDim.x-th. `ctas` and `step` are the chunk kernel's. Each CTA goes through the requests once, a run of
// them a thread, which then knows which numbers are its. (A CTA for each number, whose first warp went through all requests
// for it, grew with the square of the groups: 3000 groups of 40 requests of 8 heads on 2 behind 512 tokens took 15.6 ms, and
// take 5.0.)
constexpr int kJoinRows = 8;
template <int kD>
constexpr int kJoinThreads = kJoinRows * kD / 4;
template <int kD>
constexpr int kJoinCtasPerSm = 1280 / kJoinThreads<kD>;

template <int kD, bool kMany>
__global__ void __launch_bounds__(kJoinThreads<kD>, kJoinCtasPerSm<kD>) join_kernel(const SharedArgs a, const float* scratch, int ctas, int step, int* status) {
    constexpr int kJoin = kJoinThreads<kD>, kJoinWarps = kJoin / 32;
    extern __shared__ float2 stats[];                          // [pieces][kJoinRows]
    struct Sums {
        int64_t numbers, slots;
    };
    __shared__ Sums sums[kJoinWarps], before[kJoin + 1];         // of a warp; before a thread's requests (here, since registers are short)
    // of a number: its first row and the end of its window's rows, the first token, head, CTAs with its row tile's first and last piece
    struct Number {
        int row0, row_end, begin, head, c0, c1;
    };
    __shared__ Number its;
    __shared__ float2 joined[kJoinRows];                       // maximum, 1 / sum
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, group = a.q_heads / a.c.kv_heads;
    const int per = (a.requests - 1) / kJoin + 1;
    const int b0 = static_cast<int>(min(static_cast<int64_t>(tid) * per, static_cast<int64_t>(a.requests))), b_n = min(per, a.requests - b0);
    auto of_head = [&](const Window& w) { return Sums{(w.rows * group + kJoinRows - 1) / kJoinRows, head_slots<kPrefix>(a, w, group, step)}; };
    Sums mine = {};
    for (int i = 0; i < b_n; ++i) {
        const Sums x = of_head(load_window<kPrefix>(a, b0 + i, nullptr));
        mine.numbers += x.numbers * a.c.kv_heads, mine.slots += x.slots * a.c.kv_heads;
    }
    Sums upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t y = __shfl_up_sync(~0u, upto.numbers, d), z = __shfl_up_sync(~0u, upto.slots, d);
        if (lane >= d) upto.numbers += y, upto.slots += z;
    }
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    Sums all = {};
    const int with = min((a.requests - 1) / 32 + 1, kJoinWarps);           // warps that have requests
    for (int i = 0; i < with; ++i) {
        if (i == warp) upto.numbers += all.numbers, upto.slots += all.slots;
        all.numbers += sums[i].numbers, all.slots += sums[i].slots;
    }
    before[tid] = Sums{upto.numbers - mine.numbers, upto.slots - mine.slots};
    if (tid == 0) before[kJoin] = all;
    __syncthreads();
    // the thread that has a number says what it is, behind a barrier
    auto look_up = [&](int64_t number) {
        if (number < before[tid].numbers || number >= before[tid + 1].numbers) return;
        int64_t at = number - before[tid].numbers, base = before[tid].slots;
        Sums x = {};
        Window w = {};
        for (int i = 0; i < b_n; ++i) {
            w = load_window<kPrefix>(a, b0 + i, nullptr);
            x = of_head(w);
            if (at < x.numbers * a.c.kv_heads) break;
            at -= x.numbers * a.c.kv_heads, base += x.slots * a.c.kv_heads;
        }
        if (x.numbers == 0) return;                            // (cannot be: what was summed is summed again)
        const int64_t h = quotient(at, x.numbers), total = before[kJoin].slots, n = min(static_cast<int64_t>(ctas), total);
        const int first = static_cast<int>(at - h * x.numbers) * kJoinRows, tiles = key_tiles<kPrefix>(a, w, group, step, 0);
        // the row tiles of a prefix have its key tiles each
        base += h * x.slots + static_cast<int64_t>(first / step) * (tiles + kPieceCost);
        its = {first, w.rows * group, w.begin, static_cast<int>(h), static_cast<int>(quotient((base + kPieceCost + 1) * n - 1, total)),
               static_cast<int>(quotient((base + kPieceCost + tiles) * n - 1, total))};
    };
    look_up(blockIdx.x);
    __syncthreads();
    // (the chunk kernel before began after all lengths were written; the kernel behind may begin once it has ended)
    begin_early();
    for (int64_t number = blockIdx.x; number < before[kJoin].numbers; number += gridDim.x) {
        const int row0 = its.row0, row_end = its.row_end, begin = its.begin, head = its.head, c0 = its.c0, c1 = its.c1;
        if (c0 < c1 && HC_IN_RANGE(c0, c1 - c0 + 1, ctas, status)) {        // (else one piece: its CTA wrote it)
            auto piece = [&](int c) { return scratch + (static_cast<int64_t>(c) * 2 + (c == c0 ? 1 : 0)) * kPieceFloats; };
            const int in_tile = row0 % step, rows = min(row_end - row0, kJoinRows);
            const int r = tid % kJoinRows, quad = tid / kJoinRows;
            for (int i = quad; i <= c1 - c0; i += kD / 4)
                stats[i * kJoinRows + r] = r < rows ? __ldcg(reinterpret_cast<const float2*>(piece(c0 + i) + 256 * kD) + in_tile + r) : make_float2(-CUDART_INF_F, 0.f);
            __syncthreads();
            const int of = row0 + r;
            const int64_t at = static_cast<int64_t>(begin + of / group) * a.q_heads + head * group + of % group;
            const bool here = r < rows && HC_IN_RANGE(at, 1, static_cast<size_t>(a.tokens) * a.q_heads, status);
            if (tid < kJoinRows) {
                float top = -CUDART_INF_F, all_of = 0.f;
                for (int i = 0; i <= c1 - c0; ++i) top = fmaxf(top, stats[i * kJoinRows + r].x);
                for (int i = 0; i <= c1 - c0; ++i) {
                    const float2 st = stats[i * kJoinRows + r];
                    if (st.x != -CUDART_INF_F) all_of += st.y * exp2_fast(st.x - top);
                }
                joined[r] = make_float2(top, all_of == 0.f ? 0.f : 1.f / all_of);
                if (here) partial_stats(a, kD)[at] = make_float2(top, all_of);
            }
            __syncthreads();
            if (here) {
                const float2 join = joined[r];
                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
                for (int i = 0; i <= c1 - c0; ++i) {
                    const float4 y = __ldcg(reinterpret_cast<const float4*>(piece(c0 + i)) + quad * 256 + in_tile + r);
                    const float peak = stats[i * kJoinRows + r].x;
                    if (peak == -CUDART_INF_F) continue;
                    const float by = exp2_fast(peak - join.x);
                    o.x = fmaf(y.x, by, o.x), o.y = fmaf(y.y, by, o.y), o.z = fmaf(y.z, by, o.z), o.w = fmaf(y.w, by, o.w);
                }
                *reinterpret_cast<float4*>(a.partial + at * kD + quad * 4) = make_float4(o.x * join.y, o.y * join.y, o.z * join.y, o.w * join.y);
            }
        }
        if (!kMany || number + gridDim.x >= before[kJoin].numbers) break;
        __syncthreads();                                       // what is shared is free
        look_up(number + gridDim.x);
        __syncthreads();
    }
}

template <int kD>
cudaError_t launch_join(const Ctx& ctx, const SharedArgs& a, int step, cudaStream_t st) {
    // One CTA for each number that there can be, or, if these are not resident at once, as many as are, in a loop. (In a
    // loop 64 requests behind 16384 tokens took 51.2 us where this takes 48.3: fewer loads on their way.)
    const int64_t rows = static_cast<int64_t>(a.tokens) * (a.q_heads / a.c.kv_heads);
    const int64_t most = (rows / kJoinRows + a.requests) * a.c.kv_heads, resident = static_cast<int64_t>(ctx.sm_count) * kJoinCtasPerSm<kD>;
    const bool many = most > resident;
    return launch_early(many ? join_kernel<kD, true> : join_kernel<kD, false>, dim3(static_cast<unsigned>(many ? resident : most)), kJoinThreads<kD>,
                        sizeof(float2) * kJoinRows * ctx.sm_count, st, a, ctx.attn_pieces, ctx.sm_count, step, ctx.s.status);
}

template <int kD, int kDtype, bool kSame, Side kSide>
cudaError_t launch_chunk(const Ctx& ctx, const Args<kSide>& a, cudaStream_t st) {
    return launch_early(chunk_kernel<kD, kDtype, kSame, kSide>, dim3(ctx.sm_count), kThreads, Smem<kD>::kBytes, st, a, ctx.attn_pieces,
                        ctx.attn_arrivals, ctx.s.status);
}

template <int kD, int kDtype, Side kSide>
cudaError_t launch_rows(const Ctx& ctx, const Args<kSide>& a, cudaStream_t st) {
    const bool same = static_cast<int64_t>(a.max_new) * (a.q_heads / a.c.kv_heads) <= kTile;
    const cudaError_t e = same ? launch_chunk<kD, kDtype, true, kSide>(ctx, a, st) : launch_chunk<kD, kDtype, false, kSide>(ctx, a, st);
    if constexpr (kSide == kPrefix) return e != cudaSuccess ? e : launch_join<kD>(ctx, a, same ? kTile : 2 * kTile, st);
    return e;
}

// A kernel's shared memory; and that it was compiled with the registers which its warps share out
// among themselves (a warp would wait for ever for what the launch does not have).
template <int kD, int kDtype, bool kSame, Side kSide>
cudaError_t allow_one() {
    cudaFuncAttributes has;
    const cudaError_t e = cudaFuncGetAttributes(&has, chunk_kernel<kD, kDtype, kSame, kSide>);
    if (e != cudaSuccess) return e;
    if ((has.numRegs + 7) / 8 * 8 * kThreads < 65536) return cudaErrorInvalidConfiguration;
    return cudaFuncSetAttribute(chunk_kernel<kD, kDtype, kSame, kSide>, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<kD>::kBytes);
}

template <int kD, int kDtype, Side kSide>
cudaError_t allow_smem() {
    const cudaError_t e = allow_one<kD, kDtype, true, kSide>();
    return e != cudaSuccess ? e : allow_one<kD, kDtype, false, kSide>();
}

}  // namespace

template <Side kSide>
cudaError_t attention_chunk_setup() {
    cudaError_t e = allow_smem<64, HC_DTYPE_BF16, kSide>();
    if (e == cudaSuccess) e = allow_smem<64, HC_DTYPE_FP16, kSide>();
    if (e == cudaSuccess) e = allow_smem<128, HC_DTYPE_BF16, kSide>();
    if (e == cudaSuccess) e = allow_smem<128, HC_DTYPE_FP16, kSide>();
    return e;
}

template <Side kSide>
cudaError_t launch_attention_chunk(const Ctx& ctx, const Args<kSide>& a, int dtype, cudaStream_t st) {
    if (a.c.head_dim == 64)
        return dtype == HC_DTYPE_BF16 ? launch_rows<64, HC_DTYPE_BF16, kSide>(ctx, a, st) : launch_rows<64, HC_DTYPE_FP16, kSide>(ctx, a, st);
    return dtype == HC_DTYPE_BF16 ? launch_rows<128, HC_DTYPE_BF16, kSide>(ctx, a, st) : launch_rows<128, HC_DTYPE_FP16, kSide>(ctx, a, st);
}

}  // namespace hc
