// Argument checks that the entry points of the operators beside the read share.
#pragma once

#include <limits.h>
#include <stdint.h>

#include "hc_window_internal.h"

namespace hc {

inline bool known_block(int n) { return n >= 16 && n <= HC_KV4_MAX_BLOCK && (n & (n - 1)) == 0; }

// Device memory aligned to `align` bytes (an array of small elements).
inline int check_array(const void* p, int device, unsigned align) {
    if (p == nullptr || (reinterpret_cast<uintptr_t>(p) & (align - 1)) != 0) return HC_ERR_ARG;
    // check_ptr asks for 16-byte alignment: hand it the 16 bytes that hold the start
    return check_ptr(reinterpret_cast<const void*>(reinterpret_cast<uintptr_t>(p) & ~(uintptr_t)15),
                     device);
}

struct Span {
    uintptr_t lo, hi;
    Span(const void* p, uint64_t bytes)
        : lo(reinterpret_cast<uintptr_t>(p)), hi(reinterpret_cast<uintptr_t>(p) + bytes) {}
    bool meets(const Span& o) const { return lo < hi && o.lo < o.hi && lo < o.hi && o.lo < hi; }
};

// True if one of the first `outs` spans meets another of them or one of the rest.
inline bool any_meet(const Span* s, int outs, int n) {
    for (int i = 0; i < outs; ++i)
        for (int j = i + 1; j < n; ++j)
            if (s[i].meets(s[j])) return true;
    return false;
}

// A grid's second axis is at most 65535, and a block's bytes fit 32 bits with as many heads.
constexpr int kMaxHeads = 65535;

inline int check_cache(const hc_kv4_cache* c, int device) {
    if (c == nullptr || c->blocks < 1 || c->kv_heads < 1 || c->kv_heads > kMaxHeads || !known_block(c->block_size))
        return HC_ERR_ARG;
    if (c->head_dim != 64 && c->head_dim != 128) return HC_ERR_ARG;
    if (int e = check_ptr(c->codes, device)) return e;
    return check_ptr(c->scales, device);
}

inline uint64_t cache_tokens(const hc_kv4_cache& c) {
    return 2ull * c.blocks * c.kv_heads * c.block_size;
}

inline unsigned item(int dtype) { return dtype == HC_DTYPE_FP32 ? 4 : 2; }

// Strides of rows read 16 bytes at a time: whole 16-byte pieces, and not negative. That of an
// axis of one is never used.
inline bool good_strides(int tokens, int heads, int64_t token, int64_t head, int dtype) {
    const int64_t n = 16 / item(dtype);
    return (tokens == 1 || (token >= 0 && token % n == 0)) && (heads == 1 || (head >= 0 && head % n == 0));
}

// Bytes from the first to behind the last element of a strided [tokens][heads][dim].
inline uint64_t extent(int tokens, int heads, int dim, int64_t token, int64_t head, int dtype) {
    return ((uint64_t)(tokens - 1) * token + (uint64_t)(heads - 1) * head + dim) * item(dtype);
}

}  // namespace hc
