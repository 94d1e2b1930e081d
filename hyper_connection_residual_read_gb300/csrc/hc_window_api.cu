// C ABI of the verify-window operators: argument checks and launches.
#include <cuda_runtime.h>
#include <limits.h>
#include <stdint.h>

#include "hc_checks.h"
#include "hc_window_internal.h"

using namespace hc;

extern "C" int hc_window_plan(int requests, int table_width, int block_size, int capacity,
                              int free_capacity, const int32_t* cached_lens,
                              const int32_t* new_lens, const int32_t* free_blocks,
                              const int32_t* free_count, int32_t* block_table, int64_t* slots,
                              int32_t* request_of, int32_t* positions, int32_t* cu_lens,
                              int32_t* kv_lens, int32_t* free_left, void* stream) {
    int err;
    Ctx* c = current_ctx(&err);
    if (!c) return err;
    if (requests < 1 || requests > HC_PLAN_MAX_REQUESTS || table_width < 1 || capacity < 0 ||
        free_capacity < 0 || !known_block(block_size) || (int64_t)requests * table_width > INT_MAX)
        return HC_ERR_ARG;
    const void* ints[] = {cached_lens, new_lens, free_count, block_table, cu_lens, kv_lens, free_left};
    for (const void* p : ints)
        if (int e = check_array(p, c->device, 4)) return e;
    if (free_capacity > 0)
        if (int e = check_array(free_blocks, c->device, 4)) return e;
    if (capacity > 0) {
        if (int e = check_array(slots, c->device, 8)) return e;
        if (int e = check_array(request_of, c->device, 4)) return e;
        if (int e = check_array(positions, c->device, 4)) return e;
    }
    const uint64_t n = requests, t = capacity;
    const Span s[] = {{block_table, 4 * n * table_width}, {slots, 8 * t}, {request_of, 4 * t},
                      {positions, 4 * t}, {cu_lens, 4 * (n + 1)}, {kv_lens, 4 * n}, {free_left, 4},
                      {cached_lens, 4 * n}, {new_lens, 4 * n}, {free_blocks, 4ull * free_capacity},
                      {free_count, 4}};
    if (any_meet(s, 7, 11)) return HC_ERR_ARG;
    const PlanArgs a{requests, table_width, block_size, capacity, free_capacity, cached_lens, new_lens,
                     free_blocks, free_count, block_table, slots, request_of, positions, cu_lens,
                     kv_lens, free_left};
    return launch_plan(*c, a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? HC_OK : HC_ERR_CUDA;
}

extern "C" int hc_kv4_append(const hc_kv4_cache* cache, int tokens, int dtype, const void* k,
                             int64_t k_token_stride, int64_t k_head_stride, const void* v,
                             int64_t v_token_stride, int64_t v_head_stride, const int64_t* slots,
                             void* stream) {
    int err;
    Ctx* c = current_ctx(&err);
    if (!c) return err;
    if (int e = check_cache(cache, c->device)) return e;
    if (tokens < 0 || dtype < HC_DTYPE_BF16 || dtype > HC_DTYPE_FP32) return HC_ERR_ARG;
    if (tokens == 0) return HC_OK;
    if (!good_strides(tokens, cache->kv_heads, k_token_stride, k_head_stride, dtype) ||
        !good_strides(tokens, cache->kv_heads, v_token_stride, v_head_stride, dtype))
        return HC_ERR_ARG;
    if (int e = check_ptr(k, c->device)) return e;
    if (int e = check_ptr(v, c->device)) return e;
    if (int e = check_array(slots, c->device, 8)) return e;
    const int h = cache->kv_heads, d = cache->head_dim;
    const uint64_t n = cache_tokens(*cache);
    const Span s[] = {{cache->codes, n * (d / 2)}, {cache->scales, 4 * n},
                      {k, extent(tokens, h, d, k_token_stride, k_head_stride, dtype)},
                      {v, extent(tokens, h, d, v_token_stride, v_head_stride, dtype)},
                      {slots, 8ull * tokens}};
    if (any_meet(s, 2, 5)) return HC_ERR_ARG;
    const CacheArgs a{*cache, tokens, slots, k, v, k_token_stride, k_head_stride, v_token_stride,
                      v_head_stride, nullptr, nullptr};
    return launch_kv4_append(*c, a, dtype, static_cast<cudaStream_t>(stream)) == cudaSuccess ? HC_OK : HC_ERR_CUDA;
}

extern "C" int hc_kv4_load(const hc_kv4_cache* cache, int tokens, const int64_t* slots, int dtype,
                           void* k_out, void* v_out, void* stream) {
    int err;
    Ctx* c = current_ctx(&err);
    if (!c) return err;
    if (int e = check_cache(cache, c->device)) return e;
    if (tokens < 0 || dtype < HC_DTYPE_BF16 || dtype > HC_DTYPE_FP32) return HC_ERR_ARG;
    if (tokens == 0) return HC_OK;
    if (int e = check_ptr(k_out, c->device)) return e;
    if (int e = check_ptr(v_out, c->device)) return e;
    if (int e = check_array(slots, c->device, 8)) return e;
    const uint64_t n = cache_tokens(*cache);
    const uint64_t out = (uint64_t)tokens * cache->kv_heads * cache->head_dim * item(dtype);
    const Span s[] = {{k_out, out}, {v_out, out}, {cache->codes, n * (cache->head_dim / 2)},
                      {cache->scales, 4 * n}, {slots, 8ull * tokens}};
    if (any_meet(s, 2, 5)) return HC_ERR_ARG;
    const CacheArgs a{*cache, tokens, slots, nullptr, nullptr, 0, 0, 0, 0, k_out, v_out};
    return launch_kv4_load(*c, a, dtype, static_cast<cudaStream_t>(stream)) == cudaSuccess ? HC_OK : HC_ERR_CUDA;
}

extern "C" int hc_kv4_attention(const hc_kv4_cache* cache, int requests, int tokens, int q_heads,
                                int max_new, int table_width, float scale, int dtype, const void* q,
                                int64_t q_token_stride, int64_t q_head_stride,
                                const int32_t* cu_lens, const int32_t* kv_lens,
                                const int32_t* block_table, const uint64_t* mask, void* out,
                                float* lse, void* stream) {
    int err;
    Ctx* c = current_ctx(&err);
    if (!c) return err;
    if (int e = check_cache(cache, c->device)) return e;
    if (requests < 0 || tokens < 0 || q_heads < 1 || max_new < 0 || table_width < 1 ||
        dtype < HC_DTYPE_BF16 || dtype > HC_DTYPE_FP16 || !(scale == scale) ||
        scale - scale != 0.f)
        return HC_ERR_ARG;
    if (q_heads % cache->kv_heads != 0 || q_heads / cache->kv_heads > HC_KV4_MAX_GROUP) return HC_ERR_ARG;
    if (mask != nullptr && max_new > HC_KV4_MAX_MASKED) return HC_ERR_ARG;
    if (requests == 0 || tokens == 0 || max_new == 0) return HC_OK;
    if (!good_strides(tokens, q_heads, q_token_stride, q_head_stride, dtype)) return HC_ERR_ARG;
    if (int e = check_ptr(q, c->device)) return e;
    if (int e = check_ptr(out, c->device)) return e;
    const void* ints[] = {cu_lens, kv_lens, block_table};
    for (const void* p : ints)
        if (int e = check_array(p, c->device, 4)) return e;
    if (lse != nullptr)
        if (int e = check_array(lse, c->device, 4)) return e;
    if (mask != nullptr)
        if (int e = check_array(mask, c->device, 8)) return e;
    const int d = cache->head_dim;
    const uint64_t n = cache_tokens(*cache), rows = (uint64_t)tokens * q_heads;
    const Span s[] = {{out, rows * d * item(dtype)}, {lse, lse ? 4 * rows : 0},
                      {cache->codes, n * (d / 2)}, {cache->scales, 4 * n},
                      {q, extent(tokens, q_heads, d, q_token_stride, q_head_stride, dtype)},
                      {cu_lens, 4ull * requests + 4}, {kv_lens, 4ull * requests},
                      {block_table, 4ull * requests * table_width},
                      {mask, mask ? 8ull * tokens : 0}};
    if (any_meet(s, 2, 9)) return HC_ERR_ARG;
    const AttentionArgs a{*cache, requests, tokens, q_heads, max_new, table_width, scale, q,
                          q_token_stride, q_head_stride, cu_lens, kv_lens, block_table, mask, out, lse};
    return launch_kv4_attention(*c, a, dtype, static_cast<cudaStream_t>(stream)) == cudaSuccess ? HC_OK : HC_ERR_CUDA;
}

extern "C" int hc_token_logprobs(int tokens, int vocab, int top, int dtype, const void* logits,
                                 int64_t row_stride, const int32_t* token_ids, float* logprob,
                                 float* entropy, float* lse, int32_t* rank, int32_t* top_ids,
                                 float* top_logprobs, void* stream) {
    int err;
    Ctx* c = current_ctx(&err);
    if (!c) return err;
    if (tokens < 0 || vocab < 1 || top < 0 || top > vocab || top > HC_LOGPROBS_MAX_TOP ||
        dtype < HC_DTYPE_BF16 || dtype > HC_DTYPE_FP32 || row_stride < 0)
        return HC_ERR_ARG;
    if (tokens == 0) return HC_OK;
    if (int e = check_array(logits, c->device, item(dtype))) return e;
    const void* words[] = {token_ids, logprob, entropy, lse, rank};
    for (const void* p : words)
        if (int e = check_array(p, c->device, 4)) return e;
    if (top > 0) {
        if (int e = check_array(top_ids, c->device, 4)) return e;
        if (int e = check_array(top_logprobs, c->device, 4)) return e;
    }
    const uint64_t t = tokens;
    const Span s[] = {{logprob, 4 * t}, {entropy, 4 * t}, {lse, 4 * t}, {rank, 4 * t},
                      {top_ids, 4 * t * top}, {top_logprobs, 4 * t * top},
                      {logits, ((t - 1) * (uint64_t)row_stride + vocab) * item(dtype)},
                      {token_ids, 4 * t}};
    if (any_meet(s, 6, 8)) return HC_ERR_ARG;
    const LogprobArgs a{tokens, vocab, top, logits, row_stride, token_ids, logprob, entropy, lse, rank,
                        top_ids, top_logprobs};
    return launch_logprobs(*c, a, dtype, static_cast<cudaStream_t>(stream)) == cudaSuccess ? HC_OK : HC_ERR_CUDA;
}
