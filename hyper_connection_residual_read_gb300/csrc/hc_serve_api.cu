// C ABI of the operators of include/hc_serve.h: argument checks and launches.
#include <cuda_runtime.h>
#include <limits.h>
#include <stdint.h>

#include "hc_checks.h"
#include "hc_serve_internal.h"

using namespace hc;

extern "C" int hc_kv4_append_rotary(const hc_kv4_cache* cache, const hc_rotary* rotary, int tokens, int q_heads,
                                    int dtype, const void* q, int64_t q_token_stride, int64_t q_head_stride,
                                    const void* k, int64_t k_token_stride, int64_t k_head_stride,
                                    const void* v, int64_t v_token_stride, int64_t v_head_stride,
                                    const int32_t* positions, const int64_t* slots, void* q_out,
                                    void* stream) {
    int err;
    Ctx* c = current_ctx(&err);
    if (!c) return err;
    if (int e = check_cache(cache, c->device)) return e;
    if (rotary == nullptr || tokens < 0 || q_heads < 0 || q_heads > kMaxHeads || dtype < HC_DTYPE_BF16 || dtype > HC_DTYPE_FP32)
        return HC_ERR_ARG;
    const hc_rotary& r = *rotary;
    const int h = cache->kv_heads, d = cache->head_dim;
    if (r.dim < 0 || r.dim > d || r.dim % 16 != 0 || !(r.eps >= 0.f) || r.eps - r.eps != 0.f) return HC_ERR_ARG;
    if (r.dim > 0 && (r.length < 1 || r.axes < 1 || r.axes > HC_ROTARY_MAX_AXES)) return HC_ERR_ARG;
    if (tokens == 0) return HC_OK;
    if ((q_heads > 0 && !good_strides(tokens, q_heads, q_token_stride, q_head_stride, dtype)) ||
        !good_strides(tokens, h, k_token_stride, k_head_stride, dtype) ||
        !good_strides(tokens, h, v_token_stride, v_head_stride, dtype))
        return HC_ERR_ARG;
    const void* large[] = {k, v};
    for (const void* p : large)
        if (int e = check_ptr(p, c->device)) return e;
    if (q_heads > 0) {
        if (int e = check_ptr(q, c->device)) return e;
        if (int e = check_ptr(q_out, c->device)) return e;
    }
    if (r.dim > 0) {
        if (int e = check_ptr(r.cos_sin, c->device)) return e;
        if (int e = check_array(positions, c->device, 4)) return e;
        if (r.axis_of != nullptr)
            if (int e = check_array(r.axis_of, c->device, 4)) return e;
    }
    const void* norms[] = {r.q_norm, r.k_norm};
    for (const void* p : norms)
        if (p != nullptr)
            if (int e = check_ptr(p, c->device)) return e;
    if (int e = check_array(slots, c->device, 8)) return e;
    const uint64_t n = cache_tokens(*cache), t = tokens, bytes = item(dtype);
    const bool turned = r.dim > 0;
    const Span s[] = {{cache->codes, n * (d / 2)}, {cache->scales, 4 * n},
                      {q_out, q_heads > 0 ? t * q_heads * d * bytes : 0},
                      {q, q_heads > 0 ? extent(tokens, q_heads, d, q_token_stride, q_head_stride, dtype) : 0},
                      {k, extent(tokens, h, d, k_token_stride, k_head_stride, dtype)},
                      {v, extent(tokens, h, d, v_token_stride, v_head_stride, dtype)},
                      {slots, 8 * t}, {positions, turned ? 4 * t * r.axes : 0},
                      {r.cos_sin, turned ? 4ull * r.length * r.dim : 0},
                      {r.axis_of, turned && r.axis_of ? 2ull * r.dim : 0},
                      {r.q_norm, r.q_norm ? d * bytes : 0}, {r.k_norm, r.k_norm ? d * bytes : 0}};
    if (any_meet(s, 3, 12)) return HC_ERR_ARG;
    const RotaryArgs a{*cache, r, tokens, q_heads, q, k, v, q_token_stride, q_head_stride, k_token_stride,
                       k_head_stride, v_token_stride, v_head_stride, positions, slots, q_out};
    return launch_kv4_append_rotary(*c, a, dtype, static_cast<cudaStream_t>(stream)) == cudaSuccess ? HC_OK : HC_ERR_CUDA;
}

extern "C" int hc_kv4_attention_shared(const hc_kv4_cache* cache, int requests, int groups, int tokens, int q_heads,
                                       int max_new, int max_shared, int table_width, int prefix_width, float scale,
                                       int dtype, const void* q, int64_t q_token_stride, int64_t q_head_stride,
                                       const int32_t* cu_lens, const int32_t* kv_lens, const int32_t* block_table,
                                       const int32_t* cu_groups, const int32_t* prefix_lens,
                                       const int32_t* prefix_table, const uint64_t* mask, float* workspace,
                                       void* out, float* lse, void* stream) {
    int err;
    Ctx* c = current_ctx(&err);
    if (!c) return err;
    if (int e = check_cache(cache, c->device)) return e;
    if (requests < 0 || groups < 0 || tokens < 0 || q_heads < 1 || max_new < 0 || max_shared < 0 || table_width < 1 ||
        prefix_width < 1 || dtype < HC_DTYPE_BF16 || dtype > HC_DTYPE_FP16 || !(scale == scale) || scale - scale != 0.f)
        return HC_ERR_ARG;
    if (q_heads % cache->kv_heads != 0 || q_heads / cache->kv_heads > HC_KV4_MAX_GROUP) return HC_ERR_ARG;
    if (mask != nullptr && max_new > HC_KV4_MAX_MASKED) return HC_ERR_ARG;
    if (requests == 0 || tokens == 0 || max_new == 0) return HC_OK;
    if (groups == 0 || max_shared == 0) return HC_ERR_ARG;               // the tokens are in some group
    if (!good_strides(tokens, q_heads, q_token_stride, q_head_stride, dtype)) return HC_ERR_ARG;
    const void* large[] = {q, out, workspace};
    for (const void* p : large)
        if (int e = check_ptr(p, c->device)) return e;
    const void* ints[] = {cu_lens, kv_lens, block_table, cu_groups, prefix_lens, prefix_table};
    for (const void* p : ints)
        if (int e = check_array(p, c->device, 4)) return e;
    if (lse != nullptr)
        if (int e = check_array(lse, c->device, 4)) return e;
    if (mask != nullptr)
        if (int e = check_array(mask, c->device, 8)) return e;
    const int d = cache->head_dim;
    const uint64_t n = cache_tokens(*cache), rows = (uint64_t)tokens * q_heads;
    const Span s[] = {{out, rows * d * item(dtype)}, {lse, lse ? 4 * rows : 0}, {workspace, 4 * rows * (d + 2)},
                      {cache->codes, n * (d / 2)}, {cache->scales, 4 * n},
                      {q, extent(tokens, q_heads, d, q_token_stride, q_head_stride, dtype)},
                      {cu_lens, 4ull * requests + 4}, {kv_lens, 4ull * requests},
                      {block_table, 4ull * requests * table_width}, {cu_groups, 4ull * groups + 4},
                      {prefix_lens, 4ull * groups}, {prefix_table, 4ull * groups * prefix_width},
                      {mask, mask ? 8ull * tokens : 0}};
    if (any_meet(s, 3, 13)) return HC_ERR_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const SharedArgs prefix{{*cache, groups, tokens, q_heads, max_shared, prefix_width, scale, q, q_token_stride,
                             q_head_stride, cu_lens, prefix_lens, prefix_table, nullptr, nullptr, nullptr},
                            cu_groups, requests, 1, max_shared, workspace};
    if (launch_kv4_attention_prefix(*c, prefix, dtype, st) != cudaSuccess) return HC_ERR_CUDA;
    const SharedArgs own{{*cache, requests, tokens, q_heads, max_new, table_width, scale, q, q_token_stride,
                          q_head_stride, cu_lens, kv_lens, block_table, mask, out, lse},
                         nullptr, 0, 1, 0, workspace};
    return launch_kv4_attention_joined(*c, own, dtype, st) == cudaSuccess ? HC_OK : HC_ERR_CUDA;
}

extern "C" int hc_sample_tokens(int tokens, int vocab, int dtype, const void* logits, int64_t row_stride,
                                const float* uniform, const float* temperature, const int32_t* top_k,
                                const float* top_p, const float* min_p, int32_t* token_ids, float* logprob,
                                void* stream) {
    int err;
    Ctx* c = current_ctx(&err);
    if (!c) return err;
    if (tokens < 0 || vocab < 1 || vocab > HC_SAMPLE_MAX_VOCAB || dtype < HC_DTYPE_BF16 || dtype > HC_DTYPE_FP32 ||
        row_stride < 0)
        return HC_ERR_ARG;
    if (tokens == 0) return HC_OK;
    if (int e = check_array(logits, c->device, item(dtype))) return e;
    const void* words[] = {uniform, token_ids, logprob};
    for (const void* p : words)
        if (int e = check_array(p, c->device, 4)) return e;
    const void* settings[] = {temperature, top_k, top_p, min_p};
    for (const void* p : settings)
        if (p != nullptr)
            if (int e = check_array(p, c->device, 4)) return e;
    const uint64_t t = tokens;
    const Span s[] = {{token_ids, 4 * t}, {logprob, 4 * t},
                      {logits, ((t - 1) * (uint64_t)row_stride + vocab) * item(dtype)}, {uniform, 4 * t},
                      {temperature, temperature ? 4 * t : 0}, {top_k, top_k ? 4 * t : 0},
                      {top_p, top_p ? 4 * t : 0}, {min_p, min_p ? 4 * t : 0}};
    if (any_meet(s, 2, 8)) return HC_ERR_ARG;
    const SampleArgs a{tokens, vocab, logits, row_stride, uniform, temperature, top_k, top_p, min_p, token_ids, logprob};
    return launch_sample_tokens(*c, a, dtype, static_cast<cudaStream_t>(stream)) == cudaSuccess ? HC_OK : HC_ERR_CUDA;
}
