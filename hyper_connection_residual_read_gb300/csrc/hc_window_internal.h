// Internal declarations of the verify-window operators (include/hc_window.h).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "hc_internal.h"
#include "hc_window.h"

namespace hc {

struct PlanArgs {
    int requests, width, block_size, capacity, free_capacity;
    const int32_t* cached;
    const int32_t* added;
    const int32_t* free_blocks;
    const int32_t* free_count;
    int32_t* table;
    int64_t* slots;
    int32_t* request_of;
    int32_t* positions;
    int32_t* cu;
    int32_t* kv;
    int32_t* free_left;
};
cudaError_t launch_plan(const Ctx& ctx, const PlanArgs& a, cudaStream_t st);

// k and v are read by append and written by load (contiguous there).
struct CacheArgs {
    hc_kv4_cache c;
    int tokens;
    const int64_t* slots;
    const void* k;
    const void* v;
    int64_t k_token, k_head, v_token, v_head;   // strides in elements
    void* k_out;
    void* v_out;
};
cudaError_t launch_kv4_append(const Ctx& ctx, const CacheArgs& a, int dtype, cudaStream_t st);
cudaError_t launch_kv4_load(const Ctx& ctx, const CacheArgs& a, int dtype, cudaStream_t st);

struct AttentionArgs {
    hc_kv4_cache c;
    int requests, tokens, q_heads, max_new, width;
    float scale;
    const void* q;
    int64_t q_token, q_head;                    // strides in elements
    const int32_t* cu;
    const int32_t* kv;
    const int32_t* table;
    const uint64_t* mask;
    void* out;
    float* lse;
};
// Behind a shared prefix (hc_serve.h): the prefixes' part, whose `requests` are the groups (or `subs` shares of
// max_new tokens of each), goes to `partial`, from where the own part takes it. (A struct of its own: with these
// members the arguments of hc_kv4_attention's kernels lie elsewhere, and 8192 tokens behind 8192 took 2.4% longer.)
struct SharedArgs : AttentionArgs {
    const int32_t* groups;                      // first request of each group
    int members;                                // requests of all groups
    int subs, shared;                           // shares of a group, and tokens that it may have
    float* partial;                             // [tokens][q_heads][head_dim], then (maximum, sum) of each row
};
cudaError_t launch_kv4_attention(const Ctx& ctx, const AttentionArgs& a, int dtype, cudaStream_t st);
cudaError_t launch_kv4_attention_prefix(const Ctx& ctx, const SharedArgs& a, int dtype, cudaStream_t st);
cudaError_t launch_kv4_attention_joined(const Ctx& ctx, const SharedArgs& a, int dtype, cudaStream_t st);

struct LogprobArgs {
    int tokens, vocab, top;
    const void* logits;
    int64_t row;                                // stride in elements
    const int32_t* ids;
    float* logprob;
    float* entropy;
    float* lse;
    int32_t* rank;
    int32_t* top_ids;
    float* top_logprobs;
};
cudaError_t launch_logprobs(const Ctx& ctx, const LogprobArgs& a, int dtype, cudaStream_t st);

}  // namespace hc
