// Internal declarations of the operators of include/hc_serve.h.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "hc_internal.h"
#include "hc_serve.h"
#include "hc_window_internal.h"

namespace hc {

struct RotaryArgs {
    hc_kv4_cache c;
    hc_rotary r;
    int tokens, q_heads;
    const void* q;
    const void* k;
    const void* v;
    int64_t q_token, q_head, k_token, k_head, v_token, v_head;   // strides in elements
    const int32_t* positions;
    const int64_t* slots;
    void* q_out;
};
cudaError_t launch_kv4_append_rotary(const Ctx& ctx, const RotaryArgs& a, int dtype, cudaStream_t st);

struct SampleArgs {
    int tokens, vocab;
    const void* logits;
    int64_t row;                                // stride in elements
    const float* uniform;
    const float* temperature;                   // these four may be null
    const int32_t* top_k;
    const float* top_p;
    const float* min_p;
    int32_t* ids;
    float* logprob;
};
cudaError_t launch_sample_tokens(const Ctx& ctx, const SampleArgs& a, int dtype, cudaStream_t st);

}  // namespace hc
