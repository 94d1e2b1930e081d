// Attention over the 4-bit cache, windows of few rows behind a prefix whose requests are short: a CTA of few warps for
// each request and head.
#define HC_WINDOW_WARPS 4
#include "hc_attention.cuh"

namespace hc {

cudaError_t attention_short_setup() {
    cudaError_t e = allow_rows<64, HC_DTYPE_BF16, kJoined>();
    if (e == cudaSuccess) e = allow_rows<64, HC_DTYPE_FP16, kJoined>();
    if (e == cudaSuccess) e = allow_rows<128, HC_DTYPE_BF16, kJoined>();
    if (e == cudaSuccess) e = allow_rows<128, HC_DTYPE_FP16, kJoined>();
    return e;
}

cudaError_t launch_attention_short(const Ctx& ctx, const SharedArgs& a, int dtype, cudaStream_t st) {
    if (a.c.head_dim == 64)
        return dtype == HC_DTYPE_BF16 ? launch_rows<64, HC_DTYPE_BF16, kJoined>(ctx, a, st) : launch_rows<64, HC_DTYPE_FP16, kJoined>(ctx, a, st);
    return dtype == HC_DTYPE_BF16 ? launch_rows<128, HC_DTYPE_BF16, kJoined>(ctx, a, st) : launch_rows<128, HC_DTYPE_FP16, kJoined>(ctx, a, st);
}

}  // namespace hc
