// Groups of the 4-bit cache: eight values of an input or output type a lane, their rounding to
// codes, step and minimum, and where a slot's group lies.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "hc_window.cuh"

namespace hc {

template <int kDtype>
struct Raw8;     // 8 values of an input or output type
template <>
struct Raw8<HC_DTYPE_BF16> {
    uint4 v;
    __device__ void load(const void* p, int64_t i) {
        v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
    }
    __device__ void get(float (&x)[8]) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) x[2 * i] = bf16_lo(w[i]), x[2 * i + 1] = bf16_hi(w[i]);
    }
    __device__ void set(const float (&x)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        v = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ void store(void* p, int64_t i) const {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = v;
    }
};
template <>
struct Raw8<HC_DTYPE_FP16> {
    uint4 v;
    __device__ void load(const void* p, int64_t i) {
        v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
    }
    __device__ void get(float (&x)[8]) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            x[2 * i] = f.x, x[2 * i + 1] = f.y;
        }
    }
    __device__ void set(const float (&x)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        v = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ void store(void* p, int64_t i) const {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = v;
    }
};
template <>
struct Raw8<HC_DTYPE_FP32> {
    float4 a, b;
    __device__ void load(const void* p, int64_t i) {
        const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
        a = q[0], b = q[1];
    }
    __device__ void get(float (&x)[8]) const {
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
        x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
    __device__ void set(const float (&x)[8]) {
        a = make_float4(x[0], x[1], x[2], x[3]);
        b = make_float4(x[4], x[5], x[6], x[7]);
    }
    __device__ void store(void* p, int64_t i) const {
        float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
        q[0] = a, q[1] = b;
    }
};

// The largest bf16 <= x and the smallest bf16 >= x, of a finite x: cut to 16 bits, which
// rounds toward zero, and step one away from zero where that went the wrong way.
__device__ __forceinline__ float bf16_floor(float x) {
    const uint32_t u = __float_as_uint(x), cut = u & 0xFFFF0000u;
    return __uint_as_float((x < 0.f && cut != u) ? cut + 0x10000u : cut);
}
__device__ __forceinline__ float bf16_ceil(float x) { return -bf16_floor(-x); }

// The smallest and the largest of a thread's 8 values, NaN if one is: 16-bit types two at a
// time.
__device__ __forceinline__ float min_nan(float x, float y) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ void extremes(const Raw8<HC_DTYPE_FP32>& r, float& lo, float& hi) {
    const float x[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
    lo = hi = x[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) lo = min_nan(lo, x[i]), hi = max_nan(hi, x[i]);
}
template <typename Two>
__device__ __forceinline__ void extremes_of(const uint4& v, Two& lo, Two& hi) {
    const Two a = *reinterpret_cast<const Two*>(&v.x), b = *reinterpret_cast<const Two*>(&v.y),
              c = *reinterpret_cast<const Two*>(&v.z), d = *reinterpret_cast<const Two*>(&v.w);
    lo = __hmin2_nan(__hmin2_nan(a, b), __hmin2_nan(c, d));
    hi = __hmax2_nan(__hmax2_nan(a, b), __hmax2_nan(c, d));
}
__device__ __forceinline__ void extremes(const Raw8<HC_DTYPE_BF16>& r, float& lo, float& hi) {
    __nv_bfloat162 l, h;
    extremes_of(r.v, l, h);
    lo = min_nan(__low2float(l), __high2float(l)), hi = max_nan(__low2float(h), __high2float(h));
}
__device__ __forceinline__ void extremes(const Raw8<HC_DTYPE_FP16>& r, float& lo, float& hi) {
    __half2 l, h;
    extremes_of(r.v, l, h);
    lo = min_nan(__low2float(l), __high2float(l)), hi = max_nan(__low2float(h), __high2float(h));
}

// A group's step and minimum from its extremes: packed as the cache holds them, the minimum, and 1 / step
// (0 where the step is). False for a group that is held as NaN.
__device__ __forceinline__ bool group_steps(float lo, float hi, uint32_t& sm, float& m, float& r) {
    m = bf16_floor(lo);
    const float width = __fsub_rn(hi, m);
    float s = bf16_ceil(__fmul_rn(width, 1.0f / 15.0f));
    // 2^-126, so that 1 / s is finite
    if (s > 0.f && s < __uint_as_float(0x00800000u)) s = __uint_as_float(0x00800000u);
    const float top = __uint_as_float(0x7F7FFFFFu);
    if (!(fabsf(lo) <= top && fabsf(hi) <= top && s <= top)) {
        sm = 0x7FC07FC0u;
        return false;
    }
    r = s > 0.f ? __frcp_rn(s) : 0.f;
    sm = (__float_as_uint(s) >> 16) | (__float_as_uint(m) & 0xFFFF0000u);
    return true;
}
// A lane's 8 codes. One is at most 15 by itself: s >= width / 15 up to 2^-23, so that (x - m) / s rounds to 15 at
// most. 2^23 + 2^22 + z holds z rounded to the nearest integer, ties to even, in its low bits.
template <int kDtype>
__device__ __forceinline__ uint32_t group_codes(const Raw8<kDtype>& raw, float m, float r) {
    float x[8];
    raw.get(x);
    constexpr float kRound = 12582912.f;
    const uint64_t m2 = pair(-m, -m), r2 = pair(r, r);
    uint32_t bits[8];
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        // the product is rounded before the sum: two at a time the compiler joins them to one FMA
        const float2 z = unpair(mul2(add2(pair(x[i], x[i + 1]), m2), r2));
        bits[i] = __float_as_uint(__fadd_rn(z.x, kRound));
        bits[i + 1] = __float_as_uint(__fadd_rn(z.y, kRound));
    }
    uint32_t code = bits[7];
#pragma unroll
    for (int i = 6; i >= 0; --i) code = code * 16 + bits[i];
    return code - 0x4B400000u * 0x11111111u;
}
// Rounds one group spread over kLanes neighbouring lanes; returns the lane's 8 codes
// and, in sm, the packed bf16 step and minimum.
template <int kLanes, int kDtype>
__device__ __forceinline__ uint32_t round_group(const Raw8<kDtype>& raw, uint32_t& sm) {
    float lo, hi, m, r;
    extremes(raw, lo, hi);
#pragma unroll
    for (int d = kLanes / 2; d > 0; d >>= 1) {
        lo = min_nan(lo, __shfl_xor_sync(~0u, lo, d));
        hi = max_nan(hi, __shfl_xor_sync(~0u, hi, d));
    }
    return group_steps(lo, hi, sm, m, r) ? group_codes(raw, m, r) : 0;
}
// The same for lanes of 8 values of each half of a group.
template <int kLanes, int kDtype>
__device__ __forceinline__ uint2 round_group(const Raw8<kDtype> (&raw)[2], uint32_t& sm) {
    float lo, hi, lo2, hi2, m, r;
    extremes(raw[0], lo, hi);
    extremes(raw[1], lo2, hi2);
    lo = min_nan(lo, lo2), hi = max_nan(hi, hi2);
#pragma unroll
    for (int d = kLanes / 2; d > 0; d >>= 1) {
        lo = min_nan(lo, __shfl_xor_sync(~0u, lo, d));
        hi = max_nan(hi, __shfl_xor_sync(~0u, hi, d));
    }
    if (!group_steps(lo, hi, sm, m, r)) return make_uint2(0, 0);
    return make_uint2(group_codes(raw[0], m, r), group_codes(raw[1], m, r));
}

// Index of a slot's group among all groups of the cache, or -1 (with the status bit)
// where the slot lies outside.
__device__ __forceinline__ int64_t group_index(const hc_kv4_cache& c, int sh, int64_t slot, int kv,
                                               int head, int* status) {
    const int64_t block = slot >> sh;
    if (block >= c.blocks) {
        atomicOr(status, kStatusBounds);
        return -1;
    }
    return (((block * 2 + kv) * c.kv_heads + head) << sh) + (slot & (c.block_size - 1));
}

}  // namespace hc
