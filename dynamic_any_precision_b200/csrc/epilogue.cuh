// Epilogue arithmetic of the dense matrix products: activations in fp32, conversions between fp32 and
// the 16-bit element types.
#pragma once
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"

namespace dpa {

// ---- two fp32 values in one register pair: one instruction for both ----
struct Two {
    uint64_t v;
};
__device__ __forceinline__ Two two(float lo, float hi) {
    Two r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ Two both(float v) { return two(v, v); }
__device__ __forceinline__ float2 apart(Two a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
    return r;
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
    Two r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ Two mul2(Two a, Two b) {
    Two r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ Two add2(Two a, Two b) {
    Two r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ float ex2(float v) {   // 2^v
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float rcp(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ Two ex2(Two a) {
    const float2 f = apart(a);
    return two(ex2(f.x), ex2(f.y));
}
__device__ __forceinline__ Two rcp(Two a) {
    const float2 f = apart(a);
    return two(rcp(f.x), rcp(f.y));
}
__device__ __forceinline__ float min_nan(float a, float b) {   // NaN if either is
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// The activations, two values at a time. They use the hardware's 2^v and reciprocal: a few units in
// the last place of fp32 (6e-7) where the exponential's argument is small. The argument (v, 2p, a^2/2)
// is rounded to fp32, so towards the negative tail the relative error grows with it, to 3.8e-6 (silu),
// 8.8e-6 (gelu_tanh) and 8.2e-6 (gelu) at arguments of 85; a rounding of v itself, and so the product's
// own summation error, does as much there. Where the exponential passes 2^126 the reciprocal is flushed:
// results of silu and gelu_tanh below |v| 2^-126 (1.0e-36, 1.2e-37) become 0.
//   silu       v / (1 + exp(-v))
//   gelu_tanh  v (1 + tanh p) / 2 = v / (1 + exp(-2p)), p = sqrt(2/pi) (v + 0.044715 v^3)
//   gelu       v Phi(v) = max(v, 0) - a Phi(-a), a = |v|, with Phi(-a) = exp(-a^2/2) R(a), which
//              keeps its relative accuracy for negative v. R is a polynomial of degree 7 in
//              t = 1 / (1 + 0.35 a), fitted here to exp(a^2/2) Phi(-a) on [0, 14] for the least
//              relative error (3.1e-7; beyond 14 the exponential is 0 in fp32). a stops at 1e30, so
//              that +inf gives +inf and -inf its limit 0.
constexpr float kLog2e = 1.44269504088896341f;
__device__ __forceinline__ Two silu2(Two v) {
    return mul2(v, rcp(add2(both(1.f), ex2(mul2(v, both(-kLog2e))))));
}
__device__ __forceinline__ Two gelu_tanh2(Two v) {
    constexpr float c = -2.f * 0.797884560802865356f * kLog2e;
    const Two p = mul2(v, fma2(mul2(v, v), both(c * 0.044715f), both(c)));
    return mul2(v, rcp(add2(both(1.f), ex2(p))));
}
__device__ __forceinline__ Two gelu2(Two v) {
    const float2 f = apart(v);
    const Two a = two(min_nan(fabsf(f.x), 1e30f), min_nan(fabsf(f.y), 1e30f));
    const Two t = rcp(fma2(a, both(0.35f), both(1.f)));
    Two r = fma2(both(-0.04894237592816353f), t, both(0.20211902260780334f));   // -R
    r = fma2(r, t, both(-0.24064041674137115f));
    r = fma2(r, t, both(0.017023101449012756f));
    r = fma2(r, t, both(-0.15596133470535278f));
    r = fma2(r, t, both(-0.13335514068603516f));
    r = fma2(r, t, both(-0.14027033746242523f));
    r = fma2(r, t, both(2.7315189072396606e-05f));
    const Two e = ex2(mul2(mul2(a, both(-0.5f * kLog2e)), a));
    return fma2(mul2(r, e), a, two(fmaxf(f.x, 0.f), fmaxf(f.y, 0.f)));
}
__device__ __forceinline__ Two relu2(Two v) {   // NaN stays NaN
    const float2 f = apart(v);
    return two(f.x < 0.f ? 0.f : f.x, f.y < 0.f ? 0.f : f.y);
}

__device__ __forceinline__ Two act2(Two v, int act) {
    switch (act) {
        case DPA_ACT_RELU: return relu2(v);
        case DPA_ACT_GELU: return gelu2(v);
        case DPA_ACT_GELU_TANH: return gelu_tanh2(v);
        case DPA_ACT_SILU: return silu2(v);
        default: return v;
    }
}
__device__ __forceinline__ float act_one(float v, int act) { return apart(act2(two(v, v), act)).x; }

template <int CNT>
__device__ __forceinline__ void act_many(Two (&v)[CNT], int act) {
    switch (act) {   // one branch for the whole array
        case DPA_ACT_RELU:
#pragma unroll
            for (int j = 0; j < CNT; ++j) v[j] = relu2(v[j]);
            break;
        case DPA_ACT_GELU:
#pragma unroll
            for (int j = 0; j < CNT; ++j) v[j] = gelu2(v[j]);
            break;
        case DPA_ACT_GELU_TANH:
#pragma unroll
            for (int j = 0; j < CNT; ++j) v[j] = gelu_tanh2(v[j]);
            break;
        case DPA_ACT_SILU:
#pragma unroll
            for (int j = 0; j < CNT; ++j) v[j] = silu2(v[j]);
            break;
        default: break;
    }
}

template <bool F16>
__device__ __forceinline__ float up16(uint16_t b) {
    if constexpr (F16) return __half2float(__ushort_as_half(b));
    else return bf16_bits_to_float(b);
}
template <bool F16>
__device__ __forceinline__ uint16_t down16(float v) {
    if constexpr (F16) return __half_as_ushort(__float2half_rn(v));
    else return __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// two values in one word, the first in the low half (one instruction, off the transcendental unit
// that single conversions share with the activations)
template <bool F16>
__device__ __forceinline__ uint32_t down16x2(float lo, float hi) {
    uint32_t r;
    if constexpr (F16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

template <bool F16>
__device__ __forceinline__ float bias_at(const void* b, int64_t i) {
    return b ? up16<F16>(__ldg(static_cast<const uint16_t*>(b) + i)) : 0.f;
}

// One output: adds its residual, rounds once and stores it (`out` may be the residual itself).
template <bool F16>
__device__ __forceinline__ void store_one(const LinearArgs& a, float o, int64_t at) {
    if (a.residual)
        o += a.res32 ? static_cast<const float*>(a.residual)[at]
                     : up16<F16>(static_cast<const uint16_t*>(a.residual)[at]);
    if (a.out32) static_cast<float*>(a.out)[at] = o;
    else static_cast<uint16_t*>(a.out)[at] = down16<F16>(o);
}

}  // namespace dpa
