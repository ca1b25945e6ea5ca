// Epilogue arithmetic of the dense matrix products: activations in fp32, conversions between fp32 and
// the 16-bit element types.
#pragma once
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace dpa {

// The activations use the hardware exponential and reciprocal: a few units in the last place of
// fp32, of the size of the product's own summation error.
//   silu       v / (1 + exp(-v))
//   gelu_tanh  v (1 + tanh p) / 2 = v / (1 + exp(-2p)), p = sqrt(2/pi) (v + 0.044715 v^3)
//   gelu       v Phi(v). The tail is Phi(-a) = exp(-a^2/2) R(a), a = |v|, which keeps its relative
//              accuracy for negative v; R is a polynomial of degree 7 in t = 1 / (1 + 0.35 a),
//              fitted here to exp(a^2/2) Phi(-a) on [0, 14] for the least relative error (3.1e-7;
//              beyond 14 the exponential is 0 in fp32).
__device__ __forceinline__ float act_gelu(float v) {
    const float t = __fdividef(1.f, fmaf(0.35f, fabsf(v), 1.f));
    float r = fmaf(0.04894237592816353f, t, -0.20211902260780334f);
    r = fmaf(r, t, 0.24064041674137115f);
    r = fmaf(r, t, -0.017023101449012756f);
    r = fmaf(r, t, 0.15596133470535278f);
    r = fmaf(r, t, 0.13335514068603516f);
    r = fmaf(r, t, 0.14027033746242523f);
    r = fmaf(r, t, -2.7315189072396606e-05f);
    const float q = __expf(-0.5f * v * v) * r;   // Phi(-|v|)
    return v * (v > 0.f ? 1.f - q : q);
}
__device__ __forceinline__ float act_one(float v, int act) {
    switch (act) {
        case DPA_ACT_RELU: return v < 0.f ? 0.f : v;   // NaN stays NaN
        case DPA_ACT_GELU: return act_gelu(v);
        case DPA_ACT_GELU_TANH:
            return __fdividef(v, 1.f + __expf(-1.5957691216057308f * fmaf(0.044715f * v * v, v, v)));
        case DPA_ACT_SILU: return __fdividef(v, 1.f + __expf(-v));
        default: return v;
    }
}

template <int CNT>
__device__ __forceinline__ void act_many(float (&v)[CNT], int act) {
    switch (act) {   // one branch for the whole array
        case DPA_ACT_RELU:
#pragma unroll
            for (int j = 0; j < CNT; ++j) v[j] = act_one(v[j], DPA_ACT_RELU);
            break;
        case DPA_ACT_GELU:
#pragma unroll
            for (int j = 0; j < CNT; ++j) v[j] = act_one(v[j], DPA_ACT_GELU);
            break;
        case DPA_ACT_GELU_TANH:
#pragma unroll
            for (int j = 0; j < CNT; ++j) v[j] = act_one(v[j], DPA_ACT_GELU_TANH);
            break;
        case DPA_ACT_SILU:
#pragma unroll
            for (int j = 0; j < CNT; ++j) v[j] = act_one(v[j], DPA_ACT_SILU);
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

template <bool F16>
__device__ __forceinline__ float bias_at(const void* b, int64_t i) {
    return b ? up16<F16>(__ldg(static_cast<const uint16_t*>(b) + i)) : 0.f;
}

}  // namespace dpa
