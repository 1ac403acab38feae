// The functions a linear layer's sums go through, and their slopes.
//
// All by one quick exponential (2 u of itself and of its argument) and one quick
// division whose divisor stays small, about 10 instructions an element (the gelu
// 20): with expf and erfcf the epilogue of a 256-column tile took 4 us, more than
// the products of a K of 512.
#pragma once

#include <stdint.h>

#include "../../include/lmoe.h"

namespace lmoe {

constexpr float TANH_C = 1.5957691216057308f;  // 2 sqrt(2 / pi)

// z / (1 + e^-u) by e^-|u|, so that the divisor stays in [1, 2].
__device__ __forceinline__ float times_logistic(float z, float u)
{
    const float e = __expf(-fabsf(u));
    return __fdividef(u < 0.f ? z * e : z, 1.f + e);
}

// The normal distribution's tail Phi(-a), a >= 0: e^(-a^2/2) t P(t), t = 1 / (1 + 0.35 a),
// P the polynomial of degree 8 with the least relative error on 0 <= a <= 14 (fitted
// here: 3.2e-8, 3e-7 in fp32).  It keeps the tail's relative accuracy, which 1 - erf loses.
// e: e^(-a^2/2).
__device__ __forceinline__ float normal_tail(float a, float e)
{
    const float t = __fdividef(1.f, fmaf(0.35f, a, 1.f));
    float p = -0.02914592747752851f;
    p = fmaf(p, t, 0.1439716837960093f);
    p = fmaf(p, t, -0.2557142249928744f);
    p = fmaf(p, t, 0.15917412686130336f);
    p = fmaf(p, t, -0.023109812541916113f);
    p = fmaf(p, t, 0.10550799488766614f);
    p = fmaf(p, t, 0.11983286980729112f);
    p = fmaf(p, t, 0.13986186940214104f);
    p = fmaf(p, t, 0.13962140431170578f);
    return e * (p * t);
}

template <int FN>
__device__ __forceinline__ float apply(float z)
{
    if (FN == LMOE_FN_RELU) return z < 0.f ? 0.f : z;  // (a NaN stays)
    if (FN == LMOE_FN_SILU) return times_logistic(z, z);
    if (FN == LMOE_FN_GELU) {
        const float q = normal_tail(fabsf(z), __expf(-0.5f * z * z));
        return z * (z < 0.f ? q : 1.f - q);
    }
    if (FN == LMOE_FN_GELU_TANH) return times_logistic(z, TANH_C * fmaf(0.044715f * z, z * z, z));
    return z;
}
__device__ __forceinline__ float apply_fn(int fn, float z)
{
    switch (fn) {
    case LMOE_FN_RELU: return apply<LMOE_FN_RELU>(z);
    case LMOE_FN_SILU: return apply<LMOE_FN_SILU>(z);
    case LMOE_FN_GELU: return apply<LMOE_FN_GELU>(z);
    case LMOE_FN_GELU_TANH: return apply<LMOE_FN_GELU_TANH>(z);
    default: return z;
    }
}
template <int FN>
__device__ __forceinline__ float slope(float z)
{
    if (FN == LMOE_FN_RELU) return z > 0.f ? 1.f : (z <= 0.f ? 0.f : z);
    if (FN == LMOE_FN_GELU) {
        const float e = __expf(-0.5f * z * z), q = normal_tail(fabsf(z), e);
        return fmaf(z * 0.39894228f, e, z < 0.f ? q : 1.f - q);
    }
    if (FN == LMOE_FN_SILU || FN == LMOE_FN_GELU_TANH) {
        const float u = FN == LMOE_FN_SILU ? z : TANH_C * fmaf(0.044715f * z, z * z, z);
        const float du = FN == LMOE_FN_SILU ? 1.f : TANH_C * fmaf(3 * 0.044715f * z, z, 1.f);
        const float e = __expf(-fabsf(u)), r = __fdividef(1.f, 1.f + e);
        const float s = u < 0.f ? e * r : r, rest = u < 0.f ? r : e * r;  // the logistic function and 1 - it
        return e == 0.f ? s : fmaf(z * du, s * rest, s);  // (e = 0: z du may be infinite)
    }
    return 1.f;
}

}  // namespace lmoe
