// The functions a linear layer's sums go through, and their slopes.
//
// By one quick exponential (2 u of itself and of its argument) and one quick reciprocal
// each, two elements at a time in packed fp32 arithmetic: 7 instructions an element for
// silu and gelu by tanh, 12 for gelu.  The epilogue of a tile is bound by them where K is
// short (8192 rows 512 -> 3584, us: silu 36, gelu 40; 39 and 55 with expf's quick form and
// __fdividef one element at a time).
//
// With a = |z|, the logistic function's and the normal distribution's left tails go
// into max(z, 0) - a tail(a), right for both signs, and exact far out.
#pragma once

#include <stdint.h>

#include "../../include/lmoe.h"
#include "row_vec.cuh"

namespace lmoe {

constexpr float TANH_C = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float LOG2E = 1.4426950408889634f;

__device__ __forceinline__ float exp2_quick(float x)  // off by 2 u; results below 2^-126 are 0
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_quick(float x)  // off by 1 u
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
template <typename F>
__device__ __forceinline__ F2 each(F2 a, F f)
{
    float lo, hi;
    f2_get(a, lo, hi);
    return f2(f(lo), f(hi));
}

// max(z, 0) - |z| tail
__device__ __forceinline__ F2 less_tail(F2 z, F2 tail)
{
    const F2 a = each(z, [](float v) { return -fminf(fabsf(v), 1e30f); });  // (infinity times a tail of 0)
    return fma2(a, tail, each(z, [](float v) { return fmaxf(v, 0.f); }));
}
// z / (1 + e^-u), u of z's sign.  The tail e^-|u| / (1 + e^-|u|) by the square of e^(-|u| / 2),
// one factor times z first: it keeps values down to 2^-126.
__device__ __forceinline__ F2 times_logistic(F2 z, F2 u)
{
    const F2 h = each(u * f2(0.5f * LOG2E), [](float v) { return exp2_quick(-fabsf(v)); });
    const F2 r = each(fma2(h, h, f2(1.f)), [](float v) { return rcp_quick(v); });
    const F2 a = each(z, [](float v) { return -fminf(fabsf(v), 1e30f); });
    return fma2(a * h, h * r, each(z, [](float v) { return fmaxf(v, 0.f); }));
}

// The normal distribution's tail Phi(-a), a >= 0: e^(-a^2/2) t P(t), t = 1 / (1 + 0.35 a),
// P the polynomial of degree 8 with the least relative error on 0 <= a <= 14 (fitted
// here: 3.2e-8, 3e-7 in fp32).  It keeps the tail's relative accuracy, which 1 - erf loses.
// e: e^(-a^2/2).
__device__ __forceinline__ F2 normal_tail(F2 a, F2 e)
{
    const F2 t = each(fma2(f2(0.35f), a, f2(1.f)), [](float v) { return rcp_quick(v); });
    F2 p = f2(-0.02914592747752851f);
    p = fma2(p, t, f2(0.1439716837960093f));
    p = fma2(p, t, f2(-0.2557142249928744f));
    p = fma2(p, t, f2(0.15917412686130336f));
    p = fma2(p, t, f2(-0.023109812541916113f));
    p = fma2(p, t, f2(0.10550799488766614f));
    p = fma2(p, t, f2(0.11983286980729112f));
    p = fma2(p, t, f2(0.13986186940214104f));
    p = fma2(p, t, f2(0.13962140431170578f));
    return e * (p * t);
}
__device__ __forceinline__ F2 bell(F2 z)  // e^(-z^2/2)
{
    return each((z * z) * f2(-0.5f * LOG2E), [](float v) { return exp2_quick(v); });
}
__device__ __forceinline__ F2 magnitude(F2 z) { return each(z, [](float v) { return fabsf(v); }); }
// TANH_C (z + 0.044715 z^3)
__device__ __forceinline__ F2 tanh_arg(F2 z) { return z * fma2(z * z, f2(0.044715f * TANH_C), f2(TANH_C)); }

template <int FN>
__device__ __forceinline__ F2 apply(F2 z)
{
    if constexpr (FN == LMOE_FN_RELU) return each(z, [](float v) { return v < 0.f ? 0.f : v; });  // (a NaN stays)
    else if constexpr (FN == LMOE_FN_SILU) return times_logistic(z, z);
    else if constexpr (FN == LMOE_FN_GELU) return less_tail(z, normal_tail(magnitude(z), bell(z)));
    else if constexpr (FN == LMOE_FN_GELU_TANH) return times_logistic(z, tanh_arg(z));
    else return z;
}
// y = fn(y), the function chosen once.
template <int N>
__device__ __forceinline__ void apply_fn(int fn, F2 (&y)[N])
{
    auto all = [&](auto f) {
#pragma unroll
        for (int j = 0; j < N; ++j) y[j] = f(y[j]);
    };
    switch (fn) {
    case LMOE_FN_RELU: all([](F2 z) { return apply<LMOE_FN_RELU>(z); }); break;
    case LMOE_FN_SILU: all([](F2 z) { return apply<LMOE_FN_SILU>(z); }); break;
    case LMOE_FN_GELU: all([](F2 z) { return apply<LMOE_FN_GELU>(z); }); break;
    case LMOE_FN_GELU_TANH: all([](F2 z) { return apply<LMOE_FN_GELU_TANH>(z); }); break;
    default: break;
    }
}

// The factor of a term that fades out: infinity times zero is none.  (A NaN of z's comes back with the other factor.)
__device__ __forceinline__ F2 finite(F2 z) { return each(z, [](float v) { return fminf(fmaxf(v, -1e30f), 1e30f); }); }

template <int FN>
__device__ __forceinline__ F2 slope(F2 z)
{
    if constexpr (FN == LMOE_FN_RELU) {
        return each(z, [](float v) { return v > 0.f ? 1.f : (v <= 0.f ? 0.f : v); });
    } else if constexpr (FN == LMOE_FN_GELU) {
        // z < 0: q + z e / sqrt(2 pi), else 1 - q + ...
        const F2 e = bell(z), q = normal_tail(magnitude(z), e);
        float z0, z1, q0, q1;
        f2_get(z, z0, z1);
        f2_get(q, q0, q1);
        return fma2(finite(z) * f2(0.39894228f), e, f2(z0 < 0.f ? q0 : 1.f - q0, z1 < 0.f ? q1 : 1.f - q1));
    } else if constexpr (FN == LMOE_FN_SILU || FN == LMOE_FN_GELU_TANH) {
        const F2 u = FN == LMOE_FN_SILU ? z : tanh_arg(z);
        const F2 du = fma2(z * z, f2(3 * 0.044715f * TANH_C), f2(TANH_C));  // of gelu by tanh
        const F2 e = each(u * f2(LOG2E), [](float v) { return exp2_quick(-fabsf(v)); });
        const F2 r = each(e + f2(1.f), [](float v) { return rcp_quick(v); });
        const F2 er = e * r;  // the logistic function of u is r or er, by u's sign, and 1 - it the other
        float u0, u1, r0, r1, s0, s1;
        f2_get(u, u0, u1);
        f2_get(r, r0, r1);
        f2_get(er, s0, s1);
        // (far out z du is infinite, where r er is 0)
        const F2 zd = FN == LMOE_FN_SILU ? finite(z) : finite(z * du);
        return fma2(zd, r * er, f2(u0 < 0.f ? s0 : r0, u1 < 0.f ? s1 : r1));
    } else {
        return f2(1.f);
    }
}

}  // namespace lmoe
