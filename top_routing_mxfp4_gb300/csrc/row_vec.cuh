// Rows of bf16 or fp32 elements in registers, and sums over a row's threads.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace lmoe {

// W consecutive elements as they lie in memory (aligned: H % 8 == 0, 16-byte
// aligned rows) and as fp32.
template <typename T, int W>
struct Pack;
template <int W>
struct Pack<uint16_t, W> {
    uint32_t u[W / 2];
    __device__ __forceinline__ void load(const uint16_t *p)
    {
        if constexpr (W == 8) {
            const uint4 v = *reinterpret_cast<const uint4 *>(p);
            u[0] = v.x, u[1] = v.y, u[2] = v.z, u[3] = v.w;
        } else {
            const uint2 v = *reinterpret_cast<const uint2 *>(p);
            u[0] = v.x, u[1] = v.y;
        }
    }
    __device__ __forceinline__ void get(float (&v)[W]) const
    {
#pragma unroll
        for (int i = 0; i < W / 2; ++i) {
            v[2 * i] = __uint_as_float(u[i] << 16);
            v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
        }
    }
    __device__ __forceinline__ void set(const float (&v)[W])  // rounded to nearest even
    {
#pragma unroll
        for (int i = 0; i < W / 2; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t *>(&b);
        }
    }
    __device__ __forceinline__ void store(uint16_t *p) const
    {
        if constexpr (W == 8)
            *reinterpret_cast<uint4 *>(p) = make_uint4(u[0], u[1], u[2], u[3]);
        else
            *reinterpret_cast<uint2 *>(p) = make_uint2(u[0], u[1]);
    }
};
template <int W>
struct Pack<float, W> {
    float4 q[W / 4];
    __device__ __forceinline__ void load(const float *p)
    {
#pragma unroll
        for (int i = 0; i < W / 4; ++i) q[i] = reinterpret_cast<const float4 *>(p)[i];
    }
    __device__ __forceinline__ void get(float (&v)[W]) const
    {
#pragma unroll
        for (int i = 0; i < W / 4; ++i) v[4 * i] = q[i].x, v[4 * i + 1] = q[i].y, v[4 * i + 2] = q[i].z, v[4 * i + 3] = q[i].w;
    }
    __device__ __forceinline__ void set(const float (&v)[W])
    {
#pragma unroll
        for (int i = 0; i < W / 4; ++i) q[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    }
    __device__ __forceinline__ void store(float *p) const
    {
#pragma unroll
        for (int i = 0; i < W / 4; ++i) reinterpret_cast<float4 *>(p)[i] = q[i];
    }
};

// Sum over a row's threads (a warp, or the whole block), the same value in
// every thread and in a fixed order.  `part` is used once per call.
template <bool WARP>
__device__ __forceinline__ float row_sum(float s, float *part)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    if (WARP) return s;
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
    __syncthreads();
    const int nw = int(blockDim.x) >> 5, lane = threadIdx.x & 31;
    s = lane < nw ? part[lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    return s;
}

// Two sums over a warp at once, half a warp each from the first step on; the same in every lane.
__device__ __forceinline__ float2 warp_sum2(float a, float b)
{
    const int which = (threadIdx.x >> 4) & 1;
    float s = which ? b : a;
    s += __shfl_xor_sync(0xFFFFFFFFu, which ? a : b, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    return make_float2(__shfl_sync(0xFFFFFFFFu, s, 0), __shfl_sync(0xFFFFFFFFu, s, 16));
}

// Two fp32 values as one operand of the packed instructions.  (The assembler may join a
// product and a sum into one rounding: where two instances have to agree bit for bit, they
// say fma2.)
struct F2 {
    uint64_t v;
};
__device__ __forceinline__ F2 f2(float lo, float hi)
{
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ F2 f2(float both) { return f2(both, both); }
__device__ __forceinline__ void f2_get(F2 a, float &lo, float &hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a.v)); }
__device__ __forceinline__ F2 operator+(F2 a, F2 b)
{
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b)
{
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c)
{
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ float f2_sum(F2 a)
{
    float lo, hi;
    f2_get(a, lo, hi);
    return lo + hi;
}
// A Pack's elements as pairs, and back.
template <int W>
__device__ __forceinline__ void pairs(const Pack<uint16_t, W> &p, F2 (&v)[W / 2])
{
#pragma unroll
    for (int i = 0; i < W / 2; ++i) v[i] = f2(__uint_as_float(p.u[i] << 16), __uint_as_float(p.u[i] & 0xFFFF0000u));
}
template <int W>
__device__ __forceinline__ void pairs(const Pack<float, W> &p, F2 (&v)[W / 2])
{
#pragma unroll
    for (int i = 0; i < W / 4; ++i) v[2 * i] = f2(p.q[i].x, p.q[i].y), v[2 * i + 1] = f2(p.q[i].z, p.q[i].w);
}
template <int W>
__device__ __forceinline__ void set_pairs(Pack<uint16_t, W> &p, const F2 (&v)[W / 2])
{
#pragma unroll
    for (int i = 0; i < W / 2; ++i) {
        float lo, hi;
        f2_get(v[i], lo, hi);
        const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
        p.u[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
}
template <int W>
__device__ __forceinline__ void set_pairs(Pack<float, W> &p, const F2 (&v)[W / 2])
{
#pragma unroll
    for (int i = 0; i < W / 4; ++i) {
        f2_get(v[2 * i], p.q[i].x, p.q[i].y);
        f2_get(v[2 * i + 1], p.q[i].z, p.q[i].w);
    }
}

}  // namespace lmoe
