// Norms around a block: the norm before it (RMSNorm of the residual stream),
// and after it the norm of its output, the gate and the residual scale fused
// with the residual add and the norm before the next block.
//
//   s  = post_w ? y * rsqrt(mean(y^2) + eps) * post_w : y
//   r' = res + scale * gate * s              (rounded to the stream's type)
//   n  = bf16( r' * rsqrt(mean(r'^2) + eps) * next_w )   (r' as stored)
//
// One pass over the data: a row's elements stay in registers (8 * VPT a
// thread) between the two statistics, so y and res are read once and r' and n
// written once.  All arithmetic and both sums of squares are fp32; r' and n
// are rounded once, to nearest even.
#include <cuda_bf16.h>

#include "lmoe_internal.cuh"

namespace lmoe {
namespace {

// 8 consecutive elements as they lie in memory (16-byte aligned rows, H % 8 == 0)
// and as fp32.
template <typename T>
struct Vec8;
template <>
struct Vec8<uint16_t> {
    uint4 u;
    __device__ __forceinline__ void load(const uint16_t *p) { u = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void get(float (&v)[8]) const
    {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    __device__ __forceinline__ void set(const float (&v)[8])  // rounded to nearest even
    {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&b);
        }
        u = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ __forceinline__ void store(uint16_t *p) const { *reinterpret_cast<uint4 *>(p) = u; }
};
template <>
struct Vec8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p)
    {
        a = reinterpret_cast<const float4 *>(p)[0];
        b = reinterpret_cast<const float4 *>(p)[1];
    }
    __device__ __forceinline__ void get(float (&v)[8]) const
    {
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
    __device__ __forceinline__ void set(const float (&v)[8])
    {
        a = make_float4(v[0], v[1], v[2], v[3]);
        b = make_float4(v[4], v[5], v[6], v[7]);
    }
    __device__ __forceinline__ void store(float *p) const
    {
        reinterpret_cast<float4 *>(p)[0] = a;
        reinterpret_cast<float4 *>(p)[1] = b;
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

// R: the residual stream's type.  VPT: 8-element vectors a thread.  WARP: a
// warp takes a row (several rows a block), else a block takes one.  All of a
// row's loads are issued before the first statistic; what waits in registers
// stays in its own type.
template <typename R, int VPT, bool WARP>
__global__ void __launch_bounds__(VPT == 1 ? 1024 : 512) k_residual_norm(const NormArgs p)
{
    __shared__ float part[2][32];
    const int tid = WARP ? int(threadIdx.x & 31) : int(threadIdx.x);
    const int nt = WARP ? 32 : int(blockDim.x);
    const int64_t t = WARP ? int64_t(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5) : int64_t(blockIdx.x);
    pdl_enter();
    if (WARP && t >= p.T) return;
    const int nv = p.H >> 3;
    const int64_t row = t * p.H;
    const R *res = static_cast<const R *>(p.res) + row;
    Vec8<R> r[VPT];
    float ss = 0.f;
    if (p.y) {
        Vec8<uint16_t> y[VPT], g[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (tid + i * nt < nv) y[i].load(p.y + row + (tid + i * nt) * 8);
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (tid + i * nt < nv) r[i].load(res + (tid + i * nt) * 8);
        if (p.gate_kind == LMOE_GATE_FULL)
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                if (tid + i * nt < nv) g[i].load(static_cast<const uint16_t *>(p.gate) + row + (tid + i * nt) * 8);
        const float tg = p.gate_kind == LMOE_GATE_TOKEN ? p.scale * static_cast<const float *>(p.gate)[t] : p.scale;
        float ys = 1.f;
        if (p.post_w) {
            float q = 0.f;
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                if (tid + i * nt < nv) {
                    float v[8];
                    y[i].get(v);
#pragma unroll
                    for (int j = 0; j < 8; ++j) q = fmaf(v[j], v[j], q);
                }
            ys = __frsqrt_rn(row_sum<WARP>(q, part[0]) / float(p.H) + p.eps);
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (tid + i * nt) * 8;
            if (c >= p.H) continue;
            float v[8], a[8];
            y[i].get(v);
            if (p.post_w) {
                Vec8<float> w;
                w.load(p.post_w + c);
                w.get(a);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] *= ys * a[j];
            }
            if (p.gate_kind == LMOE_GATE_FULL) {
                g[i].get(a);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] *= a[j];
            } else if (p.gate_kind == LMOE_GATE_CHANNEL) {
                Vec8<float> w;
                w.load(static_cast<const float *>(p.gate) + c);
                w.get(a);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] *= a[j];
            }
            r[i].get(a);
#pragma unroll
            for (int j = 0; j < 8; ++j) a[j] = fmaf(tg, v[j], a[j]);
            r[i].set(a);
            r[i].store(static_cast<R *>(p.res_out) + row + c);
            r[i].get(a);  // as stored
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(a[j], a[j], ss);
        }
    } else {
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (tid + i * nt < nv) r[i].load(res + (tid + i * nt) * 8);
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (tid + i * nt < nv) {
                float a[8];
                r[i].get(a);
#pragma unroll
                for (int j = 0; j < 8; ++j) ss = fmaf(a[j], a[j], ss);
            }
    }
    if (!p.next_w) return;
    const float rs = __frsqrt_rn(row_sum<WARP>(ss, part[1]) / float(p.H) + p.eps);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = (tid + i * nt) * 8;
        if (c >= p.H) continue;
        float v[8], a[8];
        Vec8<float> w;
        w.load(p.next_w + c);
        w.get(a);
        r[i].get(v);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= rs * a[j];
        Vec8<uint16_t> n;
        n.set(v);
        n.store(p.next_out + row + c);
    }
}

template <typename R>
cudaError_t launch(const NormArgs &a, cudaStream_t st)
{
    const int nv = a.H / 8;
    if (nv <= 128) {  // a warp holds a row
        const int warps = a.T >= 152 * 16 ? 4 : 1;
        const dim3 grid(unsigned(ceil_div(a.T, warps))), block(32 * warps);
        if (nv <= 32) return launch_pdl(k_residual_norm<R, 1, true>, grid, block, 0, st, a);
        if (nv <= 64) return launch_pdl(k_residual_norm<R, 2, true>, grid, block, 0, st, a);
        return launch_pdl(k_residual_norm<R, 4, true>, grid, block, 0, st, a);
    }
    const dim3 grid{unsigned(a.T)};
    // Few rows: a vector a thread, the shortest way from load to store (1001
    // rows of 3584 fp32: 5.8 us against 6.1 with two).  Many: HBM is the bound,
    // and fewer, longer rows' worth of threads leave room for more blocks; at
    // 8192 rows of 7168, by vectors a thread:
    //   bf16 stream, y and a gate per element (587 MB)  1: 109  2: 104  3: 89.4  4: 90.6 us (6.57 TB/s at 3)
    //   fp32 stream, y, gate per token (705 MB)         1: 128  2: 125  3: 127   4: 132 us
    //   norm of a bf16 stream alone (235 MB)            1: 67   2: 60   3: 47    4: 43 us
    int vpt = a.T <= 8 * 152 ? 1 : a.res_fmt == LMOE_F32 ? 2 : a.y ? 3 : 4;
    if (nv > (vpt == 1 ? 1024 : 512 * vpt)) vpt = nv <= 1024 ? 2 : nv <= 1536 ? 3 : nv <= 2048 ? 4 : 8;
    const dim3 block(unsigned(round_up(ceil_div(nv, vpt), 32)));
    switch (vpt) {
    case 1: return launch_pdl(k_residual_norm<R, 1, false>, grid, block, 0, st, a);
    case 2: return launch_pdl(k_residual_norm<R, 2, false>, grid, block, 0, st, a);
    case 3: return launch_pdl(k_residual_norm<R, 3, false>, grid, block, 0, st, a);
    case 4: return launch_pdl(k_residual_norm<R, 4, false>, grid, block, 0, st, a);
    default: return launch_pdl(k_residual_norm<R, 8, false>, grid, block, 0, st, a);
    }
}

}  // namespace

cudaError_t launch_residual_norm(const NormArgs &a, cudaStream_t st)
{
    if (a.T == 0) return cudaSuccess;
    return a.res_fmt == LMOE_F32 ? launch<float>(a, st) : launch<uint16_t>(a, st);
}

}  // namespace lmoe
