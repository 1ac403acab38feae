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

// 8 consecutive elements as fp32 (16-byte aligned rows, H % 8 == 0)
__device__ __forceinline__ void load8(const uint16_t *p, float *v)
{
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void load8(const float *p, float *v)
{
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
// stores 8 elements in the destination's type and leaves the stored values in v
__device__ __forceinline__ void store8(uint16_t *p, float *v)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&b);
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float *p, float *v)
{
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

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
// warp takes a row (several rows a block), else a block takes one.
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
    float r[VPT][8];
    if (p.y) {
        float y[VPT][8], ss = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = tid + i * nt;
#pragma unroll
            for (int j = 0; j < 8; ++j) y[i][j] = 0.f;
            if (c < nv) load8(p.y + row + c * 8, y[i]);
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = tid + i * nt;
            if (c < nv) load8(res + c * 8, r[i]);
        }
        if (p.post_w) {
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) ss = fmaf(y[i][j], y[i][j], ss);
            ss = __frsqrt_rn(row_sum<WARP>(ss, part[0]) / float(p.H) + p.eps);
        }
        const float tg = p.gate_kind == LMOE_GATE_TOKEN ? p.scale * static_cast<const float *>(p.gate)[t] : p.scale;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = tid + i * nt;
            if (c >= nv) continue;
            if (p.post_w) {
                float w[8];
                load8(p.post_w + c * 8, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) y[i][j] *= ss * w[j];
            }
            if (p.gate_kind == LMOE_GATE_CHANNEL || p.gate_kind == LMOE_GATE_FULL) {
                float g[8];
                if (p.gate_kind == LMOE_GATE_CHANNEL)
                    load8(static_cast<const float *>(p.gate) + c * 8, g);
                else
                    load8(static_cast<const uint16_t *>(p.gate) + row + c * 8, g);
#pragma unroll
                for (int j = 0; j < 8; ++j) y[i][j] *= g[j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) r[i][j] = fmaf(tg, y[i][j], r[i][j]);
            store8(static_cast<R *>(p.res_out) + row + c * 8, r[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = tid + i * nt;
            if (c < nv) load8(res + c * 8, r[i]);
        }
    }
    if (!p.next_w) return;
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
        if (tid + i * nt < nv)
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(r[i][j], r[i][j], ss);
    const float rs = __frsqrt_rn(row_sum<WARP>(ss, part[1]) / float(p.H) + p.eps);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = tid + i * nt;
        if (c >= nv) continue;
        float w[8];
        load8(p.next_w + c * 8, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) r[i][j] *= rs * w[j];
        store8(p.next_out + row + c * 8, r[i]);
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
    auto threads = [&](int vpt) { return dim3(unsigned(round_up(ceil_div(nv, vpt), 32))); };
    if (a.T <= 304 && nv <= 1024) return launch_pdl(k_residual_norm<R, 1, false>, grid, threads(1), 0, st, a);
    if (nv <= 1024) return launch_pdl(k_residual_norm<R, 2, false>, grid, threads(2), 0, st, a);
    if (nv <= 2048) return launch_pdl(k_residual_norm<R, 4, false>, grid, threads(4), 0, st, a);
    return launch_pdl(k_residual_norm<R, 8, false>, grid, threads(8), 0, st, a);
}

}  // namespace

cudaError_t launch_residual_norm(const NormArgs &a, cudaStream_t st)
{
    if (a.T == 0) return cudaSuccess;
    return a.res_fmt == LMOE_F32 ? launch<float>(a, st) : launch<uint16_t>(a, st);
}

}  // namespace lmoe
