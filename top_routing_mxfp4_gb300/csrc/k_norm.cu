// Norms around a block: the norm before it (RMSNorm of the residual stream),
// and after it the norm of its output, the gate and the residual scale fused
// with the residual add and the norm before the next block.
//
//   s  = post_w ? y * rsqrt(mean(y^2) + eps) * post_w : y
//   r' = res + scale * gate * s              (rounded to the stream's type)
//   n  = bf16( r' * rsqrt(mean(r'^2) + eps) * next_w )   (r' as stored)
//
// One pass over the data: a row's elements stay in registers between the two statistics, so y and res are read once and r' and n
// written once.  All arithmetic and both sums of squares are fp32; r' and n
// are rounded once, to nearest even.
#include <cuda_bf16.h>

#include "lmoe_internal.cuh"

namespace lmoe {
namespace {

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

// R: the residual stream's type.  E8: eighths of a thread's elements.  WARP: a
// warp takes a row (several rows a block), else a block takes one.  All of a
// row's loads are issued before the first statistic; what waits in registers
// stays in its own type.  A thread's vectors are 16 bytes of the stream (an fp32
// one in 32-byte pieces would leave each store instruction half of its sectors:
// 125 against 113 us at 8192 rows of 7168).
template <typename R, int E8, bool WARP>
__global__ void __launch_bounds__(E8 == 1 ? 1024 : 512) k_residual_norm(const NormArgs p)
{
    constexpr int W = 16 / int(sizeof(R)), VPT = E8 * 8 / W;
    __shared__ float part[2][32];
    const int tid = WARP ? int(threadIdx.x & 31) : int(threadIdx.x);
    const int nt = WARP ? 32 : int(blockDim.x);
    const int64_t t = WARP ? int64_t(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5) : int64_t(blockIdx.x);
    pdl_enter();
    if (WARP && t >= p.T) return;
    const int nv = p.H / W;
    const int64_t row = t * p.H;
    const R *res = static_cast<const R *>(p.res) + row;
    Pack<R, W> r[VPT];
    float ss = 0.f;
    if (p.y) {
        Pack<uint16_t, W> y[VPT], g[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (tid + i * nt < nv) y[i].load(p.y + row + (tid + i * nt) * W);
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (tid + i * nt < nv) r[i].load(res + (tid + i * nt) * W);
        if (p.gate_kind == LMOE_GATE_FULL)
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                if (tid + i * nt < nv) g[i].load(static_cast<const uint16_t *>(p.gate) + row + (tid + i * nt) * W);
        const float tg = p.gate_kind == LMOE_GATE_TOKEN ? p.scale * static_cast<const float *>(p.gate)[t] : p.scale;
        float ys = 1.f;
        if (p.post_w) {
            float q = 0.f;
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                if (tid + i * nt < nv) {
                    float v[W];
                    y[i].get(v);
#pragma unroll
                    for (int j = 0; j < W; ++j) q = fmaf(v[j], v[j], q);
                }
            ys = __frsqrt_rn(row_sum<WARP>(q, part[0]) / float(p.H) + p.eps);
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (tid + i * nt) * W;
            if (c >= p.H) continue;
            float v[W], a[W];
            y[i].get(v);
            if (p.post_w) {
                Pack<float, W> w;
                w.load(p.post_w + c);
                w.get(a);
#pragma unroll
                for (int j = 0; j < W; ++j) v[j] *= ys * a[j];
            }
            if (p.gate_kind == LMOE_GATE_FULL) {
                g[i].get(a);
#pragma unroll
                for (int j = 0; j < W; ++j) v[j] *= a[j];
            } else if (p.gate_kind == LMOE_GATE_CHANNEL) {
                Pack<float, W> w;
                w.load(static_cast<const float *>(p.gate) + c);
                w.get(a);
#pragma unroll
                for (int j = 0; j < W; ++j) v[j] *= a[j];
            }
            r[i].get(a);
#pragma unroll
            for (int j = 0; j < W; ++j) a[j] = fmaf(tg, v[j], a[j]);
            r[i].set(a);
            r[i].store(static_cast<R *>(p.res_out) + row + c);
            r[i].get(a);  // as stored
#pragma unroll
            for (int j = 0; j < W; ++j) ss = fmaf(a[j], a[j], ss);
        }
    } else {
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (tid + i * nt < nv) r[i].load(res + (tid + i * nt) * W);
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (tid + i * nt < nv) {
                float a[W];
                r[i].get(a);
#pragma unroll
                for (int j = 0; j < W; ++j) ss = fmaf(a[j], a[j], ss);
            }
    }
    if (!p.next_w) return;
    const float rs = __frsqrt_rn(row_sum<WARP>(ss, part[1]) / float(p.H) + p.eps);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = (tid + i * nt) * W;
        if (c >= p.H) continue;
        float v[W], a[W];
        Pack<float, W> w;
        w.load(p.next_w + c);
        w.get(a);
        r[i].get(v);
#pragma unroll
        for (int j = 0; j < W; ++j) v[j] *= rs * a[j];
        Pack<uint16_t, W> n;
        n.set(v);
        n.store(p.next_out + row + c);
    }
}

template <typename R>
cudaError_t launch(const NormArgs &a, cudaStream_t st)
{
    const int nv = a.H / 8;  // eights a row
    if (nv <= 128) {  // a warp holds a row
        const int warps = a.T >= 152 * 16 ? 4 : 1;
        const dim3 grid(unsigned(ceil_div(a.T, warps))), block(32 * warps);
        if (nv <= 32) return launch_pdl(k_residual_norm<R, 1, true>, grid, block, 0, st, a);
        if (nv <= 64) return launch_pdl(k_residual_norm<R, 2, true>, grid, block, 0, st, a);
        return launch_pdl(k_residual_norm<R, 4, true>, grid, block, 0, st, a);
    }
    const dim3 grid{unsigned(a.T)};
    // Few rows: eight elements a thread, the shortest way from load to store (1001
    // rows of 3584 fp32: 5.7 us against 6.8 with sixteen).  Many: HBM is the
    // bound, and fewer threads a row leave room for more blocks, while an fp32
    // stream's shorter rows want the threads; by eights a thread, us:
    //   bf16 stream, y, gate per element, 8192 x 7168 (587 MB)  1: 109   2: 104   3: 89.4  4: 90.6 (6.57 TB/s at 3)
    //   bf16 stream, y, gate per token,   8192 x 3584           1: 48.3  2: 43.7  3: 42.0  4: 42.7
    //   norm of a bf16 stream alone,      8192 x 7168 (235 MB)  1: 67    2: 60    3: 47    4: 43
    //   fp32 stream, y, gate per token,   8192 x 7168 (705 MB)  1: 114   2: 113   3: 108   4: 131 (6.51 TB/s at 3)
    //                                     8192 x 5120           1: 78.6  2: 79.7  3: 80.2  4: 84.2
    //   norm of an fp32 stream alone,     8192 x 7168           1: 66.9  2: 64.3  3: 56.0  4: 70.3
    //                                     20000 x 3000          1: 59.7  2: 57.1  3: 54.6  4: 61.4
    //                                     8192 x 2048           1: 17.3  2: 17.6  3: 18.1  4: 20.1
    int e8 = 1;
    if (a.T > 8 * 152) e8 = a.res_fmt != LMOE_F32 ? (a.y ? 3 : 4) : nv > (a.y ? 768 : 300) ? 3 : 1;
    if (nv > (e8 == 1 ? 1024 : 512 * e8)) e8 = nv <= 1024 ? 2 : nv <= 1536 ? 3 : nv <= 2048 ? 4 : 8;
    const dim3 block(unsigned(round_up(ceil_div(nv, e8), 32)));
    switch (e8) {
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
