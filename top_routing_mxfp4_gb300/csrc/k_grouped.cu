// bf16 products grouped by expert, ragged groups:
//   out[q][n] = w(q) * sum_c x[src(q)][c] * W[e(q)][n][c]
// and the gated pair h[q][i] = bf16( silu(g) * u ).
//
// First, plain form: a block owns 32 rows of one group and 32 output columns,
// both operands' 32-column slices in shared memory, fp32 products and sums.
#include <cuda_bf16.h>

#include "lmoe_internal.cuh"

namespace lmoe {
namespace {

constexpr int BT = 32;

// Offsets of a group, checked: false (and the status word) unless
// 0 <= o0 <= o1 <= P.
__device__ __forceinline__ bool group_ok(const GroupedArgs &p, int o0, int o1)
{
    if (o0 >= 0 && o0 <= o1 && o1 <= p.P) return true;
    set_status(p.status, LMOE_ERR_DEVICE_CHECK);
    return false;
}

__global__ void __launch_bounds__(256) k_grouped_plain(const GroupedArgs p)
{
    __shared__ float xs[BT][BT + 1], ws[BT][BT + 1], us[BT][BT + 1];
    __shared__ int src[BT];
    pdl_enter();
    const int n0 = blockIdx.x * BT, tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    for (int e = blockIdx.y; e < p.E; e += gridDim.y) {
        const int o0 = p.offsets[e], o1 = p.offsets[e + 1];
        if (!group_ok(p, o0, o1)) continue;
        for (int r0 = o0; r0 < o1; r0 += BT) {
            __syncthreads();
            if (threadIdx.x < BT) {
                int sr = -1;
                if (r0 + tx < o1) {
                    sr = p.gather ? p.perm[r0 + tx] / p.k : r0 + tx;
                    if (sr < 0 || sr >= p.x_rows) {
                        set_status(p.status, LMOE_ERR_DEVICE_CHECK);
                        sr = -1;
                    }
                }
                src[tx] = sr;
            }
            __syncthreads();
            float a[4] = {}, b[4] = {};
            for (int c0 = 0; c0 < p.K; c0 += BT) {
                for (int i = ty; i < BT; i += 8) {
                    const bool in = c0 + tx < p.K;
                    xs[i][tx] = in && src[i] >= 0 ? bf16_bits_to_f32(p.x[int64_t(src[i]) * p.K + c0 + tx]) : 0.f;
                    const int64_t wr = (int64_t(e) * p.N + n0 + i) * p.K + c0 + tx;
                    const bool wi = in && n0 + i < p.N;
                    ws[i][tx] = wi ? bf16_bits_to_f32(p.W[wr]) : 0.f;
                    us[i][tx] = wi && p.W2 ? bf16_bits_to_f32(p.W2[wr]) : 0.f;
                }
                __syncthreads();
                for (int c = 0; c < BT; ++c)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        a[j] = fmaf(xs[ty + 8 * j][c], ws[tx][c], a[j]);
                        b[j] = fmaf(xs[ty + 8 * j][c], us[tx][c], b[j]);
                    }
                __syncthreads();
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t qr = r0 + ty + 8 * j;
                if (qr >= o1 || n0 + tx >= p.N) continue;
                float v = p.W2 ? a[j] / (1.f + __expf(-a[j])) * b[j] : a[j];
                if (p.row_w) {
                    const int64_t pr = p.perm ? p.perm[qr] : qr;
                    if (pr >= 0 && pr < p.P)
                        v *= p.row_w[pr];
                    else
                        set_status(p.status, LMOE_ERR_DEVICE_CHECK);
                }
                if (p.out_fmt == LMOE_F32)
                    static_cast<float *>(p.out)[qr * p.N + n0 + tx] = v;
                else
                    static_cast<__nv_bfloat16 *>(p.out)[qr * p.N + n0 + tx] = __float2bfloat16_rn(v);
            }
        }
    }
}

}  // namespace

cudaError_t launch_grouped(const GroupedArgs &a, cudaStream_t st)
{
    return launch_pdl(k_grouped_plain, dim3(unsigned(ceil_div(a.N, BT)), unsigned(a.E)), dim3(256), 0, st, a);
}

}  // namespace lmoe
