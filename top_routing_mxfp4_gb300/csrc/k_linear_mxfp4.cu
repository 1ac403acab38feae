// MXFP4 linear on bf16 rows: out[r][n] = bf16( sum_c x[r][c] * W[n][c] ).
//
// First, plain form: a warp owns one output feature n and eight rows; each
// lane takes every 32nd block of 32 columns (16 bytes of codes, one scale
// byte), sums the block's products of e2m1 values and x in fp32 and adds the
// sum times the block's scale.
#include <cuda_bf16.h>

#include "lmoe_internal.cuh"

namespace lmoe {
namespace {

__device__ __forceinline__ float e2m1_val(uint32_t c)
{
    // magnitudes 0, .5, 1, 1.5, 2, 3, 4, 6
    const uint32_t m = c & 7;
    const float v = m < 2 ? 0.5f * float(m) : ldexpf(1.f + 0.5f * float(m & 1), int(m >> 1) - 1);
    return (c & 8) ? -v : v;
}

__global__ void __launch_bounds__(128) k_linear_plain(const uint16_t *__restrict__ x, const uint8_t *__restrict__ q,
                                                      const uint8_t *__restrict__ s, int64_t rows, int K, int N,
                                                      uint16_t *__restrict__ out)
{
    pdl_enter();
    const int n = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int64_t r0 = int64_t(blockIdx.y) * 8;
    if (n >= N) return;
    const int KC = int(ceil_div(K, 128));
    float acc[8] = {};
    for (int b = lane; b < K / 32; b += 32) {
        const uint4 w4 = *reinterpret_cast<const uint4 *>(q + int64_t(n) * KC * 64 + b * 16);
        const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
        const float sc = e8m0_to_f32(s[tile_atom_off(n, b, KC, 128)]);
        float v[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = e2m1_val(w[i >> 3] >> (4 * (i & 7)));
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            if (r0 + r >= rows) break;
            const uint16_t *xr = x + (r0 + r) * K + b * 32;
            float d = 0.f;
#pragma unroll
            for (int i = 0; i < 32; ++i) d = fmaf(bf16_bits_to_f32(xr[i]), v[i], d);
            acc[r] = fmaf(d, sc, acc[r]);
        }
    }
#pragma unroll
    for (int r = 0; r < 8; ++r) {
        float a = acc[r];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
        if (lane == 0 && r0 + r < rows) {
            const __nv_bfloat16 h = __float2bfloat16_rn(a);
            out[(r0 + r) * N + n] = *reinterpret_cast<const uint16_t *>(&h);
        }
    }
}

}  // namespace

size_t linear_mxfp4_scratch_bytes(int64_t, int, int) { return 0; }

cudaError_t launch_linear_mxfp4(const uint16_t *x, const uint8_t *q, const uint8_t *s, int64_t rows, int K, int N,
                                uint16_t *out, void *, int32_t *, const WaitArgs &, cudaStream_t st)
{
    for (int64_t r0 = 0; r0 < rows; r0 += 8 * 65535) {  // grid.y limit
        const int64_t n = rows - r0 < 8 * 65535 ? rows - r0 : 8 * 65535;
        const cudaError_t e = launch_pdl(k_linear_plain, dim3(unsigned(ceil_div(N, 4)), unsigned(ceil_div(n, 8))),
                                         dim3(128), 0, st, x + r0 * K, q, s, n, K, N, out + r0 * N);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace lmoe
