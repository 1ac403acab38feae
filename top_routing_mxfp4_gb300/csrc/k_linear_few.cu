// Linear layer with bias, function and residual for few rows (decode batches):
//   z = x W^T + bias,  out = fn(z) + res,  pre = bf16(z)
// and the gradient by x of few rows, dx = dz W (`across`: the reduction runs over the
// weights' rows).
//
// The weight stream bounds it, so the weights are the M = 128 operand (A, K-major or,
// across, MN-major: two blocks of 64 elements) and the rows the N operand (B, K-major, 16
// to 64 of them, so that one token costs no 128 rows of copies), 64 of the reduction a
// chunk.  An output tile's K is shared by a
// cluster of KS CTAs, so that few tiles stream with the whole GPU; the ranks' sums
// are added in rank order (cluster_sum.cuh), each rank finishing a share of the rows.
// One row 3584 -> 7168 11.7 us, 64 rows 13.2 (weights that lie in L2: 7.6 us at HBM speed
// and about 4 of start, cluster sum and end); 7168 -> 28672, from HBM, 70 (5.9 TB/s, 87%).
// At 128 rows the tiles of k_linear_act win (21.1 against 17.5 us).
//
// One tile a cluster, up to two CTAs an SM: warp 0 copies, warp 1 issues the MMAs,
// four epilogue warps.  Every wait is bounded (LMOE_ERR_TIMEOUT in the status word).
#include <cuda.h>
#include <cuda_bf16.h>

#include "act_fn.cuh"
#include "cluster_sum.cuh"
#include "lmoe_internal.cuh"
#include "tc_ptx.cuh"
#include "tensor_map.cuh"

namespace lmoe {
namespace {

using namespace tc;

constexpr uint32_t A_TILE = 128 * 128;  // 128 weight rows x 64 bf16

template <int NT>
struct FCfg {
    static constexpr uint32_t B_TILE = NT * 128;
    static constexpr uint32_t STAGE = A_TILE + B_TILE;
    static constexpr uint32_t RED = ClusterSum::red_bytes(NT);
    static constexpr int PER_SM = 2;
    static constexpr int S = int((110 * 1024 - RED) / STAGE);
    static constexpr uint32_t TMEM_COLS = NT < 32 ? 32 : NT;
    static_assert(NT <= 64, "two CTAs an SM");
    static_assert(S * STAGE >= NT * 512, "the sums are staged in the ring");
};

struct FArgs {
    const void *bias, *res;
    int bias_f32, res_f32, out_f32, fn;
    int rows, N, KC, KS;
    int across;
    void *out;
    uint16_t *pre;
    int32_t *status;
    long long limit;
    int stall;
};

template <int NT>
__global__ void __launch_bounds__(192, FCfg<NT>::PER_SM)
    k_linear_few(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, const FArgs p)
{
    using C = FCfg<NT>;
    constexpr int S = C::S;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *stages = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float *red = reinterpret_cast<float *>(stages + S * C::STAGE);
    uint64_t *full = reinterpret_cast<uint64_t *>(red + C::RED / 4);
    uint64_t *empty = full + S;
    uint64_t *acc_full = empty + S;
    uint64_t *drain = acc_full + 1;
    uint64_t *red_full = drain + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(red_full + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(acc_full, 1);
        mbar_init(drain, 1);
        mbar_init(red_full, 1);
        mbar_init_fence();
        prefetch_tensormap(&tmA);
        prefetch_tensormap(&tmB);
    }
    if (warp == 1) tmem_alloc(tmem_slot, C::TMEM_COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (p.KS > 1) cluster_sync();  // the cluster's barriers are initialised
    const uint32_t tmem = *tmem_slot;
    const int rank = p.KS > 1 ? int(cluster_rank()) : 0, tile = int(blockIdx.x) / p.KS;
    const int m0 = tile * 128, cols = p.rows;
    const int k0 = rank * p.KC / p.KS, k1 = (rank + 1) * p.KC / p.KS;  // this rank's chunks
    // The first weights on their way to L2 (which the kernel before may still write them to)
    // while that kernel ends: 64 rows 3584 -> 7168 15.6 -> 14.8 us, one row 12.3 -> 11.9; twice
    // as many took longer than none.
    if (warp == 0) {
        if (elect_one())
            for (int kc = k0; kc < min(k1, k0 + S); ++kc) {
                if (p.across) {
                    tma_prefetch_2d(&tmA, m0, kc * 64);
                    tma_prefetch_2d(&tmA, m0 + 64, kc * 64);
                } else {
                    tma_prefetch_2d(&tmA, kc * 64, m0);
                }
            }
        __syncwarp();
    }
    pdl_enter();

    if (warp == 0) {
        // ---------------- copies ----------------
        int stage = 0, fills = 0;
        uint32_t phase = 0;
        bool ok = true;
        const uint64_t once = l2_policy_evict_first(), keep = l2_policy_evict_normal();
        for (int kc = k0; kc < k1; ++kc) {
            ok = mbar_wait_warp(&empty[stage], phase ^ 1, p.limit);
            if (!ok) {
                if (lane == 0) set_status(p.status, LMOE_ERR_TIMEOUT);
                break;
            }
            if (elect_one() && !(p.stall && kc == k0)) {
                uint8_t *sb = stages + stage * C::STAGE;
                mbar_arrive_expect_tx(&full[stage], C::STAGE);
                if (p.across) {
                    tma_load_2d_hint(sb, &tmA, m0, kc * 64, &full[stage], once);
                    tma_load_2d_hint(sb + 8192, &tmA, m0 + 64, kc * 64, &full[stage], once);
                } else {
                    tma_load_2d_hint(sb, &tmA, kc * 64, m0, &full[stage], once);
                }
                tma_load_2d_hint(sb + A_TILE, &tmB, kc * 64, 0, &full[stage], keep);
            }
            __syncwarp();
            ++fills;
            if (++stage == S) {
                stage = 0;
                phase ^= 1;
            }
        }
        if (!ok)  // copies still in flight land before the CTA ends (bounded)
            for (int f = fills > S ? fills - S : 0; f < fills; ++f) mbar_wait_warp(&full[f % S], (f / S) & 1, p.limit);
    } else if (warp == 1) {
        // ---------------- MMA issuer ----------------
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        const uint32_t id = idesc_bf16(uint32_t((cols + 15) & ~15)) | (p.across ? IDESC_A_MN : 0);
        const uint32_t base = smem_u32(stages), a_step = p.across ? 128 : 2;
        const uint64_t ad0 = p.across ? sdesc_mn128(base, 8192) : sdesc_k128(base), bd0 = sdesc_k128(base + A_TILE);
        for (int kc = k0; kc < k1; ++kc) {
            ok = mbar_wait_warp(&full[stage], phase, p.limit);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
                const uint64_t ad = ad0 + uint32_t(stage) * (C::STAGE >> 4), bd = bd0 + uint32_t(stage) * (C::STAGE >> 4);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)  // 4 x K = 16
                    mma_bf16(tmem, ad + a_step * kk, bd + 2 * kk, id, (kc > k0 || kk > 0) ? 1u : 0u);
                tc_commit(&empty[stage]);
            }
            __syncwarp();
            if (++stage == S) {
                stage = 0;
                phase ^= 1;
            }
        }
        if (elect_one()) {
            if (ok) {
                tc_commit(acc_full);
            } else {
                set_status(p.status, LMOE_ERR_TIMEOUT);
                tc_commit(drain);  // MMAs in flight end before the tensor memory is freed
                mbar_wait(drain, 0, p.limit);
            }
        }
        __syncwarp();
    } else {
        // ---------------- epilogue: a lane has an output column, its rows one after another ----------------
        const int q = warp & 3, n = m0 + 32 * q + lane;
        const bool mine = n < p.N;
        float bias = 0.f;
        if (p.bias && mine)
            bias = p.bias_f32 ? __ldg(static_cast<const float *>(p.bias) + n) : bf16_bits_to_f32(__ldg(static_cast<const uint16_t *>(p.bias) + n));
        // rows [c0, c1) of the tile, at most 16
        auto finish = [&](int c0, int c1, const float (&y)[16]) {
            const int64_t at = int64_t(c0) * p.N + n;
            float r[16] = {};
            if (p.res)
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (mine && c0 + j < c1)
                        r[j] = p.res_f32 ? static_cast<const float *>(p.res)[at + int64_t(j) * p.N]
                                         : bf16_bits_to_f32(static_cast<const uint16_t *>(p.res)[at + int64_t(j) * p.N]);
            F2 z[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) z[j] = f2(y[2 * j], y[2 * j + 1]) + f2(bias);
            auto store = [&](void *base, bool f32) {
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    if (!mine || c0 + j >= c1) continue;
                    float lo, hi;
                    f2_get(z[j / 2], lo, hi);
                    const int64_t i = at + int64_t(j) * p.N;
                    if (f32) static_cast<float *>(base)[i] = j & 1 ? hi : lo;
                    else static_cast<__nv_bfloat16 *>(base)[i] = __float2bfloat16_rn(j & 1 ? hi : lo);
                }
            };
            if (p.pre) store(p.pre, false);
            apply_fn(p.fn, z);
            if (p.res)
#pragma unroll
                for (int j = 0; j < 8; ++j) z[j] = z[j] + f2(r[2 * j], r[2 * j + 1]);
            store(p.out, p.out_f32);
        };
        if (!mbar_wait_warp(acc_full, 0, p.limit)) {
            if (lane == 0) set_status(p.status, LMOE_ERR_TIMEOUT);
        } else {
            tc_fence_after();
            const uint32_t tb = tmem + (uint32_t(32 * q) << 16);
            if (p.KS == 1) {
                for (int c = 0; c < cols; c += 16) {
                    uint32_t v[16];
                    tmem_ld16(tb + c, v);
                    tmem_ld_wait();
                    float y[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) y[j] = __uint_as_float(v[j]);
                    finish(c, cols, y);
                }
            } else {
                const ClusterSum cs(p.KS, rank, cols, reinterpret_cast<float *>(stages), red, red_full);
                for (int c = 0; c < cols; c += 16) {
                    uint32_t v[16];
                    tmem_ld16(tb + c, v);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (c + j < cols) cs.stage[(c + j) * 128 + 32 * q + lane] = __uint_as_float(v[j]);
                }
                if (!cs.exchange(p.limit)) {
                    if (lane == 0) set_status(p.status, LMOE_ERR_TIMEOUT);
                } else {
                    for (int c = cs.own0; c < cs.own1; c += 16) {
                        float y[16];
                        cs.sum(c, 32 * q + lane, y);
                        finish(c, cs.own1, y);
                    }
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    // nobody's shared memory goes while another CTA may still write or read it
    if (p.KS > 1) cluster_sync_end();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, C::TMEM_COLS);
}

template <int NT>
cudaError_t launch(const FewArgs &a, FArgs g, cudaStream_t st)
{
    using C = FCfg<NT>;
    CUtensorMap ma, mb;
    if (!(a.across ? make_tensor_map(&ma, a.W, MapType::BF16, a.N, a.K, 64) : make_tensor_map(&ma, a.W, MapType::BF16, a.K, a.N, 128)) ||
        !make_tensor_map(&mb, a.x, MapType::BF16, a.K, a.rows, NT, a.x_stride))
        return cudaErrorInvalidValue;
    const int64_t tiles = ceil_div(a.N, 128);
    // K is shared so that the CTAs fill the GPU's slots, two an SM, once, each with four
    // chunks at least.  One an SM took 20.8 against 15.9 us at 64 rows of 3584 -> 7168 and
    // as long at one row (12.6 against 12.5 us).
    const int64_t slots = int64_t(device_sms()) * C::PER_SM;
    int ks = 8;
    while (ks > 1 && (tiles * ks > slots || g.KC < 4 * ks)) --ks;
    g.KS = ks;
    const size_t smem = 1024 + size_t(C::S) * C::STAGE + C::RED + (2 * C::S + 3) * 8 + 8;
    const cudaError_t e = cudaFuncSetAttribute(k_linear_few<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(tiles * ks));
    cfg.blockDim = dim3(192);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(ks);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ks > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, k_linear_few<NT>, ma, mb, g);
}

}  // namespace

cudaError_t launch_linear_few(const FewArgs &a, cudaStream_t st)
{
    FArgs g{};
    g.bias = a.bias;
    g.bias_f32 = a.bias_fmt == LMOE_F32;
    g.res = a.res;
    g.res_f32 = a.res_fmt == LMOE_F32;
    g.out_f32 = a.out_fmt == LMOE_F32;
    g.fn = a.fn;
    g.rows = int(a.rows);
    g.N = a.N;
    g.KC = int(ceil_div(a.K, 64));
    g.across = a.across;
    g.out = a.out;
    g.pre = a.pre;
    g.status = a.status;
    g.limit = a.wait.limit > 0 ? a.wait.limit : 4000000000LL;  // about 2 s of SM clocks
    g.stall = a.wait.stall_first_fill;
    if (a.rows <= 16) return launch<16>(a, g, st);
    if (a.rows <= 32) return launch<32>(a, g, st);
    return launch<64>(a, g, st);
}

}  // namespace lmoe
