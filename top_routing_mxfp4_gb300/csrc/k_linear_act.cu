// Linear layer with bias, function and residual, and its gradients, on the tensor
// cores (tcgen05.mma kind::f16, fp32 accumulation in TMEM):
//   z = x W^T + bias,  out = fn(z) + res,  pre = bf16(z)
//   dz = dout fn'(pre),  dx = dz W,  dW = dz^T x,  dbias = sum of dz's rows
//
// One kernel makes all three products, D[m][n] = sum_k A(m, k) B(n, k): the operands
// are read as they lie, K-major (x and W forward, dz in dx: the reduction runs along
// a row) or MN-major (W in dx; dz and x in dW: it runs over the rows), 64 of the
// reduction a chunk, and TMA zero-fills what lies beyond an edge.
//
// Persistent CTAs: warp 0 copies (TMA), warp 1 issues the MMAs, the others are the
// epilogue (TMEM lane quarter = warp % 4), which adds bias, applies the function,
// adds the residual and stores, a row a lane, while the next tile's MMAs run in the
// other accumulator.  Every wait is bounded (LMOE_ERR_TIMEOUT in the status word).
#include <cuda.h>
#include <cuda_bf16.h>

#include "act_fn.cuh"
#include "lmoe_internal.cuh"
#include "row_vec.cuh"
#include "tc_ptx.cuh"
#include "tensor_map.cuh"

namespace lmoe {
namespace {

using namespace tc;

constexpr uint32_t A_TILE = 128 * 128;  // 128 x 64 bf16
constexpr int MAX_PARTS = 16;

template <int NT, bool PAIR>
struct LCfg {
    static constexpr int EW = 8;  // epilogue warps, two per TMEM lane quarter (32 columns each in turn)
    static constexpr int THREADS = 32 * (2 + EW);
    static constexpr int CL = PAIR ? 2 : 1;  // CTAs a tile: a pair (cta_group::2) has 256 rows of A, each CTA half of B
    static constexpr int MT = 128 * CL;
    static constexpr int BROWS = NT / CL;
    static constexpr uint32_t B_TILE = BROWS * 128;
    static constexpr uint32_t STAGE = A_TILE + B_TILE;
    static constexpr int S_RAW = int(200 * 1024 / STAGE);
    static constexpr int S = S_RAW > 8 ? 8 : S_RAW;
    static constexpr int ACC = 2;  // accumulators: a tile's epilogue overlaps the next one's MMAs
    static constexpr uint32_t TMEM_COLS = ACC * NT;
};

struct LArgs {
    int64_t M;
    int N, KC;       // chunks of the reduction
    int MTL, NTL;    // tiles
    int KS;          // parts of the reduction; with more than one, part k's sums go to out + k M N (fp32)
    // epilogue
    const void *bias, *res;
    int bias_f32, res_f32, out_f32, fn;
    int vec;         // outputs' and residual's rows take vectors of this many bytes (32, 16) or single elements (0)
    void *out;
    uint16_t *pre;
    int32_t *status;
    long long limit;
    int stall;
};

// ---- rows of outputs ---------------------------------------------------------------------

// 32 consecutive elements of a row, fp32 or bf16, as 32-bit words.
template <bool F32>
constexpr int WORDS = F32 ? 32 : 16;

template <bool F32>
__device__ __forceinline__ void row_load(uint32_t (&u)[32], const void *base, int64_t at, int n, int vec)
{
    const char *p = static_cast<const char *>(base) + at * (F32 ? 4 : 2);
    if (n == 32 && vec == 32) {
#pragma unroll
        for (int i = 0; i < WORDS<F32>; i += 8)
            asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                         : "=r"(u[i]), "=r"(u[i + 1]), "=r"(u[i + 2]), "=r"(u[i + 3]), "=r"(u[i + 4]), "=r"(u[i + 5]),
                           "=r"(u[i + 6]), "=r"(u[i + 7])
                         : "l"(p + 4 * i)
                         : "memory");
    } else if (n == 32 && vec == 16) {
#pragma unroll
        for (int i = 0; i < WORDS<F32>; i += 4) {
            const uint4 v = *reinterpret_cast<const uint4 *>(p + 4 * i);
            u[i] = v.x, u[i + 1] = v.y, u[i + 2] = v.z, u[i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < WORDS<F32>; ++i) {
            if (F32) {
                u[i] = i < n ? reinterpret_cast<const uint32_t *>(p)[i] : 0u;
            } else {
                const uint16_t *h = reinterpret_cast<const uint16_t *>(p);
                u[i] = (2 * i < n ? uint32_t(h[2 * i]) : 0u) | (2 * i + 1 < n ? uint32_t(h[2 * i + 1]) << 16 : 0u);
            }
        }
    }
}
template <bool F32>
__device__ __forceinline__ void row_add(const uint32_t (&u)[32], F2 (&y)[16])
{
#pragma unroll
    for (int i = 0; i < 16; ++i)
        y[i] = y[i] + (F32 ? f2(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1]))
                           : f2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xFFFF0000u)));
}
// Rounded to nearest even.
template <bool F32>
__device__ __forceinline__ void row_store(const F2 (&y)[16], void *base, int64_t at, int n, int vec)
{
    uint32_t u[WORDS<F32>];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        float lo, hi;
        f2_get(y[i], lo, hi);
        if constexpr (F32) {
            u[2 * i] = __float_as_uint(lo);
            u[2 * i + 1] = __float_as_uint(hi);
        } else {
            const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
            u[i] = *reinterpret_cast<const uint32_t *>(&b);
        }
    }
    char *p = static_cast<char *>(base) + at * (F32 ? 4 : 2);
    if (n == 32 && vec == 32) {
#pragma unroll
        for (int i = 0; i < WORDS<F32>; i += 8)
            asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p + 4 * i), "r"(u[i]), "r"(u[i + 1]),
                         "r"(u[i + 2]), "r"(u[i + 3]), "r"(u[i + 4]), "r"(u[i + 5]), "r"(u[i + 6]), "r"(u[i + 7])
                         : "memory");
    } else if (n == 32 && vec == 16) {
#pragma unroll
        for (int i = 0; i < WORDS<F32>; i += 4)
            *reinterpret_cast<uint4 *>(p + 4 * i) = make_uint4(u[i], u[i + 1], u[i + 2], u[i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < WORDS<F32>; ++i) {
            if (F32) {
                if (i < n) reinterpret_cast<uint32_t *>(p)[i] = u[i];
            } else {
                uint16_t *h = reinterpret_cast<uint16_t *>(p);
                if (2 * i < n) h[2 * i] = uint16_t(u[i]);
                if (2 * i + 1 < n) h[2 * i + 1] = uint16_t(u[i] >> 16);
            }
        }
    }
}

// ---- the products ------------------------------------------------------------------------

// A_MN, B_MN: the operand's reduction runs over the rows of its matrix.
template <int NT, bool PAIR, bool A_MN, bool B_MN>
__global__ void __launch_bounds__((LCfg<NT, PAIR>::THREADS), 1)
    k_linear_act(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, const LArgs p)
{
    using C = LCfg<NT, PAIR>;
    constexpr int S = C::S;
    static_assert(!B_MN || C::BROWS % 64 == 0, "blocks of 64 elements");
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *stages = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(stages + S * C::STAGE);
    uint64_t *empty = full + S;
    uint64_t *acc_full = empty + S;
    uint64_t *acc_empty = acc_full + C::ACC;
    uint64_t *drain = acc_empty + C::ACC;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int a = 0; a < C::ACC; ++a) {
            mbar_init(&acc_full[a], 1);
            mbar_init(&acc_empty[a], 32 * C::EW * C::CL);
        }
        mbar_init(drain, 1);
        mbar_init_fence();
        prefetch_tensormap(&tmA);
        prefetch_tensormap(&tmB);
    }
    if (warp == 1) PAIR ? tmem_alloc_pair(tmem_slot, C::TMEM_COLS) : tmem_alloc(tmem_slot, C::TMEM_COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (PAIR) cluster_sync();  // the pair's barriers are initialised
    const uint32_t tmem = *tmem_slot;
    pdl_enter();

    const int rank = PAIR ? int(cluster_rank()) : 0;
    const int first = int(blockIdx.x) / C::CL, step = int(gridDim.x) / C::CL;
    const int tiles = p.MTL * p.NTL, items = tiles * p.KS;
    auto tile_m = [&](int it) { return int64_t(it % tiles / p.NTL) * C::MT + rank * 128; };  // this CTA's rows
    auto tile_n = [&](int it) { return (it % tiles % p.NTL) * NT; };
    auto chunk0 = [&](int it) { return it / tiles * p.KC / p.KS; };  // an item's chunks of the reduction
    auto chunk1 = [&](int it) { return (it / tiles + 1) * p.KC / p.KS; };

    if (warp == 0) {
        // ---------------- copies ----------------
        int stage = 0, fills = 0;
        uint32_t phase = 0;
        bool ok = true, at_start = true;  // (the failure-path test withholds a CTA's first stage)
        for (int it = first; it < items && ok; it += step) {
            const int m0 = int(tile_m(it)), n0 = tile_n(it) + rank * C::BROWS, k1 = chunk1(it);
            for (int kc = chunk0(it); kc < k1; ++kc) {
                ok = mbar_wait_warp(&empty[stage], phase ^ 1, p.limit);
                if (!ok) {
                    if (lane == 0) set_status(p.status, LMOE_ERR_TIMEOUT);
                    break;
                }
                if (elect_one() && !(p.stall && at_start)) {
                    uint8_t *sa = stages + stage * C::STAGE, *sb = sa + A_TILE;
                    // the barrier of this stage: a pair's is the leader's, which announces both CTAs' bytes
                    const uint32_t bar = PAIR ? cluster_map(smem_u32(&full[stage]), 0) : 0;
                    const uint64_t policy = l2_policy_evict_normal();
                    if (rank == 0) mbar_arrive_expect_tx(&full[stage], C::STAGE * C::CL);
                    auto load = [&](void *dst, const CUtensorMap *tm, int x, int y) {
                        PAIR ? tma_load_2d_pair(dst, tm, x, y, bar, policy) : tma_load_2d_hint(dst, tm, x, y, &full[stage], policy);
                    };
                    if (A_MN) {
                        load(sa, &tmA, m0, kc * 64);
                        load(sa + 8192, &tmA, m0 + 64, kc * 64);
                    } else {
                        load(sa, &tmA, kc * 64, m0);
                    }
                    if (B_MN) {
#pragma unroll
                        for (int b = 0; b < C::BROWS / 64; ++b) load(sb + b * 8192, &tmB, n0 + 64 * b, kc * 64);
                    } else {
                        load(sb, &tmB, kc * 64, n0);
                    }
                }
                __syncwarp();
                at_start = false;
                ++fills;
                if (++stage == S) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
        // Copies still in flight after a timeout land before the CTA ends (bounded; a
        // pair's all count in on the leader's barriers).
        if (!ok && rank == 0)
            for (int f = fills > S ? fills - S : 0; f < fills; ++f) mbar_wait_warp(&full[f % S], (f / S) & 1, p.limit);
    } else if (warp == 1 && rank == 0) {
        // ---------------- MMA issuer (a pair's: the leader's) ----------------
        int stage = 0, acc = 0;
        uint32_t phase = 0, acc_phase = 0;
        bool ok = true;
        const uint32_t id = (PAIR ? idesc_bf16_pair(NT) : idesc_bf16(NT)) | (A_MN ? IDESC_A_MN : 0) | (B_MN ? IDESC_B_MN : 0);
        constexpr uint32_t a_step = A_MN ? 128 : 2, b_step = B_MN ? 128 : 2;  // 16 of the reduction, in 16-byte units
        for (int it = first; it < items && ok; it += step) {
            ok = mbar_wait_warp(&acc_empty[acc], acc_phase ^ 1, p.limit);
            tc_fence_after();
            const uint32_t d = tmem + uint32_t(acc * NT);
            const int k0 = chunk0(it), k1 = chunk1(it);
            for (int kc = k0; kc < k1 && ok; ++kc) {
                ok = mbar_wait_warp(&full[stage], phase, p.limit);
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t sa = smem_u32(stages + stage * C::STAGE), sb = sa + A_TILE;
                    const uint64_t ad = A_MN ? sdesc_mn128(sa, 8192) : sdesc_k128(sa);
                    const uint64_t bd = B_MN ? sdesc_mn128(sb, 8192) : sdesc_k128(sb);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        if (PAIR)
                            mma_bf16_pair(d, ad + a_step * kk, bd + b_step * kk, id, (kc > k0 || kk > 0) ? 1u : 0u);
                        else
                            mma_bf16(d, ad + a_step * kk, bd + b_step * kk, id, (kc > k0 || kk > 0) ? 1u : 0u);
                    PAIR ? tc_commit_pair(&empty[stage]) : tc_commit(&empty[stage]);
                }
                __syncwarp();
                if (++stage == S) {
                    stage = 0;
                    phase ^= 1;
                }
            }
            if (!ok) break;
            if (elect_one()) PAIR ? tc_commit_pair(&acc_full[acc]) : tc_commit(&acc_full[acc]);
            __syncwarp();
            if (++acc == C::ACC) {
                acc = 0;
                acc_phase ^= 1;
            }
        }
        if (!ok) {
            if (elect_one()) {
                set_status(p.status, LMOE_ERR_TIMEOUT);
                PAIR ? tc_commit_pair(drain) : tc_commit(drain);  // MMAs in flight end before the tensor memory is freed
                mbar_wait(drain, 0, p.limit);
            }
            __syncwarp();
        }
    } else if (warp >= 2) {
        // ---------------- epilogue ----------------
        __shared__ __align__(16) float s_bias[C::EW][32];
        const int q = warp & 3, half = (warp - 2) >> 2;
        int acc = 0;
        uint32_t acc_phase = 0;
        for (int it = first; it < items; it += step) {
            const int64_t m = tile_m(it) + 32 * q + lane;
            const int n0 = tile_n(it), limit = min(NT, p.N - n0);
            const bool mine = m < p.M;
            const int64_t row = (it / tiles * p.M + m) * p.N + n0;  // (parts: fp32 rows one after another)
            const uint32_t tb = tmem + (uint32_t(32 * q) << 16) + uint32_t(acc * NT);
            // what 32 columns need from memory, on its way a turn ahead: the residual, a column's bias a lane
            uint32_t r[32];
            float bias = 0.f;
            auto fetch = [&](int c) {
                if (c >= limit) return;
                if (p.res && mine) {
                    if (p.res_f32) row_load<true>(r, p.res, row + c, min(32, limit - c), p.vec);
                    else row_load<false>(r, p.res, row + c, min(32, limit - c), p.vec);
                }
                if (p.bias && c + lane < limit)
                    bias = p.bias_f32 ? __ldg(static_cast<const float *>(p.bias) + n0 + c + lane)
                                      : bf16_bits_to_f32(__ldg(static_cast<const uint16_t *>(p.bias) + n0 + c + lane));
            };
            fetch(32 * half);
            if (!mbar_wait_warp(&acc_full[acc], acc_phase, p.limit)) {
                if (lane == 0) set_status(p.status, LMOE_ERR_TIMEOUT);
                break;
            }
            tc_fence_after();
            for (int c = 32 * half; c < limit; c += 8 * C::EW) {
                uint32_t v[32];
                tmem_ld_cols<32>(tb + c, v);
                const int cols = min(32, limit - c);
                F2 y[16];
                if (p.bias) {
                    s_bias[warp - 2][lane] = bias;
                    __syncwarp();
                }
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 16; ++j) y[j] = f2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
                if (p.bias) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float4 b = *reinterpret_cast<const float4 *>(&s_bias[warp - 2][4 * j]);
                        y[2 * j] = y[2 * j] + f2(b.x, b.y);
                        y[2 * j + 1] = y[2 * j + 1] + f2(b.z, b.w);
                    }
                    __syncwarp();
                }
                if (p.pre && mine) row_store<false>(y, p.pre, row + c, cols, p.vec);
                apply_fn(p.fn, y);
                if (p.res) {
                    if (p.res_f32) row_add<true>(r, y);
                    else row_add<false>(r, y);
                }
                fetch(c + 8 * C::EW);
                if (mine) {
                    if (p.out_f32) row_store<true>(y, p.out, row + c, cols, p.vec);
                    else row_store<false>(y, p.out, row + c, cols, p.vec);
                }
                __syncwarp();
            }
            tc_fence_before();
            PAIR ? cluster_arrive_read(cluster_map(smem_u32(&acc_empty[acc]), 0)) : mbar_arrive(&acc_empty[acc]);
            if (++acc == C::ACC) {
                acc = 0;
                acc_phase ^= 1;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    // nobody's shared or tensor memory goes while the pair's other CTA may still write or read it
    if (PAIR) cluster_sync_end();
    tc_fence_after();
    if (warp == 1) PAIR ? tmem_dealloc_pair(tmem, C::TMEM_COLS) : tmem_dealloc(tmem, C::TMEM_COLS);
}

// An operand: [rows][cols] bf16, rows `stride` elements apart.
struct Operand {
    const uint16_t *p;
    int64_t rows, cols, stride;
};

template <int NT, bool PAIR, bool A_MN, bool B_MN>
cudaError_t launch(const Operand &A, const Operand &B, LArgs g, cudaStream_t st)
{
    using C = LCfg<NT, PAIR>;
    CUtensorMap ma, mb;
    if (!make_tensor_map(&ma, A.p, MapType::BF16, A.cols, A.rows, A_MN ? 64 : 128, A.stride) ||
        !make_tensor_map(&mb, B.p, MapType::BF16, B.cols, B.rows, B_MN ? 64 : C::BROWS, B.stride))
        return cudaErrorInvalidValue;
    g.MTL = int(ceil_div(g.M, C::MT));
    g.NTL = int(ceil_div(g.N, NT));
    const int64_t items = int64_t(g.MTL) * g.NTL * g.KS;
    const size_t smem = 1024 + size_t(C::S) * C::STAGE + (2 * C::S + 2 * C::ACC + 1) * 8 + 8;
    auto *kern = k_linear_act<NT, PAIR, A_MN, B_MN>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e != cudaSuccess) return e;
    const int64_t slots = device_sms() / C::CL;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned((items < slots ? items : slots) * C::CL));
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = C::CL;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = PAIR ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, ma, mb, g);
}

// Vectors of 32 or 16 bytes where every row of every tensor starts on one.
int vector_bytes(const LArgs &g)
{
    auto fits = [&](const void *p, int bytes, int v) {
        return !p || (reinterpret_cast<uintptr_t>(p) % v == 0 && int64_t(g.N) * bytes % v == 0);
    };
    for (int v : {32, 16})
        if (fits(g.out, g.out_f32 ? 4 : 2, v) && fits(g.pre, 2, v) && fits(g.res, g.res_f32 ? 4 : 2, v)) return v;
    return 0;
}

// ---- parts of the reduction ------------------------------------------------------------------

// The parts' sums added in order, then the epilogue.  W columns a thread (8: rows of all
// tensors start on 16 bytes).
template <int W>
__global__ void __launch_bounds__(256) k_split_sum(const float *part, const LArgs p)
{
    const int64_t per_row = (p.N + W - 1) / W, i = int64_t(blockIdx.x) * 256 + threadIdx.x;
    pdl_enter();
    if (i >= p.M * per_row) return;
    const int64_t m = i / per_row, at = m * p.N + (i - m * per_row) * W;
    const int n = int(i - m * per_row) * W;
    float y[W] = {};
    for (int k = 0; k < p.KS; ++k) {
        const float *s = part + int64_t(k) * p.M * p.N + at;
        if constexpr (W == 8) {
            Pack<float, 8> q;
            q.load(s);
            float v[8];
            q.get(v);
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] += v[j];
        } else {
            y[0] += *s;
        }
    }
    if (p.bias)
#pragma unroll
        for (int j = 0; j < W; ++j)
            y[j] += p.bias_f32 ? __ldg(static_cast<const float *>(p.bias) + n + j)
                               : bf16_bits_to_f32(__ldg(static_cast<const uint16_t *>(p.bias) + n + j));
    auto put = [&](void *base, bool f32) {
        if constexpr (W == 8) {
            if (f32) {
                Pack<float, 8> q;
                q.set(y);
                q.store(static_cast<float *>(base) + at);
            } else {
                Pack<uint16_t, 8> q;
                q.set(y);
                q.store(static_cast<uint16_t *>(base) + at);
            }
        } else {
            if (f32) static_cast<float *>(base)[at] = y[0];
            else static_cast<__nv_bfloat16 *>(base)[at] = __float2bfloat16_rn(y[0]);
        }
    };
    if (p.pre) put(p.pre, false);
    F2 z[(W + 1) / 2];
#pragma unroll
    for (int j = 0; j < W; j += 2) z[j / 2] = f2(y[j], W > 1 ? y[(j + 1) % W] : 0.f);
    apply_fn(p.fn, z);
#pragma unroll
    for (int j = 0; j < W; j += 2) {
        float other;
        f2_get(z[j / 2], y[j], W > 1 ? y[(j + 1) % W] : other);
    }
    if (p.res) {
        float v[W];
        if constexpr (W == 8) {
            if (p.res_f32) {
                Pack<float, 8> q;
                q.load(static_cast<const float *>(p.res) + at);
                q.get(v);
            } else {
                Pack<uint16_t, 8> q;
                q.load(static_cast<const uint16_t *>(p.res) + at);
                q.get(v);
            }
        } else {
            v[0] = p.res_f32 ? static_cast<const float *>(p.res)[at] : bf16_bits_to_f32(static_cast<const uint16_t *>(p.res)[at]);
        }
#pragma unroll
        for (int j = 0; j < W; ++j) y[j] += v[j];
    }
    put(p.out, p.out_f32);
}

// ---- the choice of tiles and parts -----------------------------------------------------------

// Tiles: rows x columns, CTAs, a chunk's bytes a CTA and its time in ns where it has the
// copies it asks for.
struct Tile {
    int M, N, ctas, bytes, chunk;
};
constexpr Tile TILES[4] = {
    {256, 256, 2, 32768, 295}, {256, 128, 2, 24576, 175}, {128, 128, 1, 32768, 213}, {128, 64, 1, 24576, 190}};

struct Plan {
    int tile, KS;
};

// The tile and the number of parts of the reduction with the least time by this model: whole
// waves of items, a chunk's time or that of its bytes at the 14 TB/s that all SMs' copies
// together get out of L2, and for parts the second kernel and its traffic.  Measured, us:
//                          256x256  256x128  128x128  128x64   256x128, 2 parts   128x128, 2 / 3 / 4 parts
//   512 rows 7168 -> 3584    39.1     28.1     34.2     54.2        -                 -
//   200 rows 7168 -> 3584    38.5     24.7     28.8     29.8       20.5              23.2
//   128 rows 7168 -> 3584    38.5     24.6     28.9     26.5       23.1              20.1 / 18.1 / 18.0
//   600 rows 7168 -> 1024    38.4     24.4     28.4     26.8       19.5              20.4 / 18.8 / -
//   331 rows 1056 -> 1000    14.1      9.6      9.9      9.2        8.2               8.4 / 8.2 / 8.7
//   300 rows  512 -> 512     10.5      6.9      7.1      5.9        7.2               7.2
//   1000 rows 1024 -> 2048   13.0      9.2      9.9     12.0        -                 -
Plan plan(int64_t M, int64_t N, int64_t K)
{
    const int64_t KC = ceil_div(K, 64);
    const int sms = device_sms();
    Plan best{0, 1};
    double least = 1e30;
    for (int t = 0; t < 4; ++t) {
        const Tile &T = TILES[t];
        const int64_t tiles = ceil_div(M, T.M) * ceil_div(N, T.N), slots = sms / T.ctas;
        for (int ks = 1; ks <= MAX_PARTS; ++ks) {
            if (ks > 1 && (tiles * ks > slots || KC < 4 * ks)) break;
            const int64_t items = tiles * ks, busy = items < slots ? items : slots;
            const double from_l2 = double(busy * T.ctas) * T.bytes / 14000;
            double ns = double(ceil_div(items, slots) * ceil_div(KC, ks)) * (from_l2 > T.chunk ? from_l2 : T.chunk);
            if (ks > 1) ns += 1000 + double(ks) * double(M) * double(N) * 8 / 5000;
            if (ns < least) {
                least = ns;
                best = {t, ks};
            }
        }
    }
    return best;
}

// Bytes of the parts.
size_t part_bytes(int64_t M, int64_t N, int64_t K)
{
    const Plan pl = plan(M, N, K);
    return pl.KS > 1 ? size_t(round_up(pl.KS * M * N * 4, 256)) : 0;
}

template <bool A_MN, bool B_MN>
cudaError_t product(const Operand &A, const Operand &B, LArgs g, int64_t K, const WaitArgs &wait, void *parts, cudaStream_t st)
{
    const Plan pl = plan(g.M, g.N, K);
    g.KC = int(ceil_div(K, 64));
    g.KS = pl.KS;
    g.vec = vector_bytes(g);
    g.limit = wait.limit > 0 ? wait.limit : 4000000000LL;  // about 2 s of SM clocks
    g.stall = wait.stall_first_fill;
    LArgs h = g;
    if (pl.KS > 1) {
        h.bias = h.res = nullptr;
        h.pre = nullptr;
        h.fn = LMOE_FN_NONE;
        h.out = parts;
        h.out_f32 = 1;
        h.vec = vector_bytes(h);
    }
    cudaError_t e;
    switch (pl.tile) {
    case 0: e = launch<256, true, A_MN, B_MN>(A, B, h, st); break;
    case 1: e = launch<128, true, A_MN, B_MN>(A, B, h, st); break;
    case 2: e = launch<128, false, A_MN, B_MN>(A, B, h, st); break;
    default: e = launch<64, false, A_MN, B_MN>(A, B, h, st); break;
    }
    if (e != cudaSuccess || pl.KS == 1) return e;
    const bool wide = g.vec && g.N % 8 == 0;
    const dim3 grid(unsigned(ceil_div(g.M * ceil_div(g.N, wide ? 8 : 1), 256)));
    const float *part = static_cast<const float *>(parts);
    return wide ? launch_pdl(k_split_sum<8>, grid, dim3(256), 0, st, part, g) : launch_pdl(k_split_sum<1>, grid, dim3(256), 0, st, part, g);
}

// ---- dz and its column sums ----------------------------------------------------------------

struct DzArgs {
    const void *dout;
    const uint16_t *pre;
    int64_t rows;
    int N, Np;       // dz's rows are Np elements apart, the columns beyond N zero
    uint16_t *dz;    // null: only the column sums
    float *part;     // [gridDim.y][N], or null
};

// A block takes 256 columns and every gridDim.y-th group of eight rows, a warp a row
// of it, a lane eight columns.  VEC: rows start on 16 bytes.
template <bool F32, int FN, bool VEC>
__global__ void __launch_bounds__(256, 4) k_act_back(const DzArgs p)
{
    __shared__ float s_cols[8][256 + 8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = (int(blockIdx.x) * 32 + lane) * 8;
    float sum[8] = {};
    pdl_enter();
    const int64_t step = int64_t(gridDim.y) * 8;
    if (c < p.Np)
        for (int64_t t0 = int64_t(blockIdx.y) * 8 + warp; t0 < p.rows; t0 += 4 * step) {
            // four rows' loads at once: one row at a time left the loads' latency open (4096 x 7168,
            // silu, sums alone: 36 us)
            Pack<float, 8> df[F32 && VEC ? 4 : 1];
            Pack<uint16_t, 8> dh[!F32 && VEC ? 4 : 1], zh[FN != LMOE_FN_NONE && VEC ? 4 : 1];
            if constexpr (VEC) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int64_t at = min(t0 + i * step, p.rows - 1) * p.N + c;
                    if constexpr (F32) df[i].load(static_cast<const float *>(p.dout) + at);
                    else dh[i].load(static_cast<const uint16_t *>(p.dout) + at);
                    if constexpr (FN != LMOE_FN_NONE) zh[i].load(p.pre + at);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t t = t0 + i * step, at = t * p.N + c;
                if (t >= p.rows) break;
                float d[8], z[8] = {};
                if constexpr (VEC) {
                    if constexpr (F32) df[i].get(d);
                    else dh[i].get(d);
                    if constexpr (FN != LMOE_FN_NONE) zh[i].get(z);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const bool in = c + j < p.N;
                        d[j] = !in ? 0.f : F32 ? static_cast<const float *>(p.dout)[at + j] : bf16_bits_to_f32(static_cast<const uint16_t *>(p.dout)[at + j]);
                        if (FN != LMOE_FN_NONE && in) z[j] = bf16_bits_to_f32(p.pre[at + j]);
                    }
                }
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    if (FN != LMOE_FN_NONE) f2_get(f2(d[j], d[j + 1]) * slope<FN>(f2(z[j], z[j + 1])), d[j], d[j + 1]);
                    sum[j] += d[j];
                    sum[j + 1] += d[j + 1];
                }
                if (p.dz) {
                    Pack<uint16_t, 8> q;
                    q.set(d);
                    q.store(p.dz + t * p.Np + c);
                }
            }
        }
    if (!p.part) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) s_cols[warp][lane * 8 + j] = sum[j];
    __syncthreads();
    const int col = int(blockIdx.x) * 256 + threadIdx.x;
    if (col >= p.N) return;
    float v = 0.f;
#pragma unroll
    for (int q = 0; q < 8; ++q) v += s_cols[q][threadIdx.x];
    p.part[int64_t(blockIdx.y) * p.N + col] = v;
}

// Groups of rows of k_act_back: as many blocks as fit at once, four an SM, and eight rows a
// block at least.
int64_t dz_splits(int64_t rows, int N)
{
    const int64_t strips = ceil_div(N, 256), want = strips < 152 * 4 ? 152 * 4 / strips : 1, most = ceil_div(rows, 8);
    return want < most ? want : most;
}

template <bool F32, bool VEC>
cudaError_t dz_fn(const DzArgs &g, int fn, dim3 grid, cudaStream_t st)
{
    switch (fn) {
    case LMOE_FN_NONE: return launch_pdl(k_act_back<F32, LMOE_FN_NONE, VEC>, grid, dim3(256), 0, st, g);
    case LMOE_FN_RELU: return launch_pdl(k_act_back<F32, LMOE_FN_RELU, VEC>, grid, dim3(256), 0, st, g);
    case LMOE_FN_SILU: return launch_pdl(k_act_back<F32, LMOE_FN_SILU, VEC>, grid, dim3(256), 0, st, g);
    case LMOE_FN_GELU: return launch_pdl(k_act_back<F32, LMOE_FN_GELU, VEC>, grid, dim3(256), 0, st, g);
    default: return launch_pdl(k_act_back<F32, LMOE_FN_GELU_TANH, VEC>, grid, dim3(256), 0, st, g);
    }
}

}  // namespace

// Up to this many rows the weights' stream is the bound (k_linear_few.cu); at 96 and 128
// it took 23.4 and 21.1 us (3584 -> 7168, 7168 -> 3584) against 18.0 and 18.0 here.
constexpr int64_t FEW = 64;

size_t linear_act_scratch_bytes(int64_t rows, int K, int N) { return rows <= FEW ? 0 : part_bytes(rows, N, K); }

cudaError_t launch_linear_act(const LinearActArgs &a, void *scratch, cudaStream_t st)
{
    if (a.rows <= FEW) return launch_linear_few(a, st);
    LArgs g{};
    g.M = a.rows;
    g.N = a.N;
    g.bias = a.bias;
    g.bias_f32 = a.bias_fmt == LMOE_F32;
    g.res = a.res;
    g.res_f32 = a.res_fmt == LMOE_F32;
    g.out_f32 = a.out_fmt == LMOE_F32;
    g.fn = a.fn;
    g.out = a.out;
    g.pre = a.pre;
    g.status = a.status;
    return product<false, false>({a.x, a.rows, a.K, a.K}, {a.W, a.N, a.K, a.K}, g, a.K, a.wait, scratch, st);
}

// dz [rows][Np] bf16 | column sums | parts of a product's reduction
size_t linear_act_back_scratch_bytes(int64_t rows, int K, int N)
{
    if (rows == 0) return 0;
    const int64_t Np = round_up(N, 8);
    const size_t dx = part_bytes(rows, K, N), dW = part_bytes(N, K, rows);
    return size_t(round_up(rows * Np * 2, 256)) + size_t(round_up(dz_splits(rows, N) * N * 4, 256)) + (dx > dW ? dx : dW);
}

cudaError_t launch_linear_act_back(const LinearActBackArgs &a, void *scratch, cudaStream_t st)
{
    cudaError_t e = cudaSuccess;
    if (a.rows == 0) {
        if (a.dW) e = cudaMemsetAsync(a.dW, 0, size_t(a.N) * a.K * (a.dW_fmt == LMOE_F32 ? 4 : 2), st);
        if (a.dbias && e == cudaSuccess) e = cudaMemsetAsync(a.dbias, 0, size_t(a.N) * 4, st);
        return e;
    }
    const int64_t Np = round_up(a.N, 8);
    uint16_t *dz = static_cast<uint16_t *>(scratch);
    float *part = reinterpret_cast<float *>(static_cast<char *>(scratch) + round_up(a.rows * Np * 2, 256));
    void *parts = reinterpret_cast<char *>(part) + round_up(dz_splits(a.rows, a.N) * a.N * 4, 256);
    // bf16 gradients that go through no function are the operand as they are
    const bool as_is = a.fn == LMOE_FN_NONE && a.dout_fmt == LMOE_BF16 && Np == a.N;
    const bool need_dz = (a.dx || a.dW) && !as_is;
    if (need_dz || a.dbias) {
        const DzArgs g{a.dout, a.pre, a.rows, a.N, int(Np), need_dz ? dz : nullptr, a.dbias ? part : nullptr};
        const dim3 grid(unsigned(ceil_div(Np, 256)), unsigned(dz_splits(a.rows, a.N)));
        const bool f32 = a.dout_fmt == LMOE_F32, vec = Np == a.N;
        e = f32 ? (vec ? dz_fn<true, true>(g, a.fn, grid, st) : dz_fn<true, false>(g, a.fn, grid, st))
                : (vec ? dz_fn<false, true>(g, a.fn, grid, st) : dz_fn<false, false>(g, a.fn, grid, st));
        if (e == cudaSuccess && a.dbias) e = launch_col_sums(part, grid.y, a.N, 1, a.dbias, nullptr, st);
        if (e != cudaSuccess) return e;
    }
    const Operand d{as_is ? static_cast<const uint16_t *>(a.dout) : dz, a.rows, a.N, Np};
    LArgs g{};
    g.status = a.status;
    if (a.dx) {
        g.M = a.rows;
        g.N = a.K;
        g.out = a.dx;
        e = product<false, true>(d, {a.W, a.N, a.K, a.K}, g, a.N, a.wait, parts, st);
        if (e != cudaSuccess) return e;
    }
    if (a.dW) {
        g.M = a.N;
        g.N = a.K;
        g.out = a.dW;
        g.out_f32 = a.dW_fmt == LMOE_F32;
        e = product<true, true>(d, {a.x, a.rows, a.K, a.K}, g, a.rows, a.wait, parts, st);
    }
    return e;
}

}  // namespace lmoe
