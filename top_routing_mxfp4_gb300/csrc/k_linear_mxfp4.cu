// MXFP4 linear on bf16 rows: out[r][n] = bf16( sum_c x[r][c] * W[n][c] ), on
// the block-scaled tensor cores (tcgen05.mma kind::mxf8f6f4, weights e2m1 with
// their E8M0 scales as stored, fp32 accumulation in TMEM).
//
// The weights need no unpacking: the packed-FP4 tensor map feeds them to the
// tensor core as they lie in memory.  The other operand of that instruction
// has 8-bit elements, so a bf16 row (8 significant bits) enters as two e4m3
// rows (4 significant bits each), x = 2^a hi + 2^(a-5) lo, with one a per 32
// columns:  a = floor(log2 amax) - 7, so |x / 2^a| < 256;
//   hi = e4m3(x / 2^a), lo = e4m3(32 (x / 2^a - hi)).
// The residual x / 2^a - hi is at most half a step of hi, at most 8 (so 32
// times it is at most 256 and neither part saturates), and a multiple of x's
// own last bit, 2^-7 of its binade: at most 4 significant bits, hence exact,
// down to elements of 2^-14 of the block's largest; below, lo rounds at 2^-14
// of 2^a, an error of at most 2^-15 2^a <= 2^-22 amax.  Both parts' products
// go into one fp32 accumulator.
//
// Bounded by the weight stream (17/32 byte a weight) up to about a hundred
// rows, then by the tensor cores at half their 8-bit rate (two parts).
//
// k_split_rows writes the two parts and their scale atoms; k_linear_mx is a
// persistent kernel over items (weight tile of 128, row tile of NB), its warps:
// 0 weight tiles and their scale atoms (TMA), 1 MMA issuer, 2-5 epilogue, 6
// the rows' two parts, 7 their scale atoms.  With few items a cluster of KS
// CTAs shares an item along K: ranks 1.. store their accumulators into rank
// 0's shared memory, which adds them in rank order.
// Every wait is bounded (LMOE_ERR_TIMEOUT in the status word).
#include <cuda.h>
#include <cuda_bf16.h>

#include "lmoe_internal.cuh"
#include "tc_ptx.cuh"

namespace lmoe {
namespace {

using namespace tc;

// ---- bf16 rows as two e4m3 rows ----------------------------------------------------------

// A block's scale byte of the hi part (a + 127; lo's is 5 less) from the
// largest magnitude's bits.  a >= -122 keeps lo's byte in range; bf16's
// smallest step, 2^-133, is then still a multiple of lo's, 2^-127 2^-9.
__device__ __forceinline__ int split_byte(uint32_t amax_bits)
{
    const int ex = int(amax_bits >> 23);
    const int b = ex - 7;  // floor(log2 amax) - 7 + 127 (a subnormal's exponent is below the clamp)
    return b < 5 ? 5 : b;
}

// Eight elements of a block with scale byte b: hi and lo codes.  An infinity
// becomes a NaN: e4m3 has none.
__device__ __forceinline__ void split8(const uint32_t (&w)[4], int b, uint2 &hi, uint2 &lo)
{
    const float inv = __uint_as_float(uint32_t(254 - b) << 23);  // 2^(127 - b), b in [5, 248]
    uint32_t h[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float v0 = __uint_as_float(w[i] << 16) * inv, v1 = __uint_as_float(w[i] & 0xFFFF0000u) * inv;
        if ((w[i] & 0x7FFFu) == 0x7F80u) v0 = __uint_as_float(0x7FFFFFFFu);
        if ((w[i] & 0x7FFF0000u) == 0x7F800000u) v1 = __uint_as_float(0x7FFFFFFFu);
        h[i] = e4m3x2(v0, v1);
        uint32_t d;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(uint16_t(h[i])));
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&d));
        l[i] = e4m3x2((v0 - f.x) * 32.f, (v1 - f.y) * 32.f);
    }
    hi = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
    lo = make_uint2(l[0] | (l[1] << 16), l[2] | (l[3] << 16));
}

__device__ __forceinline__ uint32_t amax8(const uint32_t (&w)[4])
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m = max(m, (w[i] & 0x7FFFu) << 16);
        m = max(m, w[i] & 0x7FFF0000u);
    }
    return m;
}

// x[rows][K] -> codes [2][rows][Kp] (hi, lo), scale atoms [2][tiles][KC][512];
// eight columns a thread, four threads a block of 32.
template <int NB>
__global__ void __launch_bounds__(256) k_split_rows(const uint16_t *__restrict__ x, int64_t rows, int K, int KC,
                                                    uint8_t *__restrict__ codes, uint8_t *__restrict__ atoms)
{
    pdl_enter();
    const int per = KC * 16;  // threads a row
    const int64_t n = rows * per;
    const int64_t atom_bytes = ceil_div(rows, NB) * KC * 512;
    // whole warps: four lanes share a block
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < round_up(n, 32); i += int64_t(gridDim.x) * 256) {
        const int64_t r = i / per;
        const int c = int(i - r * per) * 8;
        uint4 u = make_uint4(0, 0, 0, 0);
        if (i < n && c < K) u = *reinterpret_cast<const uint4 *>(x + r * K + c);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
        uint32_t m = amax8(w);
        m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
        if (i >= n) continue;
        const int b = split_byte(m);
        uint2 hi, lo;
        split8(w, b, hi, lo);
        uint8_t *row = codes + r * (KC * 128) + c;
        *reinterpret_cast<uint2 *>(row) = hi;
        *reinterpret_cast<uint2 *>(row + rows * (KC * 128)) = lo;
        if ((c & 31) == 0) {
            const int64_t o = tile_atom_off(r, c >> 5, KC, NB);
            atoms[o] = uint8_t(b);
            atoms[atom_bytes + o] = uint8_t(b - 5);
        }
    }
}

// ---- the product ---------------------------------------------------------------------------

constexpr int THREADS = 256;
constexpr uint32_t A_TILE = 128 * 128;  // 128 weight rows x 128 columns, one byte each once expanded

template <int NB, int KS>
struct LCfg {
    static constexpr uint32_t B_TILE = NB * 128;  // one part
    static constexpr uint32_t SF_OFF = A_TILE + 2 * B_TILE;  // scale atoms: weights, hi, lo
    static constexpr uint32_t STAGE = (SF_OFF + 3 * 512 + 1023) / 1024 * 1024;
    static constexpr uint32_t RED = (KS - 1) * 128 * NB * 4;
    static constexpr int S_RAW = int((210 * 1024 - RED) / STAGE);
    static constexpr int S = S_RAW > 12 ? 12 : S_RAW;
    static constexpr int ACC = 2;
    static constexpr int SF_COLS = 12;  // TMEM columns of a stage's scales
    static constexpr int SF_BASE = ACC * NB;
    static constexpr int COLS = SF_BASE + S * SF_COLS;
    static constexpr uint32_t TMEM_COLS = COLS <= 64 ? 64 : COLS <= 128 ? 128 : COLS <= 256 ? 256 : 512;
    static_assert(COLS <= 512 && S >= 2, "pipeline");
};

struct LArgs {
    const uint8_t *sfa, *sfb;  // weight scale atoms [MT][KC][512], row scale atoms [2][NT][KC][512]
    int64_t sfb_lo;            // bytes from the hi atoms to the lo ones
    int rows, N, MT, NTL, KC;
    uint16_t *out;
    int32_t *status;
    long long limit;
    int stall;
};

template <int NB, int KS>
__global__ void __launch_bounds__(THREADS, 1)
    k_linear_mx(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, const LArgs p)
{
    using C = LCfg<NB, KS>;
    constexpr int S = C::S;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *stages = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float *red = reinterpret_cast<float *>(stages + S * C::STAGE);  // [KS - 1][NB][128]
    uint64_t *full = reinterpret_cast<uint64_t *>(red + (KS - 1) * 128 * NB);
    uint64_t *empty = full + S;
    uint64_t *acc_full = empty + S;
    uint64_t *acc_empty = acc_full + C::ACC;
    uint64_t *drain = acc_empty + C::ACC;
    uint64_t *red_full = drain + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(red_full + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = KS > 1 ? int(cluster_rank()) : 0;
    const int first = int(blockIdx.x) / KS, step = int(gridDim.x) / KS;
    const int total = p.MT * p.NTL;
    const int k0 = rank * p.KC / KS, k1 = (rank + 1) * p.KC / KS;  // this rank's chunks of 128 columns
    if (warp == 0 && lane == 0) {
        prefetch_tensormap(&tmA);
        // the first weight tiles on their way to L2 while the previous kernel ends
        for (int kc = k0; kc < k1 && kc < k0 + S; ++kc) tma_prefetch_2d(&tmA, kc * 128, first % p.MT * 128);
    }
    if (warp == 6 && lane == 0) prefetch_tensormap(&tmB);
    if (threadIdx.x == 64) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 3);  // the three producer warps
            mbar_init(&empty[s], 1);
        }
        for (int a = 0; a < C::ACC; ++a) {
            mbar_init(&acc_full[a], 1);
            mbar_init(&acc_empty[a], 128);
        }
        mbar_init(drain, 1);
        mbar_init(red_full, KS > 1 ? (KS - 1) * 128 : 1);
        mbar_init_fence();
    }
    if (warp == 1) tmem_alloc(tmem_slot, C::TMEM_COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (KS > 1) cluster_sync();  // the cluster's barriers are initialised
    pdl_enter();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0 || warp >= 6) {
        // ---------------- producers ----------------
        int stage = 0, fills = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int it = first; it < total && ok; it += step) {
            const int mt = it % p.MT, nt = it / p.MT;
            for (int kc = k0; kc < k1; ++kc) {
                ok = mbar_wait(&empty[stage], phase ^ 1, p.limit);
                if (!__all_sync(0xFFFFFFFFu, ok)) {
                    if (lane == 0) set_status(p.status, LMOE_ERR_TIMEOUT);
                    ok = false;
                    break;
                }
                uint8_t *sb = stages + stage * C::STAGE;
                if (lane == 0) {
                    if (warp == 0) {
                        if (!(p.stall && it == first && kc == k0)) {
                            mbar_arrive_expect_tx(&full[stage], 128 * 64 + 512);  // packed FP4: 64 bytes a row
                            tma_load_2d(sb, &tmA, kc * 128, mt * 128, &full[stage]);
                            bulk_load(sb + C::SF_OFF, p.sfa + (int64_t(mt) * p.KC + kc) * 512, 512, &full[stage]);
                        }
                    } else if (warp == 6) {
                        mbar_arrive_expect_tx(&full[stage], 2 * C::B_TILE);
                        tma_load_2d(sb + A_TILE, &tmB, kc * 128, nt * NB, &full[stage]);
                        tma_load_2d(sb + A_TILE + C::B_TILE, &tmB, kc * 128, p.rows + nt * NB, &full[stage]);
                    } else {
                        const uint8_t *src = p.sfb + (int64_t(nt) * p.KC + kc) * 512;
                        mbar_arrive_expect_tx(&full[stage], 1024);
                        bulk_load(sb + C::SF_OFF + 512, src, 512, &full[stage]);
                        bulk_load(sb + C::SF_OFF + 1024, src + p.sfb_lo, 512, &full[stage]);
                    }
                }
                __syncwarp();
                ++fills;
                if (++stage == S) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
        if (!ok)  // copies still in flight land before the CTA ends (bounded)
            for (int f = fills > S ? fills - S : 0; f < fills; ++f) mbar_wait(&full[f % S], (f / S) & 1, p.limit);
    } else if (warp == 1) {
        // ---------------- MMA issuer ----------------
        int stage = 0, acc = 0;
        uint32_t phase = 0, acc_phase = 0;
        bool ok = true;
        for (int it = first; it < total && ok; it += step) {
            const uint32_t N = uint32_t((min(NB, p.rows - it / p.MT * NB) + 15) & ~15);
            ok = mbar_wait(&acc_empty[acc], acc_phase ^ 1, p.limit);
            tc_fence_after();
            const uint32_t d = tmem + uint32_t(acc * NB);
            for (int kc = k0; kc < k1 && ok; ++kc) {
                ok = mbar_wait(&full[stage], phase, p.limit);
                if (!ok) break;
                tc_fence_after();
                if (lane == 0) {
                    const uint8_t *sb = stages + stage * C::STAGE;
                    const uint32_t sfa = tmem + uint32_t(C::SF_BASE + stage * C::SF_COLS);
#pragma unroll
                    for (int i = 0; i < 3; ++i) tc_cp_sf(sfa + 4 * i, sdesc_sf(smem_u32(sb + C::SF_OFF + 512 * i)));
                    const uint64_t ad = sdesc_k128(smem_u32(sb));
#pragma unroll
                    for (int part = 0; part < 2; ++part) {
                        const uint64_t bd = sdesc_k128(smem_u32(sb + A_TILE + part * C::B_TILE));
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_mxf8f6f4(d, ad + 2 * kk, bd + 2 * kk, idesc_mxf4_e4m3(N, uint32_t(kk)), sfa,
                                         sfa + 4 + 4 * part, (kc > k0 || part > 0 || kk > 0) ? 1u : 0u);
                    }
                    tc_commit(&empty[stage]);
                }
                __syncwarp();
                if (++stage == S) {
                    stage = 0;
                    phase ^= 1;
                }
            }
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            if (lane == 0) tc_commit(&acc_full[acc]);
            __syncwarp();
            if (++acc == C::ACC) {
                acc = 0;
                acc_phase ^= 1;
            }
        }
        if (!ok) {
            if (lane == 0) {
                set_status(p.status, LMOE_ERR_TIMEOUT);
                tc_commit(drain);  // MMAs in flight end before the tensor memory is freed
                mbar_wait(drain, 0, p.limit);
            }
            __syncwarp();
        }
    } else {
        // ---------------- epilogue ----------------
        const int q = warp & 3;
        int acc = 0;
        uint32_t acc_phase = 0;
        for (int it = first; it < total; it += step) {
            const int mt = it % p.MT, row0 = it / p.MT * NB;
            const int nv = min(NB, p.rows - row0);
            const bool ok = mbar_wait(&acc_full[acc], acc_phase, p.limit);
            if (!__all_sync(0xFFFFFFFFu, ok)) {
                if (lane == 0) set_status(p.status, LMOE_ERR_TIMEOUT);
                break;
            }
            tc_fence_after();
            const uint32_t tb = tmem + (uint32_t(32 * q) << 16) + uint32_t(acc * NB);
            if (KS > 1 && rank > 0) {
                const uint32_t dst = cluster_map(smem_u32(red + (rank - 1) * 128 * NB + 32 * q + lane), 0);
                for (int c0 = 0; c0 < nv; c0 += 16) {
                    uint32_t v[16];
                    tmem_ld16(tb + c0, v);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 16; ++j) cluster_store(dst + (c0 + j) * 512, __uint_as_float(v[j]));
                }
                cluster_arrive(cluster_map(smem_u32(red_full), 0));
            } else {
                if (KS > 1) {
                    const bool in = mbar_wait_cluster(red_full, 0, p.limit);
                    if (!__all_sync(0xFFFFFFFFu, in)) {
                        if (lane == 0) set_status(p.status, LMOE_ERR_TIMEOUT);
                        break;
                    }
                }
                const int n = mt * 128 + 32 * q + lane;
                for (int c0 = 0; c0 < nv; c0 += 16) {
                    uint32_t v[16];
                    tmem_ld16(tb + c0, v);
                    tmem_ld_wait();
                    float y[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) y[j] = __uint_as_float(v[j]);
                    if (KS > 1) {
                        const float *part = red + c0 * 128 + 32 * q + lane;
#pragma unroll
                        for (int r = 0; r < KS - 1; ++r)
#pragma unroll
                            for (int j = 0; j < 16; ++j) y[j] += part[(r * NB + j) * 128];
                    }
                    if (n < p.N) {
                        __nv_bfloat16 *o =
                            reinterpret_cast<__nv_bfloat16 *>(p.out) + int64_t(row0 + c0) * p.N + n;
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (c0 + j < nv) o[int64_t(j) * p.N] = __float2bfloat16_rn(y[j]);
                    }
                }
            }
            tc_fence_before();
            mbar_arrive(&acc_empty[acc]);
            if (++acc == C::ACC) {
                acc = 0;
                acc_phase ^= 1;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (KS > 1) cluster_sync();  // nobody's shared memory goes while another rank may store into it
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, C::TMEM_COLS);
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// A map of [rows][K] elements, boxes of 128 columns x box_rows: packed FP4
// (64 bytes per 128 columns in memory, 128 in shared memory) or bytes.
bool byte_map(CUtensorMap *m, const void *base, bool fp4, int64_t K, int64_t rows, int box_rows)
{
    static const EncodeTiledFn fn = [] {
        cudaDriverEntryPointQueryResult q;
        void *f = nullptr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<EncodeTiledFn>(f);
    }();
    if (!fn) return false;
    const cuuint64_t dims[2] = {cuuint64_t(K), cuuint64_t(rows)};
    const cuuint64_t strides[1] = {cuuint64_t(fp4 ? K / 2 : K)};
    const cuuint32_t box[2] = {128, cuuint32_t(box_rows)};
    const cuuint32_t es[2] = {1, 1};
    return fn(m, fp4 ? CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2,
              const_cast<void *>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int sm_count()
{
    int dev = 0, n = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    return n > 0 ? n : 148;
}

int row_tile(int64_t rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128; }

template <int NB, int KS>
cudaError_t launch(const LArgs &a, const uint8_t *q, const uint8_t *codes, int sms, cudaStream_t st)
{
    using C = LCfg<NB, KS>;
    CUtensorMap ma, mb;
    if (!byte_map(&ma, q, true, int64_t(a.KC) * 128, a.N, 128) ||
        !byte_map(&mb, codes, false, int64_t(a.KC) * 128, 2 * int64_t(a.rows), NB))
        return cudaErrorInvalidValue;
    const size_t smem = 1024 + size_t(C::S) * C::STAGE + C::RED + (2 * C::S + 2 * C::ACC + 2) * 8 + 16;
    auto *kern = k_linear_mx<NB, KS>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e != cudaSuccess) return e;
    const int64_t items = int64_t(a.MT) * a.NTL, slots = sms / KS;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned((items < slots ? items : slots) * KS));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = KS;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = KS > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, ma, mb, a);
}

// The most ranks (1, 2, 4 or 8) with which every item still has a cluster of
// its own and every rank at least four chunks.
template <int NB>
cudaError_t pick(const LArgs &a, const uint8_t *q, const uint8_t *codes, int sms, cudaStream_t st)
{
    const int64_t items = int64_t(a.MT) * a.NTL;
    if constexpr (NB <= 32)
        if (items * 8 <= sms && a.KC >= 32) return launch<NB, 8>(a, q, codes, sms, st);
    if constexpr (NB <= 64)
        if (items * 4 <= sms && a.KC >= 16) return launch<NB, 4>(a, q, codes, sms, st);
    if (items * 2 <= sms && a.KC >= 8) return launch<NB, 2>(a, q, codes, sms, st);
    return launch<NB, 1>(a, q, codes, sms, st);
}

}  // namespace

size_t linear_mxfp4_scratch_bytes(int64_t rows, int K, int N)
{
    (void)N;
    const int64_t KC = ceil_div(K, 128), NB = row_tile(rows);
    return size_t(round_up(2 * rows * KC * 128, 256) + 2 * ceil_div(rows, NB) * KC * 512);
}

cudaError_t launch_linear_mxfp4(const uint16_t *x, const uint8_t *q, const uint8_t *s, int64_t rows, int K, int N,
                                uint16_t *out, void *scratch, int32_t *status, const WaitArgs &wait, cudaStream_t st)
{
    const int NB = row_tile(rows);
    LArgs a{};
    a.rows = int(rows);
    a.N = N;
    a.MT = int(ceil_div(N, 128));
    a.NTL = int(ceil_div(rows, NB));
    a.KC = int(ceil_div(K, 128));
    if (int64_t(a.MT) * a.NTL > INT32_MAX) return cudaErrorInvalidValue;
    uint8_t *codes = static_cast<uint8_t *>(scratch);
    uint8_t *atoms = codes + round_up(2 * rows * a.KC * 128, 256);
    a.sfa = s;
    a.sfb = atoms;
    a.sfb_lo = int64_t(a.NTL) * a.KC * 512;
    a.out = out;
    a.status = status;
    a.limit = wait.limit > 0 ? wait.limit : 4000000000LL;  // about 2 s of SM clocks
    a.stall = wait.stall_first_fill;
    const int sms = sm_count();
    const int64_t blocks = ceil_div(rows * a.KC * 16, 256);
    const dim3 grid(unsigned(blocks < int64_t(sms) * 8 ? blocks : int64_t(sms) * 8)), block(256);
    auto *split = NB == 16 ? k_split_rows<16> : NB == 32 ? k_split_rows<32> : NB == 64 ? k_split_rows<64> : k_split_rows<128>;
    const cudaError_t e = launch_pdl(split, grid, block, 0, st, x, rows, K, a.KC, codes, atoms);
    if (e != cudaSuccess) return e;
    switch (NB) {
    case 16: return pick<16>(a, q, codes, sms, st);
    case 32: return pick<32>(a, q, codes, sms, st);
    case 64: return pick<64>(a, q, codes, sms, st);
    default: return pick<128>(a, q, codes, sms, st);
    }
}

}  // namespace lmoe
