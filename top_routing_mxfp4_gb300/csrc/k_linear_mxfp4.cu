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
// of 2^a, an error of at most 2^-15 2^a <= 2^-22 amax.
//
// Bounded by the weight stream (17/32 byte a weight) up to about a hundred
// rows, then by the tensor cores at half their 8-bit rate (two parts).
//
// The two parts of a tile of NB rows are one operand of 2 NB rows, hi above lo,
// with accumulator columns of their own that the epilogue adds: a chunk of 128
// columns is four MMAs.
//
// k_linear_mx is a persistent kernel over items (weight tile of 128, row tile),
// its warps: 0 weight tiles and their scale atoms (TMA), 1 MMA issuer, 2-5
// epilogue, 6.. the rows.  Up to 16 rows, warps 6.. split the rows themselves
// as they go (each weight tile's CTAs repeat it, which costs less than a
// kernel before this one); beyond, k_split_rows has written the parts and warp
// 6 copies them.  With few items a cluster of KS CTAs shares an item along K
// (cluster_sum.cuh).
// Every wait is bounded (LMOE_ERR_TIMEOUT in the status word).
//
// Measured, 7168 -> 3584: 1, 16, 64, 512 and 8192 rows 6.7, 8.4, 10.5, 26.3 and
// 294 us (3.2 us of any dependent kernel's start among them; the last 1.43
// PFLOP/s); 7168 -> 28672: 1 row 20 us (5.4 TB/s), 16 and 64 rows 33 us: there 224
// weight tiles on 152 SMs take two whole tiles' time.
#include <cuda.h>
#include <cuda_bf16.h>

#include "cluster_sum.cuh"
#include "device_cache.h"
#include "lmoe_internal.cuh"
#include "tc_ptx.cuh"
#include "tensor_map.cuh"

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

// Byte of (row r, block b of the chunk) in the row operand's scale atoms, 128 rows an atom.
__device__ __forceinline__ int sf_off(int r, int b)
{
    return (r >> 7) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4 + b;
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

// x[rows][K] -> per tile of NB rows and chunk of 128 columns one block of bytes
// as a pipeline stage holds it: 2 NB rows of 128 codes (hi rows, then lo rows),
// 16-byte units swizzled by the row, and behind them the scale atoms; eight
// columns a thread, four threads a block of 32.
__host__ __device__ constexpr int rows_block(int NB) { return 2 * NB * 128 + (2 * NB + 127) / 128 * 512; }

template <int NB>
__global__ void __launch_bounds__(256) k_split_rows(const uint16_t *__restrict__ x, int64_t rows, int K, int KC,
                                                    uint8_t *__restrict__ blocks)
{
    pdl_enter();
    const int per = KC * 16;  // threads a row
    const int64_t n = rows * per;
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
        const int64_t tile = r / NB;
        const int rr = int(r - tile * NB);
        uint8_t *block = blocks + (tile * KC + (c >> 7)) * rows_block(NB);
        const int at = rr * 128 + ((((c >> 4) & 7) ^ (rr & 7)) << 4) + (c & 8);
        *reinterpret_cast<uint2 *>(block + at) = hi;
        *reinterpret_cast<uint2 *>(block + NB * 128 + at) = lo;  // NB % 8 == 0: the same swizzle
        if ((c & 31) == 0) {
            uint8_t *sf = block + 2 * NB * 128;
            sf[sf_off(rr, (c >> 5) & 3)] = uint8_t(b);
            sf[sf_off(NB + rr, (c >> 5) & 3)] = uint8_t(b - 5);
        }
    }
}

// ---- the product ---------------------------------------------------------------------------

constexpr uint32_t A_TILE = 128 * 128;  // 128 weight rows x 128 columns, one byte each once expanded
constexpr int MAX_KS = 8;

// FUSED: the kernel splits the rows itself.
template <int NB, bool FUSED>
struct LCfg {
    static constexpr int NC = 2 * NB;  // rows of the B operand, columns of an accumulator
    static constexpr int NAT = (NC + 127) / 128;  // its scale atoms a chunk
    static constexpr uint32_t B_TILE = NC * 128;
    static constexpr uint32_t SF_OFF = A_TILE + B_TILE;  // scale atoms: weights, rows
    static constexpr uint32_t STAGE = (SF_OFF + (1 + NAT) * 512 + 1023) / 1024 * 1024;
    // Fused: four teams of two warps take the chunks in turn, a warp half the
    // tile's rows (two rows a step, an 8-column piece a lane).
    static constexpr int TW = FUSED ? 2 : 1;
    static constexpr int TEAMS = FUSED ? 4 : 1;
    static constexpr int BW = TW * TEAMS;  // warps that bring B
    static constexpr int THREADS = 32 * (6 + BW);
    static constexpr int UNITS = FUSED ? NB / 4 : 1;
    // Small row tiles leave room for two CTAs an SM: the next call's start up
    // beside the last ones of this call, and the items spread more evenly.
    static constexpr int CTAS = FUSED ? 2 : 1;
    static constexpr int ACC = NC <= 128 ? 2 : 1;
    static constexpr int SF_COLS = 4 + 4 * NAT;  // TMEM columns of a stage's scales
    static constexpr int SF_BASE = ACC * NC;
    static constexpr uint32_t TAIL = 1024 + (2 * 12 + 2 * ACC + 2) * 8 + 16;
    // 128-row tiles run unsplit, and the room of the exchange is one more stage of
    // the ring (7168 -> 3584, 512 rows: 26.1 us, against 30.0 with a shorter ring).
    static constexpr bool SPLITS = NB < 128;
    static constexpr uint32_t RED = SPLITS ? ClusterSum::red_bytes(NB) : 0;
    static constexpr int S_RAW = int(((227 * 1024) / CTAS - 1024 - TAIL - RED) / STAGE);
    static constexpr int S = S_RAW > 12 ? 12 : S_RAW;
    static constexpr int COLS = SF_BASE + S * SF_COLS;
    static constexpr uint32_t TMEM_COLS = COLS <= 64 ? 64 : COLS <= 128 ? 128 : COLS <= 256 ? 256 : 512;
    static_assert(COLS <= 512 && int(TMEM_COLS) * CTAS <= 512 && S >= 3, "pipeline");
    // A team that comes to a slot has seen the slot freed TEAMS chunks before it: with
    // fewer slots than teams its wait could be two turns of the ring ahead, where the
    // barrier's parity says nothing.
    static_assert(S >= TEAMS, "no team more than one turn of the ring ahead");
    static constexpr size_t SMEM = size_t(S) * STAGE + RED + TAIL;
};

struct LArgs {
    const uint16_t *x;         // fused: the rows
    const uint8_t *sfa;        // weight scale atoms [MT][KC][512]
    const uint8_t *split;      // else: the split rows [NTL][KC][rows_block]
    int rows, K, N, MT, NTL, KC;
    int KS;
    uint16_t *out;
    int32_t *status;
    long long limit;
    int stall;
    int weights_ready;  // the previous kernel of the stream writes no weights
};

template <int NB, bool FUSED>
__global__ void __launch_bounds__((LCfg<NB, FUSED>::THREADS), (LCfg<NB, FUSED>::CTAS))
    k_linear_mx(const __grid_constant__ CUtensorMap tmA, const LArgs p)
{
    using C = LCfg<NB, FUSED>;
    constexpr int S = C::S;
    // 1 for 128-row tiles, and yet not a constant there: the code built for one was
    // slower (7168 -> 3584, 512 rows: 28.3 us, against 26.1).
    const int KS = p.KS;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *stages = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float *red = reinterpret_cast<float *>(stages + S * C::STAGE);  // [KS - 1][columns of this rank][128]
    uint64_t *full = reinterpret_cast<uint64_t *>(red + C::RED / 4);
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
    if (warp == 0 && lane == 0) prefetch_tensormap(&tmA);
    if (threadIdx.x == 64) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1 + C::TW);  // the weights' producer and the rows'
            mbar_init(&empty[s], 1);
        }
        for (int a = 0; a < C::ACC; ++a) {
            mbar_init(&acc_full[a], 1);
            mbar_init(&acc_empty[a], 128);
        }
        mbar_init(drain, 1);
        mbar_init(red_full, 1);
        mbar_init_fence();
    }
    if (warp == 1) tmem_alloc(tmem_slot, C::TMEM_COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (KS > 1) cluster_sync();  // the cluster's barriers are initialised
    // Behind a kernel that is known not to write them (k_split_rows, the block's
    // own kernels) the weights' warp does not wait: what came before that kernel
    // was complete when it let this one start.
    if (!p.weights_ready || warp != 0) pdl_enter();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0 || (!FUSED && warp == 6)) {
        // ---------------- copies: the weights (warp 0), the split rows (warp 6) ----------------
        int stage = 0, fills = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int it = first; it < total && ok; it += step) {
            const int mt = it % p.MT, nt = it / p.MT;
            for (int kc = k0; kc < k1; ++kc) {
                ok = mbar_wait_warp(&empty[stage], phase ^ 1, p.limit);
                if (!ok) {
                    if (lane == 0) set_status(p.status, LMOE_ERR_TIMEOUT);
                    break;
                }
                uint8_t *sb = stages + stage * C::STAGE;
                if (elect_one()) {
                    if (warp == 0) {
                        if (!(p.stall && it == first && kc == k0)) {
                            mbar_arrive_expect_tx(&full[stage], 128 * 64 + 512);  // packed FP4: 64 bytes a row
                            tma_load_2d(sb, &tmA, kc * 128, mt * 128, &full[stage]);
                            bulk_load(sb + C::SF_OFF, p.sfa + (int64_t(mt) * p.KC + kc) * 512, 512, &full[stage]);
                        }
                    } else {
                        // codes to the operand, the atoms behind them to the scales behind the weights'
                        const uint8_t *src = p.split + (int64_t(nt) * p.KC + kc) * rows_block(NB);
                        mbar_arrive_expect_tx(&full[stage], C::B_TILE + C::NAT * 512);
                        bulk_load(sb + A_TILE, src, C::B_TILE, &full[stage]);
                        bulk_load(sb + C::SF_OFF + 512, src + C::B_TILE, C::NAT * 512, &full[stage]);
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
            for (int f = fills > S ? fills - S : 0; f < fills; ++f) mbar_wait_warp(&full[f % S], (f / S) & 1, p.limit);
    } else if (FUSED && warp >= 6) {
        // ---------------- the rows, split here: team t takes chunks t, t + TEAMS, .. ----------------
        const int per = k1 - k0, mine = total > first ? (total - first + step - 1) / step : 0;
        const int fills = per * mine, r0 = (warp - 6) % C::TW * (NB / 2), c16 = (lane & 15) >> 1;
        // rows of the tile this warp has to split (the others' columns are dropped)
        const int live = p.NTL == 1 ? p.rows - r0 : NB / 2;
        // the pieces of the chunk of fill f: lanes 0-15 one row, lanes 16-31 the next
        auto fetch = [&](int f, uint4 (&u)[C::UNITS]) {
            const int i = f / per, nt = (first + i * step) / p.MT;
            const int c = (k0 + f - i * per) * 128 + (lane & 15) * 8;
#pragma unroll
            for (int j = 0; j < C::UNITS; ++j) {
                const int r = nt * NB + r0 + 2 * j + (lane >> 4);
                u[j] = f < fills && r < p.rows && c < p.K ? *reinterpret_cast<const uint4 *>(p.x + int64_t(r) * p.K + c)
                                                          : make_uint4(0, 0, 0, 0);
            }
        };
        auto split = [&](int f, const uint4 (&u)[C::UNITS]) -> bool {
            const int stage = f % S;
            if (!mbar_wait_warp(&empty[stage], uint32_t(f / S + 1) & 1, p.limit)) {
                if (lane == 0) set_status(p.status, LMOE_ERR_TIMEOUT);
                return false;
            }
            uint8_t *bt = stages + stage * C::STAGE + A_TILE, *sf = stages + stage * C::STAGE + C::SF_OFF + 512;
#pragma unroll
            for (int j = 0; j < C::UNITS; ++j) {
                if (2 * j >= live) break;
                const uint32_t w[4] = {u[j].x, u[j].y, u[j].z, u[j].w};
                uint32_t m = amax8(w);
                m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
                m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
                const int b = split_byte(m), r = r0 + 2 * j + (lane >> 4);
                uint2 hi, lo;
                split8(w, b, hi, lo);
                // 128-byte rows, 16-byte units swizzled by the row
                const int at = r * 128 + ((c16 ^ (r & 7)) << 4) + (lane & 1) * 8;
                *reinterpret_cast<uint2 *>(bt + at) = hi;
                *reinterpret_cast<uint2 *>(bt + NB * 128 + at) = lo;  // NB % 8 == 0: the same swizzle
                if ((lane & 3) == 0) {
                    sf[sf_off(r, (lane & 15) >> 2)] = uint8_t(b);
                    sf[sf_off(NB + r, (lane & 15) >> 2)] = uint8_t(b - 5);
                }
            }
            fence_async_shared();  // the tensor core reads these stores
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[stage]);
            return true;
        };
        // two chunks ahead, so that a chunk's load latency passes under the work on two others
        uint4 u0[C::UNITS], u1[C::UNITS];
        int f = (warp - 6) / C::TW;
        fetch(f, u0);
        fetch(f + C::TEAMS, u1);
        for (; f < fills; f += 2 * C::TEAMS) {
            if (!split(f, u0)) break;
            fetch(f + 2 * C::TEAMS, u0);
            if (f + C::TEAMS >= fills || !split(f + C::TEAMS, u1)) break;
            fetch(f + 3 * C::TEAMS, u1);
        }
    } else if (warp == 1) {
        // ---------------- MMA issuer ----------------
        int stage = 0, acc = 0;
        uint32_t phase = 0, acc_phase = 0;
        bool ok = true;
        for (int it = first; it < total && ok; it += step) {
            const int nv = min(NB, p.rows - it / p.MT * NB);
            const uint32_t N = uint32_t((NB + nv + 15) & ~15);  // hi rows, padding, lo rows
            ok = mbar_wait_warp(&acc_empty[acc], acc_phase ^ 1, p.limit);
            tc_fence_after();
            const uint32_t d = tmem + uint32_t(acc * C::NC);
            for (int kc = k0; kc < k1 && ok; ++kc) {
                ok = mbar_wait_warp(&full[stage], phase, p.limit);
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
                    const uint8_t *sb = stages + stage * C::STAGE;
                    const uint32_t sfa = tmem + uint32_t(C::SF_BASE + stage * C::SF_COLS);
#pragma unroll
                    for (int i = 0; i < 1 + C::NAT; ++i)
                        tc_cp_sf(sfa + 4 * i, sdesc_sf(smem_u32(sb + C::SF_OFF + 512 * i)));
                    const uint64_t ad = sdesc_k128(smem_u32(sb)), bd = sdesc_k128(smem_u32(sb + A_TILE));
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_mxf8f6f4(d, ad + 2 * kk, bd + 2 * kk, idesc_mxf4_e4m3(N, uint32_t(kk)), sfa, sfa + 4,
                                     (kc > k0 || kk > 0) ? 1u : 0u);
                    tc_commit(&empty[stage]);
                }
                __syncwarp();
                if (++stage == S) {
                    stage = 0;
                    phase ^= 1;
                }
            }
            if (!ok) break;
            if (elect_one()) tc_commit(&acc_full[acc]);
            __syncwarp();
            if (++acc == C::ACC) {
                acc = 0;
                acc_phase ^= 1;
            }
        }
        if (!ok) {
            if (elect_one()) {
                set_status(p.status, LMOE_ERR_TIMEOUT);
                tc_commit(drain);  // MMAs in flight end before the tensor memory is freed
                mbar_wait(drain, 0, p.limit);
            }
            __syncwarp();
        }
    } else {
        // ---------------- epilogue ----------------
        constexpr int CW = NB < 32 ? NB : 32;  // rows of x a step: their loads go out together
        const int q = warp & 3;
        int acc = 0;
        uint32_t acc_phase = 0;
        for (int it = first; it < total; it += step) {
            const int mt = it % p.MT, row0 = it / p.MT * NB;
            const int nv = min(NB, p.rows - row0);
            if (!mbar_wait_warp(&acc_full[acc], acc_phase, p.limit)) {
                if (lane == 0) set_status(p.status, LMOE_ERR_TIMEOUT);
                break;
            }
            tc_fence_after();
            const uint32_t tb = tmem + (uint32_t(32 * q) << 16) + uint32_t(acc * C::NC);
            auto sums = [&](int c0, float (&y)[CW]) {  // hi part + lo part of rows c0 ..
                if constexpr (NB == 8) {
                    uint32_t v[16];
                    tmem_ld16(tb, v);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 8; ++j) y[j] = __uint_as_float(v[j]) + __uint_as_float(v[8 + j]);
                } else {
                    uint32_t v[CW], l[CW];
                    tmem_ld_cols<CW>(tb + c0, v);
                    tmem_ld_cols<CW>(tb + NB + c0, l);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < CW; ++j) y[j] = __uint_as_float(v[j]) + __uint_as_float(l[j]);
                }
            };
            const int n = mt * 128 + 32 * q + lane;
            __nv_bfloat16 *o = reinterpret_cast<__nv_bfloat16 *>(p.out) + int64_t(row0) * p.N + n;
            if (KS > 1) {
                const ClusterSum cs(KS, rank, nv, reinterpret_cast<float *>(stages), red, red_full);
                for (int c0 = 0; c0 < nv; c0 += CW) {
                    float y[CW];
                    sums(c0, y);
#pragma unroll
                    for (int j = 0; j < CW; ++j)
                        if (c0 + j < nv) cs.stage[(c0 + j) * 128 + 32 * q + lane] = y[j];
                }
                if (!cs.exchange(p.limit)) {
                    if (lane == 0) set_status(p.status, LMOE_ERR_TIMEOUT);
                    break;
                }
                for (int c0 = cs.own0; c0 < cs.own1; c0 += 8) {
                    float y[8];
                    cs.sum(c0, 32 * q + lane, y);
                    if (n < p.N)
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (c0 + j < cs.own1) o[int64_t(c0 + j) * p.N] = __float2bfloat16_rn(y[j]);
                }
            } else {
                for (int c0 = 0; c0 < nv; c0 += CW) {
                    float y[CW];
                    sums(c0, y);
                    if (n < p.N)
#pragma unroll
                        for (int j = 0; j < CW; ++j)
                            if (c0 + j < nv) o[int64_t(c0 + j) * p.N] = __float2bfloat16_rn(y[j]);
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
    if (KS > 1) cluster_sync_end();  // nobody's shared memory goes while another rank may store into it
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, C::TMEM_COLS);
}

// Rows of a tile.  Up to 16 the kernel splits the rows itself, also of small
// products whose 16-row tiles run at once (512 x 512, 100 rows: 3.9 us, against
// 5.0 with 64-row tiles and the kernel before them).  Beyond, 64 or 128 rows,
// whichever takes less time when all SMs take a tile at once, wave by wave: a
// wave of 128 rows takes about 5/4 of one of 64 (7168 -> 14336, one wave each:
// 24.8 and 19.5 us).  64 and 128 rows: 7168 -> 2304, 512 rows (one wave, one)
// 21.5 and 25.1 us; 7168 -> 3584, 512 rows (two, one) 33.0 and 26.1 us;
// 7168 -> 14336, 100 rows (two, one) 31.6 and 25.8 us, 383 rows (five, three)
// 71.7 and 62.0 us.  Of 45 products measured it was wrong by at most 4%.
// The tile decides the workspace's size, which must not depend on the device that
// happens to be current, so the rule counts on the GB300's 152 SMs; the grid goes
// by the device's own number.
int row_tile(int64_t rows, int64_t K, int64_t N)
{
    if (rows <= 8) return 8;
    if (rows <= 16 || (K <= 12 * 128 && ceil_div(rows, 16) * ceil_div(N, 128) <= 152)) return 16;
    const int64_t cols = ceil_div(N, 128), waves64 = ceil_div(ceil_div(rows, 64) * cols, 152),
                  waves128 = ceil_div(ceil_div(rows, 128) * cols, 152);
    return waves64 * 4 <= waves128 * 5 ? 64 : 128;
}
bool splits_itself(int NB) { return NB <= 16; }

template <int NB, bool FUSED>
cudaLaunchConfig_t config(unsigned grid, cudaStream_t st, cudaLaunchAttribute (&attr)[2], int ks)
{
    using C = LCfg<NB, FUSED>;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(ks);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ks > 1 ? 2 : 1;
    return cfg;
}

// How many clusters of ks CTAs run at once, one CTA an SM (a cluster lies within
// one group of SMs, so sizes that do not divide a group's leave some idle), asked
// once a device; 0 where the runtime does not say.  It answers for one CTA an SM
// whenever a kernel uses tensor memory; two that fit do run side by side.
template <int NB, bool FUSED>
int max_clusters(int ks)
{
    static DeviceCache<MAX_KS + 1> known;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) cudaGetLastError();
    return known.get(dev, ks, [ks] {
        int n = 0;
        cudaLaunchAttribute attr[2];
        cudaLaunchConfig_t cfg = config<NB, FUSED>(unsigned(ks) * 512, nullptr, attr, ks);
        attr[0].val.programmaticStreamSerializationAllowed = 0;
        if (cudaOccupancyMaxActiveClusters(&n, k_linear_mx<NB, FUSED>, &cfg) == cudaSuccess) return n;
        cudaGetLastError();
        return 0;
    });
}

template <int NB, bool FUSED>
cudaError_t launch(LArgs a, const uint8_t *q, cudaStream_t st)
{
    using C = LCfg<NB, FUSED>;
    CUtensorMap ma;
    if (!make_tensor_map(&ma, q, MapType::FP4, int64_t(a.KC) * 128, a.N, 128)) return cudaErrorInvalidValue;
    auto *kern = k_linear_mx<NB, FUSED>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(C::SMEM));
    if (e != cudaSuccess) return e;
    const int sms = device_sms();
    const int64_t items = int64_t(a.MT) * a.NTL;
    // As many ranks an item as make the longest SM's share of the chunks
    // shortest, a split's exchange counted as 5 to 16 chunks (measured: 0.2 us
    // a chunk; 0.9 us for 8 rows, 3.3 us for 64), while every cluster runs at
    // once, with some to spare: the previous kernel's blocks may still hold SMs.
    a.KS = 1;
    int64_t best = ceil_div(items, sms) * a.KC;
    for (int ks = 2; C::SPLITS && ks <= MAX_KS && items * ks <= int64_t(sms) * C::CTAS && ks * 2 <= a.KC; ++ks) {
        const int64_t cost = ceil_div(items * ks, sms) * ceil_div(a.KC, ks) + 4 + NB * 3 / 16;
        if (cost < best && items * 10 <= max_clusters<NB, FUSED>(ks) * C::CTAS * 9) best = cost, a.KS = ks;
    }
    const int64_t slots = int64_t(sms) * C::CTAS / a.KS;
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg =
        config<NB, FUSED>(unsigned((items < slots ? items : slots) * a.KS), st, attr, a.KS);
    return cudaLaunchKernelEx(&cfg, kern, ma, a);
}

}  // namespace

size_t linear_mxfp4_scratch_bytes(int64_t rows, int K, int N)
{
    // The room of 128-row tiles for either size, so that more rows never need
    // less and a workspace made for the most rows serves every smaller call.
    static_assert(rows_block(128) == 2 * rows_block(64), "two small blocks in a large one");
    if (splits_itself(row_tile(rows, K, N))) return 0;
    return size_t(ceil_div(rows, 128) * ceil_div(K, 128) * rows_block(128));
}

cudaError_t launch_linear_mxfp4(const uint16_t *x, const uint8_t *q, const uint8_t *s, int64_t rows, int K, int N,
                                uint16_t *out, void *scratch, int32_t *status, const WaitArgs &wait, cudaStream_t st,
                                bool weights_ready)
{
    const int NB = row_tile(rows, K, N);
    LArgs a{};
    a.x = x;
    a.rows = int(rows);
    a.K = K;
    a.N = N;
    a.MT = int(ceil_div(N, 128));
    a.NTL = int(ceil_div(rows, NB));
    a.KC = int(ceil_div(K, 128));
    if (int64_t(a.MT) * a.NTL > INT32_MAX) return cudaErrorInvalidValue;
    a.sfa = s;
    a.out = out;
    a.status = status;
    a.limit = wait.limit > 0 ? wait.limit : 4000000000LL;  // about 2 s of SM clocks
    a.stall = wait.stall_first_fill;
    a.weights_ready = weights_ready || !splits_itself(NB);
    if (NB == 8) return launch<8, true>(a, q, st);
    if (NB == 16) return launch<16, true>(a, q, st);
    a.split = static_cast<uint8_t *>(scratch);
    const int64_t blocks = ceil_div(rows * a.KC * 16, 256), most = int64_t(device_sms()) * 8;
    const cudaError_t e = launch_pdl(NB == 64 ? k_split_rows<64> : k_split_rows<128>,
                                     dim3(unsigned(blocks < most ? blocks : most)), dim3(256), 0, st, x, rows, K, a.KC,
                                     static_cast<uint8_t *>(scratch));
    if (e != cudaSuccess) return e;
    return NB == 64 ? launch<64, false>(a, q, st) : launch<128, false>(a, q, st);
}

}  // namespace lmoe
