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
// adds the residual and hands the outputs to TMA, while the next tile's MMAs run in the
// other accumulator.  Every wait is bounded (LMOE_ERR_TIMEOUT in the status word).
//
// The tensor cores bound it where K is long (8192 rows 3584 -> 7168 219 us, 1.92 PFLOP/s,
// 99% of a library product's burst rate; 4096 rows 113; both gradients of 4096 rows with
// silu 256, of them 26 for dz), the epilogue where K is short (8192 rows 512 -> 3584 36),
// and the start, K steps and end of one round of tiles where there are few (331 rows
// 1056 -> 1000 7.0).  Both gradients' products share a launch, so that one's last round of
// tiles is filled with the other's.
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
constexpr int MAX_TURNS = 4;  // of parts: they take at most so many turns of the GPU's slots

template <int NT, bool PAIR>
struct LCfg {
    static constexpr int EW = 8;  // epilogue warps, two per TMEM lane quarter (32 columns each in turn)
    static constexpr int THREADS = 32 * (2 + EW);
    static constexpr int CL = PAIR ? 2 : 1;  // CTAs a tile: a pair (cta_group::2) has 256 rows of A, each CTA half of B
    static constexpr int MT = 128 * CL;
    static constexpr int BROWS = NT / CL;
    static constexpr uint32_t B_TILE = BROWS * 128;
    static constexpr uint32_t STAGE = A_TILE + B_TILE;
    static constexpr uint32_t BUF = 4096, BUFS = EW * BUF;  // a chunk of 32 x 32 fp32, or two of bf16, an epilogue warp
    static constexpr int S_RAW = int((225 * 1024 - BUFS) / STAGE);
    static constexpr int S = S_RAW > 8 ? 8 : S_RAW;
    static constexpr int ACC = 2;  // accumulators: a tile's epilogue overlaps the next one's MMAs
    static constexpr uint32_t TMEM_COLS = ACC * NT;
};

// A product: D [M][N], tiles row by row.
struct LJob {
    int64_t M;
    int N, KC, NTL;  // KC: chunks of the reduction; NTL: tiles a row
    int a_mn, b_mn;  // the operand's reduction runs over the rows of its matrix
    // epilogue
    const void *bias, *res;
    int bias_f32, res_f32, out_f32, fn;
    void *out;
    uint16_t *pre;
};
// Consecutive tiles of a product, whole (ks = 1) or each in ks parts of its reduction,
// whose sums go to part [tile][ks][MT][NT] (fp32).
struct LSeg {
    int job, tile0, tiles, ks;
    int item0;  // number of its first item
    float *part;
};
constexpr int MAX_SEGS = 4;

struct LArgs {
    LJob job[2];
    LSeg seg[MAX_SEGS];
    int segs, whole, items;  // items [0, whole) are whole tiles
    // GRAD: dbias [col_n], the sums of col_part's [col_parts][col_n], or null
    float *dbias;
    const float *col_part;
    int col_n, col_parts;
    int32_t *status;
    long long limit;
    int stall;
};

// ---- rows of outputs ---------------------------------------------------------------------

// A chunk of 32 x 32 elements in shared memory: row r's 16-byte pieces, swizzled as the
// tensor maps of outputs have it, so that lanes that each write or read their own row, and
// lanes that hold pieces of one row, meet no bank conflicts.
template <bool F32>
__device__ __forceinline__ uint4 *piece(uint8_t *buf, int r, int i)
{
    return reinterpret_cast<uint4 *>(buf) + (F32 ? r * 8 + (i ^ (r & 7)) : r * 4 + (i ^ ((r >> 1) & 3)));
}
// The lane's row into the chunk, rounded to nearest even.
template <bool F32>
__device__ __forceinline__ void put_row(uint8_t *buf, int lane, const F2 (&y)[16])
{
    uint32_t u[F32 ? 32 : 16];
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
#pragma unroll
    for (int i = 0; i < (F32 ? 8 : 4); ++i)
        *piece<F32>(buf, lane, i) = make_uint4(u[4 * i], u[4 * i + 1], u[4 * i + 2], u[4 * i + 3]);
}
// The lane's row of the chunk added.
template <bool F32>
__device__ __forceinline__ void add_row(uint8_t *buf, int lane, F2 (&y)[16])
{
#pragma unroll
    for (int i = 0; i < (F32 ? 8 : 4); ++i) {
        const uint4 q = *piece<F32>(buf, lane, i);
        const uint32_t u[4] = {q.x, q.y, q.z, q.w};
        if constexpr (F32) {
            y[2 * i] = y[2 * i] + f2(__uint_as_float(u[0]), __uint_as_float(u[1]));
            y[2 * i + 1] = y[2 * i + 1] + f2(__uint_as_float(u[2]), __uint_as_float(u[3]));
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                y[4 * i + j] = y[4 * i + j] + f2(__uint_as_float(u[j] << 16), __uint_as_float(u[j] & 0xFFFF0000u));
        }
    }
}
// A chunk of a matrix, a few rows' pieces an access, in registers; and from there into the
// buffer.  rows, cols: how many of the 32 there are.
template <bool F32>
__device__ __forceinline__ void load_chunk(uint4 (&r)[8], const void *at, int64_t N, int lane, int rows, int cols)
{
    constexpr int L = F32 ? 8 : 4, E = F32 ? 4 : 8;  // lanes a row, elements a piece
    const int row = lane / L, col = lane % L * E;
#pragma unroll
    for (int i = 0; i < L; ++i)
        if (row + i * (32 / L) < rows && col < cols)
            r[i] = *reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(at) +
                                                    ((row + i * (32 / L)) * N + col) * (F32 ? 4 : 2));
}
template <bool F32>
__device__ __forceinline__ void put_chunk(uint8_t *buf, const uint4 (&r)[8], int lane)
{
    constexpr int L = F32 ? 8 : 4;
#pragma unroll
    for (int i = 0; i < L; ++i) *piece<F32>(buf, lane / L + i * (32 / L), lane % L) = r[i];
}

// The chunk (fp32) stored a column a lane, n rows of it, N elements apart; with the residual
// added.
__device__ __forceinline__ float read1(const float *p) { return *p; }
__device__ __forceinline__ float read1(const uint16_t *p) { return bf16_bits_to_f32(*p); }
template <bool F32, typename Out, typename Res = float>
__device__ __forceinline__ void put_columns(uint8_t *buf, int lane, int n, int64_t N, Out *out, const Res *res = nullptr)
{
    float v[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = res && i < n ? read1(res + i * N) : 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        v[i] += reinterpret_cast<const float *>(piece<true>(buf, i, lane >> 2))[lane & 3];
        if (i >= n) continue;
        if constexpr (F32) out[i * N] = v[i];
        else reinterpret_cast<__nv_bfloat16 *>(out)[i * N] = __float2bfloat16_rn(v[i]);
    }
}

// ---- the products ------------------------------------------------------------------------

// Between the epilogue warps alone.
template <int WARPS>
__device__ __forceinline__ void epilogue_sync()
{
    asm volatile("bar.sync 1, %0;" ::"n"(32 * WARPS) : "memory");
}

// GRAD: one or two products whose operands may run either way; else one of K-major operands
// (the choice between operands' orders cost 27.9 -> 29.6 us at 512 rows 7168 -> 3584).
// COPIED: all rows of outputs and residual start on 16 bytes, so whole pieces are copied; else
// single elements (a gradient's rows always do: K % 8 == 0).
template <int NT, bool PAIR, bool GRAD, bool COPIED>
__global__ void __launch_bounds__((LCfg<NT, PAIR>::THREADS), 1)
    k_linear_act(const __grid_constant__ CUtensorMap tmA0, const __grid_constant__ CUtensorMap tmB0,
                 const __grid_constant__ CUtensorMap tmA1, const __grid_constant__ CUtensorMap tmB1,
                 const __grid_constant__ CUtensorMap tmOut0, const __grid_constant__ CUtensorMap tmOut1,
                 const __grid_constant__ CUtensorMap tmPre, const __grid_constant__ LArgs p)
{
    using C = LCfg<NT, PAIR>;
    constexpr int S = C::S;
    static_assert(C::BROWS % 64 == 0, "blocks of 64 elements");
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *stages = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *bufs = stages + S * C::STAGE;
    uint64_t *full = reinterpret_cast<uint64_t *>(bufs + C::BUFS);
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
        prefetch_tensormap(&tmA0);
        prefetch_tensormap(&tmB0);
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
    // This CTA's items: whole tiles, every step-th, then parts, handed out from the other end (the
    // first CTAs may have one whole tile more).
    const int part0 = p.whole + step - 1 - first, begin = first < p.whole ? first : part0;
    auto next = [&](int it) {
        if (it >= p.whole || it + step < p.whole) return it + step;
        return part0;
    };
    struct Item {
        int job, m, n, k0, k1;  // m, n: first row and column of the tile
        float *part;            // of its sums [MT][NT], or null
    };
    auto item = [&](int it) {
        int s = 0;
        while (s + 1 < p.segs && p.seg[s + 1].item0 <= it) ++s;
        const LSeg &g = p.seg[s];
        const LJob &j = p.job[GRAD ? g.job : 0];
        const int l = it - g.item0, k = l / g.tiles, at = l - k * g.tiles, tile = g.tile0 + at;
        Item r;
        r.job = GRAD ? g.job : 0;
        r.m = tile / j.NTL * C::MT;
        r.n = tile % j.NTL * NT;
        r.k0 = int(int64_t(k) * j.KC / g.ks);
        r.k1 = int(int64_t(k + 1) * j.KC / g.ks);
        r.part = g.ks > 1 ? g.part + (int64_t(at) * g.ks + k) * (C::MT * NT) : nullptr;
        return r;
    };

    if (warp == 0) {
        // ---------------- copies ----------------
        int stage = 0, fills = 0;
        uint32_t phase = 0;
        bool ok = true, at_start = true;  // (the failure-path test withholds a CTA's first stage)
        for (int it = begin; it < p.items && ok; it = next(it)) {
            const Item w = item(it);
            const int m0 = w.m + rank * 128, n0 = w.n + rank * C::BROWS;
            const CUtensorMap *tmA = GRAD && w.job ? &tmA1 : &tmA0, *tmB = GRAD && w.job ? &tmB1 : &tmB0;
            const bool a_mn = GRAD && p.job[w.job].a_mn, b_mn = GRAD && p.job[w.job].b_mn;
            for (int kc = w.k0; kc < w.k1; ++kc) {
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
                    if (a_mn) {
                        load(sa, tmA, m0, kc * 64);
                        load(sa + 8192, tmA, m0 + 64, kc * 64);
                    } else {
                        load(sa, tmA, kc * 64, m0);
                    }
                    if (b_mn) {
#pragma unroll
                        for (int b = 0; b < C::BROWS / 64; ++b) load(sb + b * 8192, tmB, n0 + 64 * b, kc * 64);
                    } else {
                        load(sb, tmB, kc * 64, n0);
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
        for (int it = begin; it < p.items && ok; it = next(it)) {
            const Item w = item(it);
            const bool a_mn = GRAD && p.job[w.job].a_mn, b_mn = GRAD && p.job[w.job].b_mn;
            const uint32_t id = (PAIR ? idesc_bf16_pair(NT) : idesc_bf16(NT)) | (a_mn ? IDESC_A_MN : 0) | (b_mn ? IDESC_B_MN : 0);
            const uint32_t a_step = a_mn ? 128 : 2, b_step = b_mn ? 128 : 2;  // 16 of the reduction, in 16-byte units
            const uint32_t base = smem_u32(stages);
            const uint64_t ad0 = a_mn ? sdesc_mn128(base, 8192) : sdesc_k128(base);  // of stage 0
            const uint64_t bd0 = b_mn ? sdesc_mn128(base + A_TILE, 8192) : sdesc_k128(base + A_TILE);
            ok = mbar_wait_warp(&acc_empty[acc], acc_phase ^ 1, p.limit);
            tc_fence_after();
            const uint32_t d = tmem + uint32_t(acc * NT);
            const int k0 = w.k0, k1 = w.k1;
            for (int kc = k0; kc < k1 && ok; ++kc) {
                ok = mbar_wait_warp(&full[stage], phase, p.limit);
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t ad = ad0 + uint32_t(stage) * (C::STAGE >> 4), bd = bd0 + uint32_t(stage) * (C::STAGE >> 4);
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
        // 32 rows x 32 columns at a time.  Outputs go through shared memory and are copied from there
        // by TMA, the residual comes the other way round in whole pieces of rows: stored from the
        // lanes' registers, a row a lane, every 16 or 32 bytes were a request to L2 of their own
        // (6000 rows 128 -> 3000, fp32 residual and output, pre: 57 us, 10.5 million requests).
        __shared__ __align__(16) float s_bias[C::EW][32];
        const int q = warp & 3, half = (warp - 2) >> 2;
        uint8_t *buf = bufs + (warp - 2) * C::BUF, *pre_buf = buf + C::BUF / 2;
        // These warps wait for the first tile anyway: the column sums of dz, in k_col_sums' order (16
        // strands), here two of them a warp.  A launch of its own for them took 1.5 to 3.5 us (333 x 1056 x 1000
        // 12.4 against 10.9, one row 3584 -> 7168 40.0 against 36.5, 8192 x 512 x 256 25.8 against 22.5).
        if (GRAD && p.dbias) {
            constexpr int STRANDS = 16;
            float(*s_cols)[32] = reinterpret_cast<float(*)[32]>(bufs);  // [STRANDS]
            for (int64_t c0 = int64_t(blockIdx.x) * 32; c0 < p.col_n; c0 += int64_t(gridDim.x) * 32) {
                const int64_t c = c0 + lane;
                for (int strand = warp - 2; strand < STRANDS; strand += C::EW) {
                    float v = 0.f;
                    if (c < p.col_n)
                        for (int g = strand; g < p.col_parts; g += 8 * STRANDS) {
                            float r[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                r[i] = g + i * STRANDS < p.col_parts ? p.col_part[int64_t(g + i * STRANDS) * p.col_n + c] : 0.f;
#pragma unroll
                            for (int i = 0; i < 8; ++i) v += r[i];
                        }
                    s_cols[strand][lane] = v;
                }
                epilogue_sync<C::EW>();
                if (warp == 2 && c < p.col_n) {
                    float v = s_cols[0][lane];
#pragma unroll
                    for (int i = 1; i < STRANDS; ++i) v += s_cols[i][lane];
                    p.dbias[c] = v;
                }
                epilogue_sync<C::EW>();
            }
        }
        int acc = 0;
        uint32_t acc_phase = 0;
        for (int it = begin; it < p.items; it = next(it)) {
            const Item w = item(it);
            const LJob &j = p.job[GRAD ? w.job : 0];
            const int64_t m = w.m + rank * 128 + 32 * q;  // the warp's first row
            const int n0 = w.n, limit = min(NT, j.N - n0), rows = int(min(int64_t(32), j.M - m));
            const uint32_t tb = tmem + (uint32_t(32 * q) << 16) + uint32_t(acc * NT);
            // what 32 columns need from memory, on its way a turn ahead: the residual, a column's bias a lane
            uint4 r[8];
            float bias = 0.f;
            auto fetch = [&](int c) {
                if (c >= limit || w.part) return;
                if (COPIED && j.res) {
                    const int64_t at = m * j.N + n0 + c;
                    if (j.res_f32) load_chunk<true>(r, static_cast<const float *>(j.res) + at, j.N, lane, rows, limit - c);
                    else load_chunk<false>(r, static_cast<const uint16_t *>(j.res) + at, j.N, lane, rows, limit - c);
                }
                if (j.bias && c + lane < limit)
                    bias = j.bias_f32 ? __ldg(static_cast<const float *>(j.bias) + n0 + c + lane)
                                      : bf16_bits_to_f32(__ldg(static_cast<const uint16_t *>(j.bias) + n0 + c + lane));
            };
            fetch(32 * half);
            if (!mbar_wait_warp(&acc_full[acc], acc_phase, p.limit)) {
                if (lane == 0) set_status(p.status, LMOE_ERR_TIMEOUT);
                break;
            }
            tc_fence_after();
            if (w.part) {
                float *sums = w.part + int64_t(rank * 128 + 32 * q + lane) * NT;
                for (int c = 32 * half; c < limit; c += 8 * C::EW) {
                    uint32_t v[32];
                    tmem_ld_cols<32>(tb + c, v);
                    tmem_ld_wait();
                    if (lane < rows)
#pragma unroll
                        for (int i = 0; i < 32; i += 8)
                            asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(sums + c + i), "r"(v[i]),
                                         "r"(v[i + 1]), "r"(v[i + 2]), "r"(v[i + 3]), "r"(v[i + 4]), "r"(v[i + 5]),
                                         "r"(v[i + 6]), "r"(v[i + 7])
                                         : "memory");
                    __syncwarp();
                }
            }
            for (int c = 32 * half; c < limit && !w.part; c += 8 * C::EW) {
                uint32_t v[32];
                tmem_ld_cols<32>(tb + c, v);
                F2 y[16];
                if (j.bias) s_bias[warp - 2][lane] = bias;
                if (COPIED && elect_one()) bulk_wait_read<0>();  // the copies of the chunk before have read the buffers
                __syncwarp();
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) y[i] = f2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
                if (j.bias) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float4 b = *reinterpret_cast<const float4 *>(&s_bias[warp - 2][4 * i]);
                        y[2 * i] = y[2 * i] + f2(b.x, b.y);
                        y[2 * i + 1] = y[2 * i + 1] + f2(b.z, b.w);
                    }
                    __syncwarp();
                }
                if constexpr (!COPIED) {
                    // Rows that start anywhere: turned round, so that a lane has a column and an access is a
                    // piece of one row.
                    const int n_rows = c + lane < limit ? rows : 0;
                    const int64_t at = m * j.N + n0 + c + lane;
                    if (j.pre) {
                        put_row<true>(buf, lane, y);
                        __syncwarp();
                        put_columns<false>(buf, lane, n_rows, j.N, j.pre + at);
                        __syncwarp();
                    }
                    apply_fn(j.fn, y);
                    put_row<true>(buf, lane, y);
                    __syncwarp();
                    if (j.out_f32) {
                        float *o = static_cast<float *>(j.out) + at;
                        if (!j.res) put_columns<true>(buf, lane, n_rows, j.N, o);
                        else if (j.res_f32) put_columns<true>(buf, lane, n_rows, j.N, o, static_cast<const float *>(j.res) + at);
                        else put_columns<true>(buf, lane, n_rows, j.N, o, static_cast<const uint16_t *>(j.res) + at);
                    } else {
                        uint16_t *o = static_cast<uint16_t *>(j.out) + at;
                        if (!j.res) put_columns<false>(buf, lane, n_rows, j.N, o);
                        else if (j.res_f32) put_columns<false>(buf, lane, n_rows, j.N, o, static_cast<const float *>(j.res) + at);
                        else put_columns<false>(buf, lane, n_rows, j.N, o, static_cast<const uint16_t *>(j.res) + at);
                    }
                    __syncwarp();
                    fetch(c + 8 * C::EW);
                } else {
                    if (j.pre) {
                        put_row<false>(pre_buf, lane, y);
                        fence_async_shared();
                        __syncwarp();
                        if (rows > 0 && elect_one()) {
                            tma_store_2d(&tmPre, n0 + c, int(m), pre_buf);
                            bulk_commit();
                        }
                        __syncwarp();
                    }
                    apply_fn(j.fn, y);
                    if (j.pre && (j.out_f32 || (j.res && j.res_f32))) {  // which take pre's half of the buffer too
                        if (elect_one()) bulk_wait_read<0>();
                        __syncwarp();
                    }
                    if (j.res) {
                        if (j.res_f32) {
                            put_chunk<true>(buf, r, lane);
                            __syncwarp();
                            add_row<true>(buf, lane, y);
                        } else {
                            put_chunk<false>(buf, r, lane);
                            __syncwarp();
                            add_row<false>(buf, lane, y);
                        }
                        __syncwarp();
                    }
                    fetch(c + 8 * C::EW);
                    if (j.out_f32) put_row<true>(buf, lane, y);
                    else put_row<false>(buf, lane, y);
                    fence_async_shared();
                    __syncwarp();
                    if (rows > 0 && elect_one()) {
                        tma_store_2d(GRAD && w.job ? &tmOut1 : &tmOut0, n0 + c, int(m), buf);
                        bulk_commit();
                    }
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
        if (elect_one()) bulk_wait_read<0>();
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    // nobody's shared or tensor memory goes while the pair's other CTA may still write or read it
    if (PAIR) cluster_sync_end();
    tc_fence_after();
    if (warp == 1) PAIR ? tmem_dealloc_pair(tmem, C::TMEM_COLS) : tmem_dealloc(tmem, C::TMEM_COLS);
}

// ---- parts of the reduction ------------------------------------------------------------------

// The parts' sums added in order, then the epilogue: eight columns a thread, the blocks of
// a tile one after another.
template <int MT, int NT>
__global__ void __launch_bounds__(256) k_split_sum(const __grid_constant__ LArgs p)
{
    constexpr int PER = MT * NT / 8 / 256;  // blocks a tile
    int at = int(blockIdx.x) / PER, s = 0;
    while (p.seg[s].ks == 1 || at >= p.seg[s].tiles) {
        if (p.seg[s].ks > 1) at -= p.seg[s].tiles;
        ++s;
    }
    const LSeg &g = p.seg[s];
    const LJob &j = p.job[g.job];
    const int e = int(blockIdx.x) % PER * 256 + threadIdx.x, tile = g.tile0 + at;
    const int64_t m = int64_t(tile / j.NTL) * MT + e / (NT / 8);
    const int n = tile % j.NTL * NT + e % (NT / 8) * 8, left = j.N - n;
    pdl_enter();
    if (m >= j.M || left <= 0) return;
    const float *sums = g.part + int64_t(at) * g.ks * (MT * NT) + e * 8;
    F2 y[4] = {f2(0.f), f2(0.f), f2(0.f), f2(0.f)}, v[4];
    for (int k = 0; k < g.ks; ++k) {
        Pack<float, 8> q;
        q.load(sums + int64_t(k) * (MT * NT));
        pairs(q, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = y[i] + v[i];
    }
    const bool wide = j.N % 8 == 0;
    const int64_t to = m * j.N + n;
    auto add = [&](const void *base, bool f32, int64_t from) {  // eight elements of bias or residual
        if (wide) {
            if (f32) {
                Pack<float, 8> q;
                q.load(static_cast<const float *>(base) + from);
                pairs(q, v);
            } else {
                Pack<uint16_t, 8> q;
                q.load(static_cast<const uint16_t *>(base) + from);
                pairs(q, v);
            }
        } else {
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                f[i] = i >= left ? 0.f : f32 ? static_cast<const float *>(base)[from + i]
                                             : bf16_bits_to_f32(static_cast<const uint16_t *>(base)[from + i]);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = f2(f[2 * i], f[2 * i + 1]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = y[i] + v[i];
    };
    auto put = [&](void *base, bool f32) {
        if (wide) {
            if (f32) {
                Pack<float, 8> q;
                set_pairs(q, y);
                q.store(static_cast<float *>(base) + to);
            } else {
                Pack<uint16_t, 8> q;
                set_pairs(q, y);
                q.store(static_cast<uint16_t *>(base) + to);
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float lo, hi;
            f2_get(y[i / 2], lo, hi);
            const float f = i & 1 ? hi : lo;
            if (i >= left) continue;
            if (f32) static_cast<float *>(base)[to + i] = f;
            else static_cast<__nv_bfloat16 *>(base)[to + i] = __float2bfloat16_rn(f);
        }
    };
    if (j.bias) add(j.bias, j.bias_f32, n);
    if (j.pre) put(j.pre, false);
    apply_fn(j.fn, y);
    if (j.res) add(j.res, j.res_f32, to);
    put(j.out, j.out_f32);
}

// ---- the choice of tiles and parts -----------------------------------------------------------

// Tiles: rows x columns, CTAs, a chunk's bytes a CTA and its time in ns where it has the
// copies it asks for.
struct Tile {
    int M, N, ctas, bytes, chunk;
};
constexpr Tile TILES[4] = {
    {256, 256, 2, 32768, 295}, {256, 128, 2, 24576, 175}, {128, 128, 1, 32768, 213}, {128, 64, 1, 24576, 190}};

// What a product's sizes and epilogue say of its time.
struct Size {
    int64_t M, N, K;
    int extra;  // residual and pre: 0 to 2
};
// The tile, and how many tiles of each product are split into how many parts (the last
// ones; none: ks = 1).
struct Plan {
    int tile = 0;
    int64_t split[2] = {0, 0};
    int ks[2] = {1, 1};
};

// The least time by a model of one or two products in one launch, the longer reduction
// first: whole tiles in turns of the GPU's slots; a chunk's time, or that of its bytes at
// the 14 TB/s that all SMs' copies together get out of L2; an epilogue that shows where
// the reduction is short, and at the end; parts for what is left after whole turns (or for
// all where that is less than a turn), or for the longer product where its tiles are few,
// with the second kernel and its traffic.  Measured, us:
//                          256x256  256x128  128x128  128x64   256x128, 2 parts   128x128, 2 / 3 / 4 parts
//   512 rows 7168 -> 3584    38.3     27.9     33.8     53.5        -                 -
//   200 rows 7168 -> 3584    37.6     24.3     28.3     29.9       20.4              22.9
//   128 rows 7168 -> 3584    37.6     24.2     28.5     26.2       23.3              19.9 / 17.9 / 18.0
//   600 rows 7168 -> 1024    37.5     24.1     28.0     26.5       19.3              20.3 / 18.5 / -
//   331 rows 1056 -> 1000    13.2      9.2      9.5      7.8        8.1               8.2 / 8.2 / 8.6
//   300 rows  512 -> 512      9.5      6.4      6.6      5.3        7.2               7.2
//   1000 rows 1024 -> 2048   12.0      8.6      9.4     11.0        -                 -
Plan plan(const Size *size, int jobs)
{
    const int sms = device_sms();
    const int last = jobs - 1;
    Plan best;
    double least = 1e300;
    for (int t = 0; t < 4; ++t) {
        const Tile &T = TILES[t];
        const int64_t slots = sms / T.ctas;
        const int turns_n = T.N / 64;  // 32 columns at a time, of an epilogue warp
        int64_t KC[2] = {0, 0}, tiles[2] = {0, 0}, total = 0;
        double epi[2] = {0, 0}, tail = 0;
        for (int j = 0; j < jobs; ++j) {
            KC[j] = ceil_div(size[j].K, 64);
            tiles[j] = ceil_div(size[j].M, T.M) * ceil_div(size[j].N, T.N);
            epi[j] = 1500 + turns_n * (450 + 500 * size[j].extra);  // from tile to tile
            tail = 500 + turns_n * (350 + 400 * size[j].extra);     // the last one's
            total += tiles[j];
        }
        auto chunk = [&](int64_t items) {
            const double from_l2 = double((items < slots ? items : slots) * T.ctas) * T.bytes / 14000;
            return from_l2 > T.chunk ? from_l2 : double(T.chunk);
        };
        const double c = chunk(total);
        // n whole tiles of a product, one after another
        auto whole = [&](int j, double n) {
            const double main = KC[j] * c;
            return n <= 0 ? 0. : main > epi[j] ? n * main : main + (n - 1) * epi[j];
        };
        auto offer = [&](double ns, const Plan &p) {
            if (ns < least) {
                least = ns;
                best = p;
            }
        };
        auto traffic = [&](double parts_of_tiles) { return 1000 + parts_of_tiles * T.M * T.N * 8 / 3000; };
        // when the slots end that have one tile of product 0 more than the others, and the others
        double more, less;
        auto turns = [&](int64_t n_last) {
            const int64_t t0 = jobs > 1 ? tiles[0] : 0, all = t0 + n_last;
            const int64_t q0 = t0 / slots, q = all / slots;
            const bool extra = t0 % slots > 0, partial = all % slots > 0;
            less = whole(0, double(q0)) + whole(last, double(q - q0 + partial));
            more = extra ? whole(0, double(q0 + 1)) + whole(last, double(q - q0 + partial - 1)) : less;
            if (more < less) more = less;
        };
        turns(tiles[last]);
        Plan p;
        p.tile = t;
        offer(more + tail, p);
        if (total < slots) {
            for (int k0 = 2; k0 <= MAX_PARTS && KC[0] >= 4 * k0; ++k0) {
                const int64_t len = ceil_div(KC[0], k0);
                int64_t items = 0;
                double bytes = 0;
                for (int j = 0; j < jobs; ++j) {
                    const int64_t k = ceil_div(KC[j], len);
                    p.ks[j] = int(k > MAX_PARTS ? MAX_PARTS : k);
                    p.split[j] = p.ks[j] > 1 ? tiles[j] : 0;
                    items += tiles[j] * p.ks[j];
                    if (p.ks[j] > 1) bytes += double(p.ks[j]) * double(size[j].M) * double(size[j].N) * 8;
                }
                if (items > slots) break;
                offer(double(len) * chunk(items) + 1000 + bytes / 3000, p);
            }
            continue;
        }
        if (const int64_t r = total % slots; r > 0 && r <= tiles[last]) {
            turns(tiles[last] - r);
            const int64_t room = jobs > 1 ? slots - tiles[0] % slots : 0;  // slots that end early
            for (int ks = 2; ks <= MAX_PARTS && KC[last] >= 4 * ks && r * ks <= MAX_TURNS * slots; ++ks) {
                const double n = double(ceil_div(r * ks, slots) * ceil_div(KC[last], ks)) * c;
                const double end = r * ks <= room ? (less + n < more ? more : less + n) : more + n;
                p.split[last] = r;
                p.ks[last] = ks;
                offer(end + traffic(double(r * ks)), p);
            }
        }
        if (jobs > 1 && tiles[0] < slots) {
            p = Plan();
            p.tile = t;
            p.split[0] = tiles[0];
            for (int ks = 2; ks <= MAX_PARTS && KC[0] >= 4 * ks && tiles[0] * ks <= MAX_TURNS * slots; ++ks) {
                const double len = double(ceil_div(KC[0], ks)) * c, one = KC[1] * c > epi[1] ? KC[1] * c : epi[1];
                p.ks[0] = ks;
                offer((double(tiles[0] * ks) * len + double(tiles[1]) * one) / double(slots) + (len > one ? len : one) +
                          traffic(double(tiles[0] * ks)),
                      p);
            }
        }
    }
    return best;
}

// Room for the parts of any plan of these products, of each by itself, and of any with fewer
// rows: no plan has more parts than MAX_TURNS allow, nor a product more than one for every
// four chunks of its reduction.  (What one plan needs does not grow with the rows: none at
// 8192 rows 7168 -> 3584, 15 MB at 333.)
size_t part_room(const Size *size, int jobs)
{
    const int64_t sms = device_sms();
    size_t most = 0;
    for (const Tile &T : TILES) {
        int64_t parts = 0;
        for (int j = 0; j < jobs; ++j) {
            const int64_t ks = ceil_div(ceil_div(size[j].K, 64), 4);
            if (ks > 1) parts += ceil_div(size[j].M, T.M) * ceil_div(size[j].N, T.N) * (ks < MAX_PARTS ? ks : MAX_PARTS);
        }
        const int64_t cap = sms / T.ctas * MAX_TURNS;
        const size_t n = size_t(parts < cap ? parts : cap) * T.M * T.N * 4;
        most = n > most ? n : most;
    }
    return most;
}

// An operand: [rows][cols] bf16, rows `stride` elements apart; mn: the reduction runs over its rows.
struct Operand {
    const uint16_t *p;
    int64_t rows, cols, stride;
    bool mn;
};

template <int NT, bool PAIR, bool GRAD, bool COPIED>
cudaError_t launch(const Operand (*ops)[2], int jobs, const LArgs &g, cudaStream_t st)
{
    using C = LCfg<NT, PAIR>;
    CUtensorMap maps[2][2], out[2], pre;
    for (int j = 0; j < jobs; ++j) {
        const Operand &A = ops[j][0], &B = ops[j][1];
        if (!make_tensor_map(&maps[j][0], A.p, MapType::BF16, A.cols, A.rows, A.mn ? 64 : 128, A.stride) ||
            !make_tensor_map(&maps[j][1], B.p, MapType::BF16, B.cols, B.rows, B.mn ? 64 : C::BROWS, B.stride))
            return cudaErrorInvalidValue;
        const LJob &b = g.job[j];
        if (!COPIED) out[j] = maps[0][0];  // (not used)
        else if (!make_store_map(&out[j], b.out, b.out_f32, b.N, b.M)) return cudaErrorInvalidValue;
    }
    if (jobs == 1) {  // (not used)
        maps[1][0] = maps[1][1] = maps[0][0];
        out[1] = out[0];
    }
    pre = out[0];
    if (COPIED && g.job[0].pre && !make_store_map(&pre, g.job[0].pre, false, g.job[0].N, g.job[0].M))
        return cudaErrorInvalidValue;
    const size_t smem = 1024 + size_t(C::S) * C::STAGE + C::BUFS + (2 * C::S + 2 * C::ACC + 1) * 8 + 8;
    auto *kern = k_linear_act<NT, PAIR, GRAD, COPIED>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e != cudaSuccess) return e;
    const int slots = device_sms() / C::CL;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned((g.items < slots ? g.items : slots) * C::CL));
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
    e = cudaLaunchKernelEx(&cfg, kern, maps[0][0], maps[0][1], maps[1][0], maps[1][1], out[0], out[1], pre, g);
    if (e != cudaSuccess || g.items == g.whole) return e;
    int split = 0;
    for (int s = 0; s < g.segs; ++s) split += g.seg[s].ks > 1 ? g.seg[s].tiles : 0;
    return launch_pdl(k_split_sum<C::MT, NT>, dim3(unsigned(split * (C::MT * NT / 8 / 256))), dim3(256), 0, st, g);
}

// Whether every row of every tensor starts on 16 bytes.
bool rows_on_16(const LJob &g)
{
    auto fits = [&](const void *p, int bytes) { return !p || int64_t(g.N) * bytes % 16 == 0; };
    return fits(g.out, g.out_f32 ? 4 : 2) && fits(g.pre, 2) && fits(g.res, g.res_f32 ? 4 : 2);
}

template <bool GRAD, bool COPIED>
cudaError_t on_tile(int tile, const Operand (*ops)[2], int jobs, const LArgs &g, cudaStream_t st)
{
    switch (tile) {
    case 0: return launch<256, true, GRAD, COPIED>(ops, jobs, g, st);
    case 1: return launch<128, true, GRAD, COPIED>(ops, jobs, g, st);
    case 2: return launch<128, false, GRAD, COPIED>(ops, jobs, g, st);
    default: return launch<64, false, GRAD, COPIED>(ops, jobs, g, st);
    }
}

// One product or two, the longer reduction first; ops[j]: A and B of product j.
template <bool GRAD>
cudaError_t products(const Operand (*ops)[2], const Size *size, int jobs, const Plan &pl, LArgs g, const WaitArgs &wait,
                     void *parts, cudaStream_t st)
{
    const Tile &T = TILES[pl.tile];
    float *part = static_cast<float *>(parts);
    int64_t tiles[2] = {0, 0}, items = 0;
    for (int j = 0; j < jobs; ++j) {
        LJob &b = g.job[j];
        b.M = size[j].M;
        b.N = int(size[j].N);
        b.KC = int(ceil_div(size[j].K, 64));
        b.NTL = int(ceil_div(size[j].N, T.N));
        b.a_mn = ops[j][0].mn;
        b.b_mn = ops[j][1].mn;
        tiles[j] = ceil_div(size[j].M, T.M) * b.NTL;
    }
    for (int parted = 0; parted < 2; ++parted) {  // whole tiles first
        for (int j = 0; j < jobs; ++j) {
            const int64_t n = parted ? pl.split[j] : tiles[j] - pl.split[j];
            if (n == 0) continue;
            const int ks = parted ? pl.ks[j] : 1;
            g.seg[g.segs++] = {j, int(tiles[j] - n) * parted, int(n), ks, int(items), parted ? part : nullptr};
            if (parted) part += n * ks * T.M * T.N;
            items += n * ks;
        }
        if (!parted) g.whole = int(items);
    }
    if (items > INT32_MAX / 2) return cudaErrorInvalidValue;
    g.items = int(items);
    g.limit = wait.limit > 0 ? wait.limit : 4000000000LL;  // about 2 s of SM clocks
    g.stall = wait.stall_first_fill;
    if constexpr (!GRAD)
        if (!rows_on_16(g.job[0])) return on_tile<GRAD, false>(pl.tile, ops, jobs, g, st);
    return on_tile<GRAD, true>(pl.tile, ops, jobs, g, st);
}

// ---- dz and its column sums ----------------------------------------------------------------
//
// dz is fp32 until the column sums have it, and is rounded to bf16 for the two products: the
// tensor cores take operands of one type, and the other operand, x or W, is bf16.  Half a step
// of every term leaves dx and dW 2.3e-3 of their size from 64 bits, where rounding bf16 results
// alone leaves 1.7e-3.  dz as two bf16 pieces would keep it, at twice the products' time (214 of
// the 256 us at 4096 rows 3584 -> 7168).

struct DzArgs {
    const void *dout;
    const uint16_t *pre;
    int64_t rows;
    int N, Np;       // dz's rows are Np elements apart, the columns beyond N zero
    uint16_t *dz;    // null: only the column sums
    float *part;     // [gridDim.y][N], or null
};

// A block takes 256 columns and every gridDim.y-th group of eight rows, a warp a row
// of it, a lane eight columns.  VEC: rows start on 16 bytes.  (fp32 gradients through a
// function spill 60 to 90 bytes at the 64 registers that four blocks an SM leave; the sums
// alone of 4096 x 7168, silu, read 5.1 TB/s all the same, 34.7 us, bf16 ones 4.7 TB/s, 24.9.)
template <bool F32, int FN, bool VEC>
__global__ void __launch_bounds__(256, 4) k_act_back(const DzArgs p)
{
    __shared__ float s_cols[8][256 + 8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = (int(blockIdx.x) * 32 + lane) * 8;
    float sum[8] = {};
    pdl_enter();
    constexpr int B = FN == LMOE_FN_NONE && !F32 ? 8 : 4;
    const int64_t step = int64_t(gridDim.y) * 8;
    if (c < p.Np)
        for (int64_t t0 = int64_t(blockIdx.y) * 8 + warp; t0 < p.rows; t0 += B * step) {
            // several rows' loads at once: one row at a time left the loads' latency open (4096 x 7168,
            // silu, dz and sums: 36 against 26 us)
            Pack<float, 8> df[F32 && VEC ? B : 1];
            Pack<uint16_t, 8> dh[!F32 && VEC ? B : 1], zh[FN != LMOE_FN_NONE && VEC ? B : 1];
            if constexpr (VEC) {
#pragma unroll
                for (int i = 0; i < B; ++i) {
                    const int64_t at = min(t0 + i * step, p.rows - 1) * p.N + c;
                    if constexpr (F32) df[i].load(static_cast<const float *>(p.dout) + at);
                    else dh[i].load(static_cast<const uint16_t *>(p.dout) + at);
                    if constexpr (FN != LMOE_FN_NONE) zh[i].load(p.pre + at);
                }
            }
#pragma unroll
            for (int i = 0; i < B; ++i) {
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

// Up to this many rows the weights' stream is the bound (k_linear_few.cu).  us there and here,
// 64 rows: 3584 -> 7168 13.2 and 15.9, 7168 -> 3584 14.6 and 16.7, 7168 -> 28672 64 and 73,
// 1024 -> 1024 6.0 and 6.6, 512 -> 512 6.7 and 6.2; dx of 3584 -> 7168 12.5 and 15.1.  96 and 128
// rows took it 23.4 and 21.1 (3584 -> 7168, 7168 -> 3584) against 18.6 and 17.5 here.
constexpr int64_t FEW = 64;

size_t linear_act_scratch_bytes(int64_t rows, int K, int N)
{
    const Size size{rows, N, K, 0};
    return rows > FEW ? part_room(&size, 1) : 0;
}

cudaError_t launch_linear_act(const LinearActArgs &a, void *scratch, cudaStream_t st)
{
    if (a.rows <= FEW) {
        FewArgs f{};
        f.x = a.x;
        f.x_stride = a.K;
        f.rows = a.rows;
        f.W = a.W;
        f.K = a.K;
        f.N = a.N;
        f.bias = a.bias;
        f.res = a.res;
        f.bias_fmt = a.bias_fmt;
        f.res_fmt = a.res_fmt;
        f.out_fmt = a.out_fmt;
        f.fn = a.fn;
        f.out = a.out;
        f.pre = a.pre;
        f.status = a.status;
        f.wait = a.wait;
        return launch_linear_few(f, st);
    }
    LArgs g{};
    LJob &j = g.job[0];
    j.bias = a.bias;
    j.bias_f32 = a.bias_fmt == LMOE_F32;
    j.res = a.res;
    j.res_f32 = a.res_fmt == LMOE_F32;
    j.out_f32 = a.out_fmt == LMOE_F32;
    j.fn = a.fn;
    j.out = a.out;
    j.pre = a.pre;
    g.status = a.status;
    const Size size{a.rows, a.N, a.K, (a.res != nullptr) + (a.pre != nullptr)};
    const Operand ops[1][2] = {{{a.x, a.rows, a.K, a.K, false}, {a.W, a.N, a.K, a.K, false}}};
    return products<false>(ops, &size, 1, plan(&size, 1), g, a.wait, scratch, st);
}

// dz [rows][Np] bf16 | column sums | parts of the products' reductions
size_t linear_act_back_scratch_bytes(int64_t rows, int K, int N)
{
    if (rows == 0) return 0;
    const int64_t Np = round_up(N, 8);
    const Size products[2] = {{N, K, rows, 0}, {rows, K, N, 0}};  // dW, dx (few rows' goes another way)
    return size_t(round_up(rows * Np * 2, 256)) + size_t(round_up(dz_splits(rows, N) * N * 4, 256)) +
           part_room(products, rows > FEW ? 2 : 1);
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
        // the products' kernel adds the groups' sums up on the way, where there is one
        if (e == cudaSuccess && a.dbias && !a.dW && (!a.dx || a.rows <= FEW))
            e = launch_col_sums(part, grid.y, a.N, 1, a.dbias, nullptr, st);
        if (e != cudaSuccess) return e;
    }
    // both products in one launch, the longer reduction first
    const Operand d{as_is ? static_cast<const uint16_t *>(a.dout) : dz, a.rows, a.N, Np, false};
    Operand ops[2][2];
    Size size[2];
    LArgs g{};
    g.status = a.status;
    g.dbias = a.dbias;
    g.col_part = part;
    g.col_n = a.N;
    g.col_parts = int(dz_splits(a.rows, a.N));
    int jobs = 0;
    auto dx = [&] {
        if (!a.dx) return;
        g.job[jobs].out = a.dx;
        size[jobs] = {a.rows, a.K, a.N, 0};
        ops[jobs][0] = d;
        ops[jobs++][1] = {a.W, a.N, a.K, a.K, true};
    };
    auto dW = [&] {
        if (!a.dW) return;
        g.job[jobs].out = a.dW;
        g.job[jobs].out_f32 = a.dW_fmt == LMOE_F32;
        size[jobs] = {a.N, a.K, a.rows, 0};
        ops[jobs][0] = d;
        ops[jobs][0].mn = true;
        ops[jobs++][1] = {a.x, a.rows, a.K, a.K, true};
    };
    if (a.dx && a.rows <= FEW) {  // the weights' stream is the bound
        FewArgs f{};
        f.x = d.p;
        f.x_stride = Np;
        f.rows = a.rows;
        f.W = a.W;
        f.across = true;
        f.K = a.N;
        f.N = a.K;
        f.out = a.dx;
        f.status = a.status;
        f.wait = a.wait;
        e = launch_linear_few(f, st);
        if (e != cudaSuccess) return e;
        dW();
    } else if (a.N >= a.rows) {
        dx();
        dW();
    } else {
        dW();
        dx();
    }
    return jobs ? products<true>(ops, size, jobs, plan(size, jobs), g, a.wait, parts, st) : e;
}

}  // namespace lmoe
