// bf16 products grouped by expert, ragged groups:
//   out[q][n] = w(q) * sum_c x[src(q)][c] * W[e(q)][n][c]
// and the gated pair h[q][i] = bf16( silu(g) * u ), on the tensor cores
// (tcgen05.mma kind::f16, fp32 accumulation in TMEM).
//
// The weight rows are the M = 128 operand (A), the expert's rows the N operand
// (B, both K-major, 64 columns = one 128-byte swizzle row a chunk), so N
// follows the group's rows (16..NT in steps of 16) and a short group costs no
// tensor work on padding.  For the gated pair an A tile holds 64 features:
// of each TMEM lane quarter's 32 rows, 16 of the gate matrix and the same 16
// of the up matrix, so both products of a feature meet in one warp and the
// accumulator is no larger than a plain one.
//
// Work items (expert, row tile of NT, weight tile), row tile fastest, so an A
// tile is read from HBM once and the row tiles that share it run side by side
// out of L2.  The item list is never written down: every CTA scans the offsets
// into per-expert tile counts in shared memory and finds its items by a warp
// search.
//
// Persistent CTA: warp 0 streams A (TMA; gated: another warp the up rows), warp
// 1 issues the MMAs, the next 4 or 8 are the epilogue (TMEM lane quarter =
// warp % 4), then those that bring B (boxes of 16 or 32 rows where a group's
// rows are consecutive, gather4 copies of four rows each where they come through
// the permutation), and one that hands out items.
// 256-row tiles are worked on by pairs of CTAs (cta_group::2).
// Where the host can tell that the items cannot fill the GPU, a cluster of KS
// CTAs shares an item along K (cluster_sum.cuh).
// Every wait is bounded (LMOE_ERR_TIMEOUT in the status word).
//
// Measured (896 experts, 3584 <-> 512): gate and up of 64 tokens 609 to 623 us
// (7.3 TB/s), of 8192 tokens 1072 to 1111 us by card (90 to 93% of the floor by
// bytes), weighted down of 64 and 8192 tokens 317 and 820 us.  With several
// hundred gathered rows an expert the copies of B bound it (8 experts x 1024 rows,
// 4096 x 4096: 200 us, 1.37 PFLOP/s; in expert order 1.55).
#include <cuda.h>
#include <cuda_bf16.h>

#include <type_traits>

#include "cluster_sum.cuh"
#include "lmoe_internal.cuh"
#include "tc_ptx.cuh"
#include "tensor_map.cuh"

namespace lmoe {
namespace {

using namespace tc;

constexpr uint32_t A_TILE = 128 * 128;  // 128 rows x 64 bf16

template <int NT, bool SWIGLU, bool GATHER, int KS>
struct GCfg {
    // Warps that bring B: one warp's gather4 copies, issued one after another,
    // held the chunks up (a gate/up pass of 8192 tokens over 896 experts took
    // 3.78 ms with one, 2.12 ms with two).
    static constexpr int BW = !GATHER || NT <= 32 ? 1 : NT == 64 ? 4 : 8;
    // Epilogue warps, one or two per TMEM lane quarter (two take 16-column chunks
    // in turn): with four, short reductions (K = 512) waited for the epilogue.
    static constexpr int EW = NT >= 128 ? 8 : 4;
    static constexpr int B0 = 2 + EW;  // the first warp that brings B
    static constexpr int A2 = B0 + BW;  // the second A warp (SWIGLU: the up rows)
    static constexpr int FEED = A2 + (SWIGLU ? 1 : 0);  // the warp that hands out items
    static constexpr int THREADS = 32 * (FEED + 1);
    static_assert(THREADS * 8 >= 2048, "the scan of the offsets takes 8 experts a thread");
    // The largest row tile is shared by a pair of CTAs (cta_group::2): 256
    // weight rows, each CTA bringing 128 of them and half of B.
    static constexpr bool PAIR = NT == 256;
    static constexpr int CL = PAIR ? 2 : KS;  // CTAs of a cluster
    static constexpr uint32_t B_TILE = (PAIR ? NT / 2 : NT) * 128;
    static constexpr int COPIES = (int(B_TILE) / 512 + BW - 1) / BW;  // gather4 copies a warp issues a chunk, at most
    static constexpr uint32_t STAGE = A_TILE + B_TILE;
    static constexpr int BOX = NT < 32 ? 16 : 32;  // rows of a B box
    static constexpr uint32_t RED = KS > 1 ? ClusterSum::red_bytes(NT) : 0;
    static constexpr int S_RAW = int((200 * 1024 - RED) / STAGE);
    static constexpr int S = S_RAW > 10 ? 10 : S_RAW;
    static constexpr int Q = 4;    // items handed out ahead
    static constexpr int CONSUMERS = (FEED + (PAIR ? FEED - 1 : 0));  // warps that take them (a pair's second MMA warp idles)
    static constexpr int ACC = 2;  // accumulators: an item's epilogue overlaps the next one's MMAs
    static constexpr uint32_t TMEM_COLS = ACC * NT < 32 ? 32 : ACC * NT;
};

struct GArgs {
    const int32_t *offsets, *perm;
    const float *row_w;
    const uint8_t *x;  // gathered rows' bytes
    int64_t P, x_rows, x_bytes;
    int E, k, N, MT, KC;
    int max_items;  // no valid groups have more
    int32_t *counter;  // items handed out so far (zero at the start); null: every CTA takes each grid-th
    void *out;
    int32_t *status;
    long long limit;
    int stall;
    int weights_once;  // most weight tiles have one row tile: their lines leave L2 first
};

struct GItem {
    int e, m, row0, nv;  // expert, weight tile, first row, rows
};

// Finds a CTA's items, in ascending order; every lane of a warp calls at().
template <int NT>
struct Walk {
    const int32_t *s_tiles, *s_off;
    int E, MT, e = 0;
    __device__ GItem at(int it)
    {
        const int t = it / MT;  // s_tiles[e] * MT <= it < s_tiles[e + 1] * MT
        const int lane = threadIdx.x & 31;
        for (;;) {
            const int c = e + 1 + lane;
            const unsigned b = __ballot_sync(0xFFFFFFFFu, c < E && s_tiles[c] <= t);
            const int n = __popc(b);
            e += n;
            if (n < 32) break;
            // far: in steps of 64 first (a step of 32 each from expert 0 took a first item of 896
            // experts up to 3 us)
            const int f = e + 64 * (lane + 1);
            e += 64 * __popc(__ballot_sync(0xFFFFFFFFu, f < E && s_tiles[f] <= t));
        }
        const int nt = s_tiles[e + 1] - s_tiles[e], l = it - s_tiles[e] * MT;
        GItem r;
        r.e = e;
        r.m = l / nt;
        const int n = l - r.m * nt;
        r.row0 = s_off[e] + n * NT;
        r.nv = min(NT, s_off[e + 1] - r.row0);
        return r;
    }
};

// F32: the output's type (else bf16).
template <int NT, bool SWIGLU, bool GATHER, int KS, bool F32>
__global__ void __launch_bounds__((GCfg<NT, SWIGLU, GATHER, KS>::THREADS), 1)
    k_grouped(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmA2,
              const __grid_constant__ CUtensorMap tmB, const GArgs p)
{
    using C = GCfg<NT, SWIGLU, GATHER, KS>;
    constexpr int S = C::S, THREADS = C::THREADS;
    constexpr bool PAIR = C::PAIR;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *stages = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float *red = reinterpret_cast<float *>(stages + S * C::STAGE);  // KS > 1 only
    uint64_t *full = reinterpret_cast<uint64_t *>(red + C::RED / 4);
    uint64_t *empty = full + S;
    uint64_t *acc_full = empty + S;
    uint64_t *acc_empty = acc_full + C::ACC;
    uint64_t *drain = acc_empty + C::ACC;
    uint64_t *red_full = drain + 1;
    uint64_t *item_full = red_full + 1;
    uint64_t *item_empty = item_full + C::Q;
    int32_t *s_item = reinterpret_cast<int32_t *>(item_empty + C::Q);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(s_item + C::Q);
    int32_t *warp_tot = reinterpret_cast<int32_t *>(tmem_slot + 2);
    int32_t *s_off = warp_tot + 32;
    int32_t *s_tiles = s_off + p.E + 1;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], C::BW + (SWIGLU ? 2 : 1));  // one arrival of each producer warp
            mbar_init(&empty[s], 1);
        }
        for (int a = 0; a < C::ACC; ++a) {
            mbar_init(&acc_full[a], 1);
            mbar_init(&acc_empty[a], 32 * C::EW * (PAIR ? 2 : 1));
        }
        mbar_init(drain, 1);
        mbar_init(red_full, 1);
        for (int i = 0; i < C::Q; ++i) {
            mbar_init(&item_full[i], 1);
            mbar_init(&item_empty[i], C::CONSUMERS);
        }
        mbar_init_fence();
    }
    if (warp == 0 && lane == 0) {
        prefetch_tensormap(&tmA);
        if (SWIGLU) prefetch_tensormap(&tmA2);
    }
    if (warp == C::B0 && lane == 0) prefetch_tensormap(&tmB);
    if (warp == 1) PAIR ? tmem_alloc_pair(tmem_slot, C::TMEM_COLS) : tmem_alloc(tmem_slot, C::TMEM_COLS);
    pdl_enter();
    if (GATHER) {
        // few rows: what the chain offsets -> perm -> x waits for next, on its way to L2
        const int64_t line = int64_t(blockIdx.x) * THREADS + threadIdx.x;
        if (p.P <= 32 * THREADS && threadIdx.x * 32 < p.P) prefetch_l2(p.perm + threadIdx.x * 32);
        if (p.x_bytes <= 1 << 20 && line * 128 < p.x_bytes) prefetch_l2(p.x + line * 128);
    }
    // Row tiles per expert, scanned, 8 experts a thread; a group that breaks
    // 0 <= o0 <= o1 <= P is empty and reported.
    bool bad = false;
    {
        const int e0 = threadIdx.x * 8;
        int o[9], cnt[8], sum = 0;
#pragma unroll
        for (int j = 0; j < 9; ++j) o[j] = e0 + j <= p.E ? __ldg(p.offsets + e0 + j) : 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const bool in = e0 + j < p.E, ok = o[j] >= 0 && o[j] <= o[j + 1] && o[j + 1] <= p.P;
            bad |= in && !ok;
            cnt[j] = in && ok ? (o[j + 1] - o[j] + NT - 1) / NT : 0;
            sum += cnt[j];
        }
        int incl = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, incl, d);
            if (lane >= d) incl += v;
        }
        if (lane == 31) warp_tot[warp] = incl;
        tc_fence_before();
        bad = __syncthreads_or(bad);
        tc_fence_after();
        int base = lane < warp ? warp_tot[lane] : 0;  // at most 32 warps
        base = __reduce_add_sync(0xFFFFFFFFu, base) + incl - sum;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (e0 + j <= p.E) {
                s_off[e0 + j] = o[j];
                s_tiles[e0 + j] = base;
            }
            base += cnt[j];
        }
        if (e0 + 8 == p.E && p.E == 8 * THREADS) {  // the one entry beyond the last thread's eight
            s_off[p.E] = o[8];
            s_tiles[p.E] = base;
        }
        __syncthreads();
    }
    if (C::CL > 1) cluster_sync();  // the cluster's barriers are initialised
    const uint32_t tmem = *tmem_slot;
    // Around a bad group others may overlap, so that there are more tiles than
    // any valid groups have: no more than those are worked off, and none where
    // the tile counts may have wrapped.
    int total = s_tiles[p.E] * p.MT;
    if (bad) {
        if (threadIdx.x == 0) set_status(p.status, LMOE_ERR_DEVICE_CHECK);
        const int64_t most = int64_t(p.E) * ceil_div(p.P, NT) * p.MT;
        total = most > INT32_MAX ? 0 : min(total, p.max_items);
    }
    const int rank = C::CL > 1 ? int(cluster_rank()) : 0;
    const int first = int(blockIdx.x) / C::CL, step = int(gridDim.x) / C::CL;
    // this rank's K chunks
    const int k0 = KS > 1 ? rank * p.KC / KS : 0, k1 = KS > 1 ? (rank + 1) * p.KC / KS : p.KC;
    Walk<NT> walk{s_tiles, s_off, p.E, p.MT};
    // This CTA's items, in order, NO_MORE after the last and LOST where the wait for
    // one ran out; every lane of a warp calls it.  Many items are handed out as
    // CTAs come free: SMs do not all stream equally fast, and groups differ (a
    // weighted down projection of 64 tokens over 896 experts: its CTAs ended
    // between 351 and 421 us with each grid-th item).
    constexpr int NO_MORE = -1, LOST = -2;
    int feed_q = 0, feed_next = first;
    uint32_t feed_phase = 0;
    auto next_item = [&]() -> int {
        if (!p.counter) {
            const int it = feed_next;
            feed_next += step;
            return it < total ? it : NO_MORE;
        }
        const bool ok = PAIR ? mbar_wait_cluster_warp(&item_full[feed_q], feed_phase, p.limit)
                             : mbar_wait_warp(&item_full[feed_q], feed_phase, p.limit);
        if (!ok) {
            if (lane == 0) set_status(p.status, LMOE_ERR_TIMEOUT);
            return LOST;
        }
        const int it = reinterpret_cast<volatile int32_t *>(s_item)[feed_q];
        __syncwarp();
        if (lane == 0)
            PAIR ? cluster_arrive_read(cluster_map(smem_u32(&item_empty[feed_q]), 0)) : mbar_arrive(&item_empty[feed_q]);
        if (++feed_q == C::Q) {
            feed_q = 0;
            feed_phase ^= 1;
        }
        return it;
    };

    // Copies still in flight after a timeout land before the CTA ends (bounded).
    // (A pair's copies all count in on the leader's barriers.)
    auto settle = [&](int fills) {
        if (PAIR && rank > 0) return;
        for (int f = fills > S ? fills - S : 0; f < fills; ++f) mbar_wait_warp(&full[f % S], (f / S) & 1, p.limit);
    };

    if (warp == 0 || (warp >= C::B0 && warp < C::FEED)) {
        // ---------------- producers: A (warp 0 and, gated, warp A2), B (warps B0 ..) ----------------
        __shared__ int4 s_ids[GATHER ? C::BW : 1][C::COPIES];  // the rows of the warps' gather4 copies
        const bool isA = warp == 0 || warp == C::A2;
        const uint64_t policy = isA && p.weights_once ? l2_policy_evict_first() : l2_policy_evict_normal();
        const int bw = warp - C::B0;  // B: this warp's copies are bw, bw + BW, ...
        [[maybe_unused]] int4 *ids = s_ids[GATHER && !isA ? bw : 0];
        int stage = 0, fills = 0;
        uint32_t phase = 0;
        bool ok = true;
        bool at_start = true;  // (the failure-path test withholds a CTA's first weight copy)
        for (; ok; at_start = false) {
            const int it = next_item();
            if (it < 0) {
                ok = it != LOST;
                break;
            }
            const GItem w = walk.at(it);
            // This CTA's rows of the tile: all, or a pair's half of them (rounded to whole
            // MMA columns).  A pair's second CTA does not arrive on the stage's barrier, so
            // each of its warps has to have a copy in every chunk, if only of padding:
            // one without could fall a whole turn of the ring behind the MMAs.
            const int half = PAIR ? (w.nv + 31) / 32 * 16 : 0;
            const int b0 = PAIR ? rank * half : 0;
            const int bn = PAIR ? max(0, min(half, w.nv - b0)) : w.nv;  // rows of the group among them
            const int copies = GATHER ? (PAIR ? max(half / 4, C::BW) : (bn + 3) / 4)
                                      : ((PAIR ? half : bn) + C::BOX - 1) / C::BOX;
            static_assert(!PAIR || C::B_TILE >= C::BW * 512, "room for a copy of each warp");
            const int mtile = PAIR ? 2 * w.m + rank : w.m;  // this CTA's 128 weight rows
            const int mine = copies > bw ? (copies - bw + C::BW - 1) / C::BW : 0;
            // bytes this warp's barrier arrival announces: a pair's leader those of both CTAs (an
            // arrival from the other CTA, with the release it needs, would take over 1000 cycles a stage)
            const uint32_t announce = (isA ? (SWIGLU ? A_TILE / 2 : A_TILE) : uint32_t(mine) * (GATHER ? 512u : C::BOX * 128u)) *
                                      (PAIR ? 2 : 1);
            if (GATHER && !isA) {
                __syncwarp();
                for (int i = lane; i < mine; i += 32) {
                    int r[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int l = 4 * (bw + C::BW * i) + j;
                        r[j] = 0;
                        if (l < bn) {
                            const int pr = __ldg(p.perm + w.row0 + b0 + l);
                            r[j] = pr / p.k;
                            if (pr < 0 || r[j] >= p.x_rows) {
                                set_status(p.status, LMOE_ERR_DEVICE_CHECK);
                                r[j] = 0;
                            }
                        }
                    }
                    ids[i] = make_int4(r[0], r[1], r[2], r[3]);
                }
                __syncwarp();
            }
            for (int kc = k0; kc < k1; ++kc) {
                ok = mbar_wait_warp(&empty[stage], phase ^ 1, p.limit);
                if (!ok) {
                    if (lane == 0) set_status(p.status, LMOE_ERR_TIMEOUT);
                    break;
                }
                uint8_t *sb = stages + stage * C::STAGE;
                // the barrier of this stage: a pair's is the leader's
                const uint32_t bar = PAIR ? cluster_map(smem_u32(&full[stage]), 0) : 0;
                auto expect = [&] {
                    if (!PAIR || rank == 0) mbar_arrive_expect_tx(&full[stage], announce);
                };
                auto load = [&](void *dst, const CUtensorMap *tm, int y) {
                    PAIR ? tma_load_2d_pair(dst, tm, kc * 64, y, bar, policy)
                         : tma_load_2d_hint(dst, tm, kc * 64, y, &full[stage], policy);
                };
                if (isA) {
                    if (elect_one() && !(p.stall && at_start && kc == k0)) {
                        if (SWIGLU) {
                            expect();
                            const CUtensorMap *tm = warp == 0 ? &tmA : &tmA2;
                            uint8_t *dst = sb + (warp == 0 ? 0 : 2048);
#pragma unroll
                            for (int j = 0; j < 4; ++j) load(dst + j * 4096, tm, w.e * p.N + mtile * 64 + 16 * j);
                        } else {
                            expect();
                            load(sb, &tmA, w.e * p.N + mtile * 128);
                        }
                    }
                } else {
                    if (elect_one()) {
                        expect();
                        for (int i = 0; i < mine; ++i) {
                            const int c = bw + C::BW * i;
                            if (!GATHER)
                                load(sb + A_TILE + c * C::BOX * 128, &tmB, w.row0 + b0 + c * C::BOX);
                            else if (PAIR)
                                tma_gather4_pair(sb + A_TILE + c * 512, &tmB, kc * 64, ids[i], bar);
                            else
                                tma_gather4(sb + A_TILE + c * 512, &tmB, kc * 64, ids[i], &full[stage]);
                        }
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
        if (!ok) settle(fills);
    } else if (warp == 1 && (!PAIR || rank == 0)) {
        // ---------------- MMA issuer (a pair's: the leader's) ----------------
        int stage = 0, acc = 0;
        uint32_t phase = 0, acc_phase = 0;
        bool ok = true;
        while (ok) {
            const int it = next_item();
            if (it < 0) {
                ok = it != LOST;
                break;
            }
            const GItem w = walk.at(it);
            const uint32_t id =
                PAIR ? idesc_bf16_pair(uint32_t((w.nv + 31) & ~31)) : idesc_bf16(uint32_t((w.nv + 15) & ~15));
            ok = mbar_wait_warp(&acc_empty[acc], acc_phase ^ 1, p.limit);
            tc_fence_after();
            const uint32_t d = tmem + uint32_t(acc * NT);
            for (int kc = k0; kc < k1 && ok; ++kc) {
                ok = mbar_wait_warp(&full[stage], phase, p.limit);
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
                    const uint8_t *sb = stages + stage * C::STAGE;
                    const uint64_t ad = sdesc_k128(smem_u32(sb)), bd = sdesc_k128(smem_u32(sb + A_TILE));
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)  // 4 x K = 16 per 128-byte row
                        if (PAIR)
                            mma_bf16_pair(d, ad + 2 * kk, bd + 2 * kk, id, (kc > k0 || kk > 0) ? 1u : 0u);
                        else
                            mma_bf16(d, ad + 2 * kk, bd + 2 * kk, id, (kc > k0 || kk > 0) ? 1u : 0u);
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
                PAIR ? tc_commit_pair(drain) : tc_commit(drain);  // this CTA's MMAs in flight end before the tensor memory is freed
                mbar_wait(drain, 0, p.limit);
            }
            __syncwarp();
        }
    } else if (warp >= 2 && warp < C::B0) {
        // ---------------- epilogue ----------------
        const int q = warp & 3;
        int acc = 0;
        uint32_t acc_phase = 0;
        const int half = (warp - 2) >> 2;  // which of the quarter's warps
        // lane l: pairs and weights of rows l, l + 32, .. of an item's tile.  Under the
        // output's traffic a load takes several microseconds, so an item's pairs are
        // requested two items ahead and its weights one.
        constexpr int NW = NT > 32 ? NT / 32 : 1;
        const bool weighted = !SWIGLU && p.row_w;
        auto take = [&](GItem &w, int (&pr)[NW]) -> bool {
            const int it = next_item();
            if (it < 0) return false;
            w = walk.at(it);
            if (weighted && p.perm)
#pragma unroll
                for (int i = 0; i < NW; ++i) pr[i] = __ldg(p.perm + w.row0 + min(32 * i + lane, w.nv - 1));
            return true;
        };
        auto weigh = [&](const GItem &w, const int (&pr)[NW], float (&rw)[NW]) {
            if (!weighted) return;
#pragma unroll
            for (int i = 0; i < NW; ++i) {
                const int q = p.perm ? pr[i] : w.row0 + min(32 * i + lane, w.nv - 1);
                const bool in = q >= 0 && q < p.P;
                if (!in) set_status(p.status, LMOE_ERR_DEVICE_CHECK);
                rw[i] = __ldg(p.row_w + (in ? q : 0));
            }
        };
        auto process = [&](const GItem &w, const float (&rw)[NW]) -> bool {
            if (!mbar_wait_warp(&acc_full[acc], acc_phase, p.limit)) {
                if (lane == 0) set_status(p.status, LMOE_ERR_TIMEOUT);
                return false;
            }
            tc_fence_after();
            const uint32_t tb = tmem + (uint32_t(32 * q) << 16) + uint32_t(acc * NT);
            // the lane's output column (gated: lanes 0-15 hold the gates of 16 features, 16-31 the ups)
            const int mtile = PAIR ? 2 * w.m + rank : w.m;
            const int n = SWIGLU ? mtile * 64 + 16 * q + (lane & 15) : mtile * 128 + 32 * q + lane;
            const bool mine = n < p.N;
            using Out = typename std::conditional<F32, float, __nv_bfloat16>::type;
            using Out2 = typename std::conditional<F32, float2, __nv_bfloat162>::type;
            const bool pairs = p.N % 2 == 0;  // neighbouring outputs in one store
            auto round1 = [](float v) -> Out {
                if constexpr (F32) return v;
                else return __float2bfloat16_rn(v);
            };
            auto round2 = [](float lo, float hi) -> Out2 {
                if constexpr (F32) return make_float2(lo, hi);
                else return __floats2bfloat162_rn(lo, hi);
            };
            // 16 rows from c0 on (rows [c0, c1) of them wanted) of the tile: weight or gate, round, store
            auto finish = [&](int c0, int c1, float (&y)[16]) {
                const int odd = lane & 1, up = lane >> 4;
                Out *const base = static_cast<Out *>(p.out) + int64_t(w.row0 + c0) * p.N;
                const int64_t N = p.N;
                if constexpr (SWIGLU) {
                    // both halves of the warp gate: lanes 0-15 the even rows, 16-31 the odd ones
                    float h[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float r = __shfl_xor_sync(0xFFFFFFFFu, up ? y[2 * i] : y[2 * i + 1], 16);
                        const float g = up ? r : y[2 * i], u = up ? y[2 * i + 1] : r;
                        // g sigmoid(g) by exp(-|g|), so that the divisor stays in [1, 2]: one beyond
                        // 2^126 (g < -87.3) would make the quick division's result 0
                        const float e = expf(-fabsf(g));
                        h[i] = __fdividef(g < 0.f ? g * e : g, 1.f + e) * u;
                    }
                    if (pairs) {
                        int row = c0 + 2 * odd + up;
                        Out *o = base + (2 * odd + up) * N + (n & ~1);
#pragma unroll
                        for (int i = 0; i < 8; i += 2, row += 4, o += 4 * N) {
                            const float r = __shfl_xor_sync(0xFFFFFFFFu, odd ? h[i] : h[i + 1], 1);
                            if (mine && row < c1)
                                *reinterpret_cast<Out2 *>(o) = odd ? round2(r, h[i + 1]) : round2(h[i], r);
                        }
                    } else {
                        int row = c0 + up;
                        Out *o = base + up * N + n;
#pragma unroll
                        for (int i = 0; i < 8; ++i, row += 2, o += 2 * N)
                            if (mine && row < c1) *o = round1(h[i]);
                    }
                    return;
                }
                if (p.row_w) {
                    float v = rw[0];
#pragma unroll
                    for (int i = 1; i < NW; ++i) v = c0 / 32 == i ? rw[i] : v;
#pragma unroll
                    for (int j = 0; j < 16; ++j) y[j] *= __shfl_sync(0xFFFFFFFFu, v, (c0 & 31) + j);
                }
                if (pairs) {  // even lanes store the even rows' pairs of columns, odd lanes the odd rows'
                    int row = c0 + odd;
                    Out *o = base + odd * N + (n & ~1);
#pragma unroll
                    for (int j = 0; j < 16; j += 2, row += 2, o += 2 * N) {
                        const float r = __shfl_xor_sync(0xFFFFFFFFu, odd ? y[j] : y[j + 1], 1);
                        if (mine && row < c1)
                            *reinterpret_cast<Out2 *>(o) = odd ? round2(r, y[j + 1]) : round2(y[j], r);
                    }
                } else {
                    Out *o = base + n;
#pragma unroll
                    for (int j = 0; j < 16; ++j, o += N)
                        if (mine && c0 + j < c1) *o = round1(y[j]);
                }
            };
            if (KS > 1) {
                static_assert(KS == 1 || NT == 16, "one chunk of columns");
                const ClusterSum cs(KS, rank, w.nv, reinterpret_cast<float *>(stages), red, red_full);
                uint32_t v[16];
                tmem_ld16(tb, v);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (j < w.nv) cs.stage[j * 128 + 32 * q + lane] = __uint_as_float(v[j]);
                if (!cs.exchange(p.limit)) {
                    if (lane == 0) set_status(p.status, LMOE_ERR_TIMEOUT);
                    return false;
                }
                const int c0 = cs.own0, c1 = cs.own1;  // this rank's rows
                float y[16];
                cs.sum(c0, 32 * q + lane, y);
                finish(c0, c1, y);
            } else {
                for (int c0 = 16 * half; c0 < w.nv; c0 += 4 * C::EW) {
                    uint32_t v[16];
                    tmem_ld16(tb + c0, v);
                    tmem_ld_wait();
                    float y[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) y[j] = __uint_as_float(v[j]);
                    finish(c0, w.nv, y);
                }
            }
            tc_fence_before();
            PAIR ? cluster_arrive_read(cluster_map(smem_u32(&acc_empty[acc]), 0)) : mbar_arrive(&acc_empty[acc]);
            if (++acc == C::ACC) {
                acc = 0;
                acc_phase ^= 1;
            }
            return true;
        };
        // w0 in hand with its weights, w1 with its pairs; weights in two sets by
        // turns, so that no copy waits for a load
        GItem w0, w1, w2;
        int pr[NW];
        float ra[NW], rb[NW];
        bool have0 = take(w0, pr), have1 = false, have2 = false;
        if (have0) {
            weigh(w0, pr, ra);
            have1 = take(w1, pr);
        }
        while (have0) {
            if (have1) weigh(w1, pr, rb);
            have2 = have1 && take(w2, pr);
            if (!process(w0, ra) || !have1) break;
            if (have2) weigh(w2, pr, ra);
            w0 = w2;
            const GItem cur = w1;
            have1 = have2 && take(w1, pr);
            if (!process(cur, rb)) break;
            have0 = have2;
        }
    } else if (warp == C::FEED && p.counter && rank == 0) {
        // ---------------- item feed (a pair's: the leader's, for both CTAs) ----------------
        int q = 0;
        uint32_t phase = 0;
        for (bool more = true; more;) {
            if (!mbar_wait_warp(&item_empty[q], phase ^ 1, p.limit)) {
                if (lane == 0) set_status(p.status, LMOE_ERR_TIMEOUT);
                break;
            }
            int it = 0;
            if (lane == 0) {
                it = atomicAdd(p.counter, 1);
                it = it < total ? it : NO_MORE;
                s_item[q] = it;
                if (PAIR) cluster_store_i32(cluster_map(smem_u32(&s_item[q]), 1), it);
                if (PAIR) cluster_arrive(cluster_map(smem_u32(&item_full[q]), 1));
                mbar_arrive(&item_full[q]);
            }
            more = __shfl_sync(0xFFFFFFFFu, it, 0) >= 0;
            if (++q == C::Q) {
                q = 0;
                phase ^= 1;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    // nobody's shared or tensor memory goes while another CTA may still write or read it
    if (C::CL > 1) cluster_sync_end();
    tc_fence_after();
    if (warp == 1) PAIR ? tmem_dealloc_pair(tmem, C::TMEM_COLS) : tmem_dealloc(tmem, C::TMEM_COLS);
}

template <int NT, bool SWIGLU, bool GATHER, int KS, bool F32 = false>
cudaError_t launch(const GroupedArgs &a, GArgs g, int64_t items, int sms, cudaStream_t st)
{
    using C = GCfg<NT, SWIGLU, GATHER, KS>;
    CUtensorMap ma, ma2, mb;
    if (!make_tensor_map(&ma, a.W, MapType::BF16, a.K, int64_t(a.E) * a.N, SWIGLU ? 16 : 128) ||
        !make_tensor_map(&ma2, SWIGLU ? a.W2 : a.W, MapType::BF16, a.K, int64_t(a.E) * a.N, SWIGLU ? 16 : 128) ||
        !make_tensor_map(&mb, a.x, MapType::BF16, a.K, a.x_rows, GATHER ? 1 : C::BOX))
        return cudaErrorInvalidValue;
    const size_t smem = 1024 + size_t(C::S) * C::STAGE + C::RED + (2 * C::S + 2 * C::ACC + 2 + 2 * C::Q) * 8 +
                        C::Q * 4 + 8 + 128 + size_t(2 * a.E + 2) * 4;
    auto *kern = k_grouped<NT, SWIGLU, GATHER, KS, F32>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e != cudaSuccess) return e;
    const int64_t slots = sms / C::CL;
    const unsigned grid = unsigned((items < slots ? items : slots) * C::CL);
    // At four items a CTA and more they are handed out by a counter (cleared
    // here; it costs a call a microsecond or two).
    if (KS == 1 && items >= 4 * slots) {
        e = cudaMemsetAsync(g.counter, 0, sizeof(int32_t), st);
        if (e != cudaSuccess) return e;
    } else {
        g.counter = nullptr;
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
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
    cfg.numAttrs = C::CL > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, ma, ma2, mb, g);
}

template <int NT, int KS>
cudaError_t pick(const GroupedArgs &a, const GArgs &g, int64_t items, int sms, cudaStream_t st)
{
    if (a.W2)
        return a.gather ? launch<NT, true, true, KS>(a, g, items, sms, st)
                        : launch<NT, true, false, KS>(a, g, items, sms, st);
    if (a.out_fmt == LMOE_F32)
        return a.gather ? launch<NT, false, true, KS, true>(a, g, items, sms, st)
                        : launch<NT, false, false, KS, true>(a, g, items, sms, st);
    return a.gather ? launch<NT, false, true, KS>(a, g, items, sms, st)
                    : launch<NT, false, false, KS>(a, g, items, sms, st);
}

}  // namespace

cudaError_t launch_grouped(const GroupedArgs &a, cudaStream_t st)
{
    GArgs g{};
    g.offsets = a.offsets;
    g.perm = a.perm;
    g.row_w = a.row_w;
    g.P = a.P;
    g.x_rows = a.x_rows;
    g.x = reinterpret_cast<const uint8_t *>(a.x);
    g.x_bytes = a.x_rows * a.K * 2;
    g.E = a.E;
    g.k = a.k;
    g.N = a.N;
    g.MT = int(ceil_div(a.N, a.W2 ? 64 : 128));
    g.KC = int(ceil_div(a.K, 64));
    g.out = a.out;
    g.status = a.status;
    g.counter = a.status + 1;  // the status word's neighbour in the workspace
    g.limit = a.wait.limit > 0 ? a.wait.limit : 4000000000LL;  // about 2 s of SM clocks
    g.stall = a.wait.stall_first_fill;
    // Row tile: the smallest that holds a group of average size and a quarter
    // more, so that most groups are one tile.
    const int64_t active = a.P < a.E ? a.P : a.E;
    const int64_t rows = ceil_div(a.P * 5, active * 4);
    const int NT = rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : rows <= 128 ? 128 : 256;
    // most tiles there can be, whatever the groups are
    if (NT == 256) g.MT = int(ceil_div(a.N, a.W2 ? 128 : 256));  // pairs of weight tiles
    const int64_t by_rows = (a.P + active * (NT - 1)) / NT;
    const int64_t items = (by_rows < a.P ? by_rows : a.P) * g.MT;
    if (items > INT32_MAX) return cudaErrorInvalidValue;
    g.max_items = int(items);
    // Weights read by one row tile each need no place in L2, gathered rows (read
    // by every weight tile) do.  896 experts, gate and up of 8192 tokens 1163 ->
    // 1094 us, down of 64 325 -> 317 us; with several row tiles an expert it
    // costs 1 to 2% (8 experts of 1024 rows 207 -> 210 us), and beside a large
    // row tile's fp32 output as much (down of 8192 tokens 921 -> 955 us).
    g.weights_once = a.P <= active * NT && (a.gather || NT < 256);
    const int sms = device_sms();
    if (NT == 16) {
        // Items that cannot fill the GPU: several CTAs along K an item, each at least 4 chunks.
        if (items * 8 <= sms && g.KC >= 32) return pick<16, 8>(a, g, items, sms, st);
        if (items * 4 <= sms && g.KC >= 16) return pick<16, 4>(a, g, items, sms, st);
        if (items * 2 <= sms && g.KC >= 8) return pick<16, 2>(a, g, items, sms, st);
        return pick<16, 1>(a, g, items, sms, st);
    }
    switch (NT) {
    case 32: return pick<32, 1>(a, g, items, sms, st);
    case 64: return pick<64, 1>(a, g, items, sms, st);
    case 128: return pick<128, 1>(a, g, items, sms, st);
    default: return pick<256, 1>(a, g, items, sms, st);
    }
}

}  // namespace lmoe
