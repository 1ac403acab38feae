// Sums of a cluster's accumulators, for items split along K: each of the KS
// CTAs holds [columns][128] fp32 partial sums of the same output tile, and each
// adds up a contiguous share of the columns, in rank order, so the result does
// not depend on which rank comes first.
//
// Every rank stages its sums in its own shared memory (the pipeline's ring,
// idle once the item's products are done; one item a cluster) and sends each
// other rank its columns with one bulk copy; scalar stores into another CTA's
// shared memory took several times as long (64 columns: 23.6 against 13 us for
// a whole call).
#pragma once
#include "tc_ptx.cuh"

namespace lmoe {

struct ClusterSum {
    int KS, rank, cols, share;  // cols: columns of the tile that hold rows; share: columns a rank adds
    int own0, own1;             // this rank's columns
    float *stage;               // [cols][128], this rank's sums
    float *red;                 // [KS - 1][own][128], the other ranks' sums of this rank's columns
    uint64_t *bar;              // its one arrival: the expecting thread's

    __device__ ClusterSum(int KS_, int rank_, int cols_, float *stage_, float *red_, uint64_t *bar_)
        : KS(KS_), rank(rank_), cols(cols_), share((cols_ + KS_ - 1) / KS_), stage(stage_), red(red_), bar(bar_)
    {
        own0 = begin(rank);
        own1 = begin(rank + 1);
    }
    // Rank t's columns: [begin(t), begin(t + 1)).
    __device__ int begin(int t) const { return min(cols, t * share); }
    // Bytes of `red` a tile of at most max_cols columns needs, for any KS <= 8.
    static constexpr uint32_t red_bytes(int max_cols) { return uint32_t(max_cols + 8) * 512; }

    // By the 128 epilogue threads (named barrier 1), all columns staged: send,
    // and wait for the others'.  False on timeout (one answer a warp).
    __device__ bool exchange(long long limit) const
    {
        tc::fence_async_shared();
        asm volatile("bar.sync 1, 128;" ::: "memory");
        if (threadIdx.x == 64) {
            tc::mbar_arrive_expect_tx(bar, uint32_t(KS - 1) * (own1 - own0) * 512);
            for (int i = 1; i < KS; ++i) {
                const int t = rank + i < KS ? rank + i : rank + i - KS, n = begin(t + 1) - begin(t), slot = rank < t ? rank : rank - 1;
                if (n > 0)
                    tc::cluster_copy(tc::cluster_map(tc::smem_u32(red + slot * n * 128), t), stage + begin(t) * 128,
                                     n * 512, tc::cluster_map(tc::smem_u32(bar), t));
            }
        }
        __syncwarp();
        return tc::mbar_wait_warp(bar, 0, limit);
    }
    // The sums of columns [c0, min(c0 + CW, end)) (this rank's) and row `row` of the tile.
    template <int CW>
    __device__ void sum(int c0, int row, float (&y)[CW]) const
    {
        const int own = own1 - own0;
#pragma unroll
        for (int j = 0; j < CW; ++j) y[j] = 0.f;
        for (int r = 0; r < KS; ++r) {
            const float *part = (r == rank ? stage + c0 * 128 : red + ((r < rank ? r : r - 1) * own + c0 - own0) * 128) + row;
#pragma unroll
            for (int j = 0; j < CW; ++j)
                if (c0 + j < own1) y[j] += part[j * 128];
        }
    }
};

}  // namespace lmoe
