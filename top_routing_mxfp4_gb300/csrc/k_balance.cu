// Balance loss of a router, per-expert counts, and the gradient by the logits.
//
//   p = softmax(logits[t]),  f_e = counts_e E / (k N),  P_e = 1/N sum_t p_te
//   loss = ( sum_e f_e P_e,  1/N sum_t lse_t^2 )
//   dlogits_te = s (cb/N p_te (f_e - sum_j f_j p_tj) + cz 2/N lse_t p_te)
//                + sum over slots i of e: w_i (dw_i - sum_j w_j dw_j)
//
// The counts depend on the picks alone, which are a few percent of the logits'
// bytes: they are counted first, and then one pass over the logits gives the
// probabilities' sums and the whole gradient, each logit read once and each
// gradient written once.  HBM bounds it (32768 tokens of 896 experts, top 16, all outputs:
// 48.7 us of the 36 that the bytes take, 36 of them the pass over the logits; of 64 experts
// 17.6), and at few tokens the start and end of its launches (64 tokens 6.6).
//
// A warp takes a row: a lane holds the same columns in every row it meets, so the
// sums over the tokens stay in its registers (fp32) until the end; each block
// writes its sums and a cluster adds the blocks' in order.  Integer atomics count
// (in shared memory; any order gives the same counts); nothing else is atomic, so
// a call repeats bit for bit.
#include "act_fn.cuh"
#include "lmoe_internal.cuh"
#include "row_vec.cuh"
#include "tc_ptx.cuh"

namespace lmoe {
namespace {

constexpr int kCountCluster = 8, kCountParts = 16;
constexpr int kFinalCtas = 8;  // of the cluster that adds up the blocks' sums
// Up to this many picks every block counts them all by itself; more are counted by a kernel
// of their own.  us, by itself and by the kernel: 4096 picks of 896 experts 8.9 and 11.4, 8192
// 9.7 and 11.3, 12288 10.8 and 11.6, 16384 12.4 and 11.8; of 64 experts 12288 8.3 and 8.7,
// 16384 9.6 and 8.8; of 2048 experts 12288 16.3 and 17.4, 16384 17.8 and 17.4.
constexpr int64_t kOwnCount = 12288;
// Up to this many tokens are the work of one cluster, which needs no second kernel.  us, one
// cluster and two kernels: of 896 experts 64 tokens 6.2 and 7.5, 128 7.5 and 7.8, 192 8.3 and
// 7.9, 256 10.3 and 8.9; of 2048 experts 128 11.1 and 12.9, 192 17.3 and 17.4, 256 19.4 and 17.3;
// of 64 experts 128 5.4 and 6.6, 256 6.2 and 6.8.
constexpr int64_t kOneCluster = 128;

__device__ __forceinline__ float warp_max(float v)
{
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(v) : "f"(v));
    return v;
}
__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// Adds the picks p of [p0, P) in steps of `step` to the block's counts, and the
// tokens they belong to (those of slot 0) to *tokens.  Eight picks' loads at a time.
__device__ __forceinline__ void count_picks(const BalanceArgs &a, int64_t p0, int64_t step, int32_t *s_counts,
                                            int32_t *s_tokens)
{
    const int64_t P = a.T * a.k;
    int tokens = 0;
    for (int64_t p = p0; p < P; p += 8 * step) {
        int e[8];
        bool in[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t q = p + i * step;
            in[i] = q < P;
            e[i] = in[i] ? __ldg(a.idx + q) : 0;
            const uint32_t t = uint32_t(q) / uint32_t(a.k);
            if (in[i] && a.mask) in[i] = __ldg(a.mask + t) != 0;
            tokens += in[i] && uint32_t(q) == t * uint32_t(a.k);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (!in[i]) continue;
            if (uint32_t(e[i]) < uint32_t(a.E))
                atomicAdd(s_counts + e[i], 1);
            else
                set_status(a.status, LMOE_ERR_DEVICE_CHECK);
        }
    }
    tokens = __reduce_add_sync(0xFFFFFFFFu, tokens);
    if ((threadIdx.x & 31) == 0 && tokens) atomicAdd(s_tokens, tokens);
}

// Rows of counts lie this many apart: the experts', the tokens, whole 16 bytes.
__host__ __device__ constexpr int count_stride(int E) { return (E + 4) & ~3; }

// Many picks: the counts of kCountParts clusters (the entry behind the experts: tokens).
// A cluster's CTAs count for themselves, then each adds up a share of the experts.
__global__ void __cluster_dims__(kCountCluster, 1, 1) __launch_bounds__(512) k_balance_count(const BalanceArgs a)
{
    extern __shared__ int32_t s_counts[];
    const int Cs = count_stride(a.E), rank = int(tc::cluster_rank());
    for (int e = threadIdx.x; e < Cs; e += blockDim.x) s_counts[e] = 0;
    pdl_enter();
    __syncthreads();
    count_picks(a, int64_t(blockIdx.x) * blockDim.x + threadIdx.x, int64_t(gridDim.x) * blockDim.x, s_counts, s_counts + a.E);
    __syncthreads();
    tc::cluster_sync();
    int32_t *out = a.count_part + int64_t(blockIdx.x / kCountCluster) * Cs;
    for (int e = rank * int(blockDim.x) + threadIdx.x; e < Cs; e += kCountCluster * int(blockDim.x)) {
        int n = 0;
#pragma unroll
        for (int r = 0; r < kCountCluster; ++r) n += tc::cluster_load_i32(tc::cluster_map(tc::smem_u32(s_counts + e), r));
        out[e] = n;
    }
    __syncthreads();
    tc::cluster_sync_end();  // no CTA's counts go while another reads them
}

// A row's logits, the next row's and the column sums in registers: fewer warps for wider rows.
// 32768 tokens, us: of 256 experts, 512, 768, 1024 threads 21.8, 21.1, 22.7; of 384, 512, 640, 768
// threads 26.7, 28.6, 29.4; of 896, 320, 384, 448, 512, 576 threads 49.9, 48.1, 49.1, 50.2, 68.7
// (which spills); 14000 of 2048, 192, 256, 320 threads 54.0, 52.5, 90 (spills).
template <int NV>
constexpr int ROW_THREADS = NV <= 2 ? 768 : NV <= 4 ? 512 : NV <= 8 ? 384 : 256;

// NV: 128 columns each; VEC: E % 4 == 0, a lane's columns are fours of them.
// own: the block counts the picks itself.  one: the grid is one cluster, which adds up its
// blocks' sums itself.
template <int NV, bool VEC, bool GRAD>
__global__ void __launch_bounds__(ROW_THREADS<NV>, 1) k_balance_rows(const BalanceArgs a, bool own, bool one)
{
    constexpr int kBlock = ROW_THREADS<NV>, kWarps = kBlock / 32;
    extern __shared__ __align__(16) float s_mem[];
    const int Ep = (a.E + 3) & ~3, Cs = count_stride(a.E);
    float *s_f = s_mem;                                             // [Ep]: scale * coef_balance / N * f
    float *s_row = s_mem + Ep;                                      // [kWarps][Ep]
    int32_t *s_counts = reinterpret_cast<int32_t *>(s_row + kWarps * Ep);  // [Cs]
    __shared__ float s_z[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float *mine = s_row + warp * Ep;
    for (int e = threadIdx.x; e < Cs; e += kBlock) s_counts[e] = 0;
    if (GRAD && a.topk_w)
        for (int e = threadIdx.x; e < kWarps * Ep; e += kBlock) s_row[e] = 0.f;
    pdl_enter();
    // a lane's columns: fours of consecutive ones, or (E % 4) single ones, 32 lanes apart
    auto col = [&](int i) { return VEC ? ((i >> 2) * 32 + lane) * 4 + (i & 3) : i * 32 + lane; };
    auto get4 = [&](const float *p, int i, float none, float (&q)[4]) {  // the lane's i-th four of a row
        if (VEC) {
            float4 r = make_float4(none, none, none, none);
            if (col(4 * i) < a.E) r = *reinterpret_cast<const float4 *>(p + col(4 * i));
            q[0] = r.x, q[1] = r.y, q[2] = r.z, q[3] = r.w;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) q[j] = col(4 * i + j) < a.E ? p[col(4 * i + j)] : none;
        }
    };
    auto put4 = [&](float *p, int i, const float (&q)[4]) {
        if (VEC) {
            if (col(4 * i) < a.E) *reinterpret_cast<float4 *>(p + col(4 * i)) = make_float4(q[0], q[1], q[2], q[3]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (col(4 * i + j) < a.E) p[col(4 * i + j)] = q[j];
        }
    };
    const int64_t step = int64_t(gridDim.x) * kWarps;
    auto counts_in = [&](int64_t t) { return t >= a.T ? 0u : a.mask ? uint32_t(__ldg(a.mask + t)) : 1u; };
    // what a row needs, on its way while the row before is worked on (and not looked at before:
    // with the ids checked and the mask compared where they are loaded a warp waited for them)
    float next[NV * 4];
    int ne = -1;
    float nw = 0.f, ng = 0.f;
    auto load = [&](int64_t t) {
        const float *l = a.logits + t * a.E;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float q[4];
            get4(l, i, -INFINITY, q);
#pragma unroll
            for (int j = 0; j < 4; ++j) next[4 * i + j] = q[j];
        }
        if (GRAD && a.topk_w && lane < a.k) {
            ne = __ldg(a.idx + t * a.k + lane);
            nw = __ldg(a.topk_w + t * a.k + lane);
            ng = __ldg(a.dtopk_w + t * a.k + lane);
        }
    };
    // the first row, before the counts
    int64_t t = int64_t(warp) * gridDim.x + blockIdx.x;
    uint32_t in = counts_in(t), in_next = counts_in(t + step);
    if (in) load(t);
    __syncthreads();
    if (own) {
        count_picks(a, threadIdx.x, kBlock, s_counts, s_counts + a.E);
    } else {
        // four experts a thread, eight parts' counts at a time
        for (int i = threadIdx.x; i < Cs / 4 * (kCountParts / 8); i += kBlock) {
            const int e = i % (Cs / 4) * 4, b = i / (Cs / 4) * 8;
            int4 n = make_int4(0, 0, 0, 0);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int4 q = *reinterpret_cast<const int4 *>(a.count_part + int64_t(b + j) * Cs + e);
                n.x += q.x, n.y += q.y, n.z += q.z, n.w += q.w;
            }
            atomicAdd(s_counts + e, n.x);
            atomicAdd(s_counts + e + 1, n.y);
            atomicAdd(s_counts + e + 2, n.z);
            atomicAdd(s_counts + e + 3, n.w);
        }
    }
    const float up = GRAD && a.scale ? __ldg(a.scale) : 1.f;
    __syncthreads();
    const int tokens = s_counts[a.E];
    const float inv_n = tokens > 0 ? 1.f / float(tokens) : 0.f;
    const float cb = GRAD ? up * a.coef_balance * inv_n * (float(a.E) / float(a.k) * inv_n) : 0.f;
    const float cz = GRAD ? up * a.coef_z * 2.f * inv_n : 0.f;
    if (GRAD)
        for (int e = threadIdx.x; e < Ep; e += kBlock) s_f[e] = e < a.E ? float(s_counts[e]) * cb : 0.f;
    if (blockIdx.x == 0) {
        for (int e = threadIdx.x; e < a.E; e += kBlock) a.counts[e] = s_counts[e];
        if (threadIdx.x == 0) *a.tokens = tokens;
    }
    __syncthreads();

    F2 acc[NV * 2];
#pragma unroll
    for (int i = 0; i < NV * 2; ++i) acc[i] = f2(0.f);
    float z = 0.f;
    for (; t < a.T; t += step) {
        float *d = GRAD ? a.dlogits + t * a.E : nullptr;
        const uint32_t in_after = counts_in(t + 2 * step);
        F2 v[NV * 2];
        float m = -INFINITY;
        int e = -1;
        float w = 0.f, g = 0.f;
        if (in) {
#pragma unroll
            for (int i = 0; i < NV * 2; ++i) {
                v[i] = f2(next[2 * i], next[2 * i + 1]);
                m = fmaxf(m, fmaxf(next[2 * i], next[2 * i + 1]));
            }
            e = uint32_t(ne) < uint32_t(a.E) ? ne : -1, w = nw, g = ng;
        }
        if (in_next) load(t + step);
        const bool here = in != 0;
        in = in_next;
        in_next = in_after;
        if (!here) {
            if (GRAD) {
                const float none[4] = {};
#pragma unroll
                for (int i = 0; i < NV; ++i) put4(d, i, none);
            }
            continue;
        }
        m = warp_max(m);
        // all -infinity: no probabilities (a NaN among them is no maximum, but makes the sum NaN)
        if (m == -INFINITY) m = 0.f;
        // (the difference first: its terms times log2 e could overflow)
        const F2 l2e = f2(LOG2E), off = f2(-m);
        F2 s2 = f2(0.f), f2s = f2(0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float q[4];
            f2_get((v[2 * i] + off) * l2e, q[0], q[1]);
            f2_get((v[2 * i + 1] + off) * l2e, q[2], q[3]);
            v[2 * i] = f2(exp2_quick(q[0]), exp2_quick(q[1]));
            v[2 * i + 1] = f2(exp2_quick(q[2]), exp2_quick(q[3]));
            s2 = s2 + (v[2 * i] + v[2 * i + 1]);
            if (GRAD) {
                get4(s_f, i, 0.f, q);
                f2s = fma2(f2(q[0], q[1]), v[2 * i], fma2(f2(q[2], q[3]), v[2 * i + 1], f2s));
            }
        }
        // the sums of the exponentials, of f times them, and of the slots' w dw
        const bool gate = GRAD && a.topk_w;
        float s, sf = 0.f, sg = 0.f;
        if (GRAD) {
            if (gate) sg = warp_sum(w * g);
            const float2 both = warp_sum2(f2_sum(s2), f2_sum(f2s));
            s = both.x, sf = both.y;
        } else {
            s = warp_sum(f2_sum(s2));
        }
        if (gate) {
            g = w * (g - sg);
            const unsigned same = __match_any_sync(0xFFFFFFFFu, e);
            if (__any_sync(0xFFFFFFFFu, e >= 0 && (same & (same - 1)))) {  // an expert twice: one slot after another
                for (int j = 0; j < a.k; ++j) {
                    if (lane == j && e >= 0) mine[e] += g;
                    __syncwarp();
                }
            } else if (e >= 0) {
                mine[e] = g;
            }
            __syncwarp();
        }
        const float inv = s == 0.f ? 0.f : 1.f / s;
        const float lse = s == 0.f ? 0.f : m + logf(s);
        z = fmaf(lse, lse, z);
        const F2 inv2 = f2(inv), base = f2(fmaf(cz, lse, -sf * inv));
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            acc[2 * i] = fma2(v[2 * i], inv2, acc[2 * i]);
            acc[2 * i + 1] = fma2(v[2 * i + 1], inv2, acc[2 * i + 1]);
            if (!GRAD) continue;
            const F2 p0 = v[2 * i] * inv2, p1 = v[2 * i + 1] * inv2;
            float f[4], q[4] = {};
            get4(s_f, i, 0.f, f);
            if (gate) get4(mine, i, 0.f, q);
            f2_get(fma2(p0, f2(f[0], f[1]) + base, f2(q[0], q[1])), q[0], q[1]);
            f2_get(fma2(p1, f2(f[2], f[3]) + base, f2(q[2], q[3])), q[2], q[3]);
            put4(d, i, q);
        }
        if (gate) {
            __syncwarp();
            if (e >= 0) mine[e] = 0.f;
            __syncwarp();
        }
    }
    // the block's sums
#pragma unroll
    for (int i = 0; i < NV * 2; ++i) {
        float lo, hi;
        f2_get(acc[i], lo, hi);
        if (col(2 * i) < a.E) mine[col(2 * i)] = lo;
        if (col(2 * i + 1) < a.E) mine[col(2 * i + 1)] = hi;
    }
    if (lane == 0) s_z[warp] = z;
    __syncthreads();
    float zs = 0.f;
    if (threadIdx.x == 0)
        for (int w = 0; w < kWarps; ++w) zs += s_z[w];
    float *out = one ? s_f : a.part + int64_t(blockIdx.x) * (a.E + 1);
    for (int e = threadIdx.x; e < a.E; e += kBlock) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v += s_row[w * Ep + e];
        out[e] = v;
    }
    if (!one) {
        if (threadIdx.x == 0) out[a.E] = zs;
        return;
    }
    __shared__ float s_loss[2][kFinalCtas];  // rank 0's: the ranks' shares
    const int rank = int(tc::cluster_rank());
    auto at_rank0 = [&](float *p) { return tc::cluster_map(tc::smem_u32(p), 0); };
    __syncthreads();
    tc::cluster_sync();
    float loss = 0.f;
    const float scale = float(a.E) / float(a.k) * inv_n;
    for (int e = rank * kBlock + threadIdx.x; e < a.E; e += kFinalCtas * kBlock) {
        float v = 0.f;
#pragma unroll
        for (int r = 0; r < kFinalCtas; ++r) v += __int_as_float(tc::cluster_load_i32(tc::cluster_map(tc::smem_u32(s_f + e), r)));
        v *= inv_n;
        a.probs[e] = v;
        loss = fmaf(float(s_counts[e]) * scale, v, loss);
    }
    loss = warp_sum(loss);
    if (lane == 0) s_z[warp] = loss;
    __syncthreads();
    if (threadIdx.x == 0) {
        loss = 0.f;
        for (int w = 0; w < kWarps; ++w) loss += s_z[w];
        tc::cluster_store_i32(at_rank0(&s_loss[0][rank]), __float_as_int(loss));
        tc::cluster_store_i32(at_rank0(&s_loss[1][rank]), __float_as_int(zs * inv_n));
    }
    __syncthreads();
    tc::cluster_sync();  // (and no CTA's sums go while another reads them)
    if (rank == 0 && threadIdx.x < 2) {
        loss = 0.f;
#pragma unroll
        for (int r = 0; r < kFinalCtas; ++r) loss += s_loss[threadIdx.x][r];
        a.loss[threadIdx.x] = loss;
    }
}

// The blocks' sums added in order (within strands, added in order), probs, and the losses.
// One cluster: each CTA takes COLS columns at a time, L of a strand's loads in flight; rank
// 0 adds the CTAs' shares of the loss.  Few columns are shared by all the CTAs, with more
// strands (5000 tokens of 200 experts 11.5 against 13.9 us).
constexpr int kFinalThreads = 1024;
template <int COLS, int L>
__global__ void __cluster_dims__(kFinalCtas, 1, 1) __launch_bounds__(kFinalThreads) k_balance_final(const BalanceArgs a, int blocks)
{
    constexpr int STRANDS = kFinalThreads / COLS;
    __shared__ float s[STRANDS][COLS + 1];
    __shared__ float s_warp[COLS / 32], s_loss[kFinalCtas];
    const int at = threadIdx.x % COLS, strand = threadIdx.x / COLS;
    const int rank = int(tc::cluster_rank());
    tc::cluster_sync();  // rank 0 runs before another rank stores into its shared memory; while the kernel before ends
    pdl_enter();
    const int tokens = *a.tokens;
    const float inv_n = tokens > 0 ? 1.f / float(tokens) : 0.f;
    const float scale = float(a.E) / float(a.k) * inv_n;
    float loss = 0.f;
    // column E holds the sums of lse^2
    for (int c = rank * COLS + at; c - at <= a.E; c += kFinalCtas * COLS) {
        const int n = strand == 0 && c < a.E ? a.counts[c] : 0;
        float v = 0.f;
        if (c <= a.E)
            for (int b = strand; b < blocks; b += L * STRANDS) {
                float q[L];
#pragma unroll
                for (int i = 0; i < L; ++i) q[i] = b + i * STRANDS < blocks ? a.part[int64_t(b + i * STRANDS) * (a.E + 1) + c] : 0.f;
#pragma unroll
                for (int i = 0; i < L; ++i) v += q[i];
            }
        s[strand][at] = v;
        __syncthreads();
        if (strand == 0) {
#pragma unroll
            for (int q = 1; q < STRANDS; ++q) v += s[q][at];
            v *= inv_n;
            if (c < a.E) {
                a.probs[c] = v;
                loss = fmaf(float(n) * scale, v, loss);
            } else if (c == a.E) {
                a.loss[1] = v;
            }
        }
        __syncthreads();
    }
    if (strand == 0) {
        loss = warp_sum(loss);
        if (at % 32 == 0) s_warp[at / 32] = loss;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        loss = 0.f;
        for (int q = 0; q < COLS / 32; ++q) loss += s_warp[q];
        tc::cluster_store_i32(tc::cluster_map(tc::smem_u32(&s_loss[rank]), 0), __float_as_int(loss));
    }
    __syncthreads();
    tc::cluster_sync();
    if (rank == 0 && threadIdx.x == 0) {
        loss = 0.f;
#pragma unroll
        for (int r = 0; r < kFinalCtas; ++r) loss += s_loss[r];
        a.loss[0] = loss;
    }
}

template <int NV, bool VEC, bool GRAD>
cudaError_t rows(const BalanceArgs &a, unsigned grid, bool own, bool one, cudaStream_t st)
{
    constexpr int kBlock = ROW_THREADS<NV>;
    constexpr auto bytes = [](int E) { return size_t(1 + kBlock / 32) * ((E + 3) & ~3) * 4 + size_t(count_stride(E)) * 4; };
    const size_t smem = bytes(a.E);
    auto *kern = k_balance_rows<NV, VEC, GRAD>;
    // the most of any width: another host thread's narrower call does not lower it before this launch
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(bytes(NV * 128)));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kBlock);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kFinalCtas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = one ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, a, own, one);
}

template <int NV>
cudaError_t pick(const BalanceArgs &a, unsigned grid, bool own, bool one, cudaStream_t st)
{
    if (a.E % 4 == 0)
        return a.dlogits ? rows<NV, true, true>(a, grid, own, one, st) : rows<NV, true, false>(a, grid, own, one, st);
    return a.dlogits ? rows<NV, false, true>(a, grid, own, one, st) : rows<NV, false, false>(a, grid, own, one, st);
}

// Few rows are the work of one cluster, which needs no second kernel.
bool one_cluster(int64_t T) { return T <= kOneCluster; }

unsigned row_blocks(int64_t T)
{
    return one_cluster(T) ? unsigned(kFinalCtas) : unsigned(T < 152 ? T : 152);
}

size_t count_bytes(int64_t T, int E, int k)
{
    return T * k > kOwnCount ? size_t(round_up(int64_t(kCountParts) * count_stride(E) * 4, 256)) : 0;
}

}  // namespace

// tokens (256 bytes) | counts of k_balance_count's parts | sums of the row blocks
size_t balance_scratch_bytes(int64_t T, int E, int k)
{
    return 256 + count_bytes(T, E, k) + size_t(row_blocks(T)) * size_t(E + 1) * 4;
}

cudaError_t launch_balance(BalanceArgs a, void *scratch, cudaStream_t st)
{
    char *s = static_cast<char *>(scratch);
    a.tokens = reinterpret_cast<int32_t *>(s);
    a.count_part = reinterpret_cast<int32_t *>(s + 256);
    a.part = reinterpret_cast<float *>(s + 256 + count_bytes(a.T, a.E, a.k));
    const bool own = a.T * a.k <= kOwnCount, one = one_cluster(a.T);
    const unsigned grid = row_blocks(a.T);
    cudaError_t e = cudaSuccess;
    if (!own)
        e = launch_pdl(k_balance_count, dim3(kCountParts * kCountCluster), dim3(512), size_t(count_stride(a.E)) * 4, st, a);
    if (e != cudaSuccess) return e;
    const int nv = int(ceil_div(a.E, 128));
    if (nv <= 1) e = pick<1>(a, grid, own, one, st);
    else if (nv <= 2) e = pick<2>(a, grid, own, one, st);
    else if (nv <= 4) e = pick<4>(a, grid, own, one, st);
    else if (nv <= 7) e = pick<7>(a, grid, own, one, st);
    else if (nv <= 8) e = pick<8>(a, grid, own, one, st);
    else e = pick<16>(a, grid, own, one, st);
    if (e != cudaSuccess || one) return e;
    return launch_pdl(a.E < 256 ? k_balance_final<32, 10> : k_balance_final<128, 20>, dim3(kFinalCtas), dim3(kFinalThreads), 0, st, a,
                      int(grid));
}

}  // namespace lmoe
