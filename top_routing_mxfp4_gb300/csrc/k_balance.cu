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
// gradient written once.  HBM bounds it.
//
// A warp takes a row: a lane holds the same columns in every row it meets, so the
// sums over the tokens stay in its registers (fp32) until the end; each block
// writes its sums and a cluster adds the blocks' in order.  Integer atomics count
// (in shared memory; any order gives the same counts); nothing else is atomic, so
// a call repeats bit for bit.
#include "lmoe_internal.cuh"
#include "tc_ptx.cuh"

namespace lmoe {
namespace {

constexpr int kCountBlocks = 32;
// Up to this many picks every block counts them all by itself; more are counted by
// a kernel of their own.
constexpr int64_t kOwnCount = 16384;

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// Adds the picks p of [p0, P) in steps of `step` to the block's counts, and the
// tokens they belong to (those of slot 0) to *tokens.
__device__ __forceinline__ void count_picks(const BalanceArgs &a, int64_t p0, int64_t step, int32_t *s_counts,
                                            int32_t *s_tokens)
{
    const int64_t P = a.T * a.k;
    int tokens = 0;
    for (int64_t p = p0; p < P; p += step) {
        const int64_t t = int64_t(uint32_t(p) / uint32_t(a.k));
        if (a.mask && !a.mask[t]) continue;
        if (p == t * a.k) ++tokens;
        const int e = __ldg(a.idx + p);
        if (uint32_t(e) < uint32_t(a.E))
            atomicAdd(s_counts + e, 1);
        else
            set_status(a.status, LMOE_ERR_DEVICE_CHECK);
    }
    tokens = __reduce_add_sync(0xFFFFFFFFu, tokens);
    if ((threadIdx.x & 31) == 0 && tokens) atomicAdd(s_tokens, tokens);
}

// Many picks: the counts of kCountBlocks blocks, [block][E + 1] (the last: tokens).
__global__ void __launch_bounds__(1024) k_balance_count(const BalanceArgs a)
{
    extern __shared__ int32_t s_counts[];
    for (int e = threadIdx.x; e <= a.E; e += blockDim.x) s_counts[e] = 0;
    pdl_enter();
    __syncthreads();
    count_picks(a, int64_t(blockIdx.x) * blockDim.x + threadIdx.x, int64_t(gridDim.x) * blockDim.x, s_counts, s_counts + a.E);
    __syncthreads();
    int32_t *out = a.count_part + int64_t(blockIdx.x) * (a.E + 1);
    for (int e = threadIdx.x; e <= a.E; e += blockDim.x) out[e] = s_counts[e];
}

// A row's logits and the column sums in registers: half the warps beyond 1024 columns.
template <int NV>
constexpr int ROW_THREADS = NV <= 8 ? 512 : 256;

// NV: 128 columns each; VEC: E % 4 == 0, a lane's columns are fours of them.
// own: the block counts the picks itself.
template <int NV, bool VEC, bool GRAD>
__global__ void __launch_bounds__(ROW_THREADS<NV>, 1) k_balance_rows(const BalanceArgs a, bool own)
{
    constexpr int kBlock = ROW_THREADS<NV>, kWarps = kBlock / 32;
    extern __shared__ __align__(16) float s_mem[];
    const int Ep = (a.E + 3) & ~3;
    float *s_f = s_mem;                                             // [Ep]
    float *s_row = s_mem + Ep;                                      // [kWarps][Ep]
    int32_t *s_counts = reinterpret_cast<int32_t *>(s_row + kWarps * Ep);  // [E + 1]
    __shared__ float s_z[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float *mine = s_row + warp * Ep;
    for (int e = threadIdx.x; e <= a.E; e += kBlock) s_counts[e] = 0;
    for (int e = threadIdx.x; e < kWarps * Ep; e += kBlock) s_row[e] = 0.f;
    pdl_enter();
    __syncthreads();
    if (own) {
        count_picks(a, threadIdx.x, kBlock, s_counts, s_counts + a.E);
    } else {
        for (int e = threadIdx.x; e <= a.E; e += kBlock) {
            int32_t n = 0;
#pragma unroll 8
            for (int b = 0; b < kCountBlocks; ++b) n += a.count_part[int64_t(b) * (a.E + 1) + e];
            s_counts[e] = n;
        }
    }
    __syncthreads();
    const int tokens = s_counts[a.E];
    const float inv_n = tokens > 0 ? 1.f / float(tokens) : 0.f;
    const float scale = float(a.E) / float(a.k) * inv_n;
    for (int e = threadIdx.x; e < Ep; e += kBlock) s_f[e] = e < a.E ? float(s_counts[e]) * scale : 0.f;
    if (blockIdx.x == 0) {
        for (int e = threadIdx.x; e < a.E; e += kBlock) a.counts[e] = s_counts[e];
        if (threadIdx.x == 0) *a.tokens = tokens;
    }
    __syncthreads();

    const float up = GRAD && a.scale ? __ldg(a.scale) : 1.f;
    const float cb = GRAD ? up * a.coef_balance * inv_n : 0.f, cz = GRAD ? up * a.coef_z * 2.f * inv_n : 0.f;
    auto col = [&](int i) { return VEC ? ((i >> 2) * 32 + lane) * 4 + (i & 3) : i * 32 + lane; };
    auto each4 = [&](auto f) {  // the lane's columns, by fours of registers
#pragma unroll
        for (int i = 0; i < NV; ++i) f(i);
    };
    float acc[NV * 4];
#pragma unroll
    for (int i = 0; i < NV * 4; ++i) acc[i] = 0.f;
    float z = 0.f;
    for (int64_t t = int64_t(warp) * gridDim.x + blockIdx.x; t < a.T; t += int64_t(gridDim.x) * kWarps) {
        float v[NV * 4] = {};
        const float *l = a.logits + t * a.E;
        float *d = GRAD ? a.dlogits + t * a.E : nullptr;
        auto store = [&] {
            each4([&](int i) {
                if (VEC) {
                    if (col(4 * i) < a.E)
                        *reinterpret_cast<float4 *>(d + col(4 * i)) = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (col(4 * i + j) < a.E) d[col(4 * i + j)] = v[4 * i + j];
                }
            });
        };
        if (a.mask && !a.mask[t]) {
            if (GRAD) store();
            continue;
        }
        each4([&](int i) {
            if (VEC) {
                float4 q = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
                if (col(4 * i) < a.E) q = *reinterpret_cast<const float4 *>(l + col(4 * i));
                v[4 * i] = q.x, v[4 * i + 1] = q.y, v[4 * i + 2] = q.z, v[4 * i + 3] = q.w;
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) v[4 * i + j] = col(4 * i + j) < a.E ? l[col(4 * i + j)] : -INFINITY;
            }
        });
        // the slot's way through the gate weights
        if (GRAD && a.topk_w) {
            float w = 0.f, g = 0.f;
            int e = -1;
            if (lane < a.k) {
                e = __ldg(a.idx + t * a.k + lane);
                w = __ldg(a.topk_w + t * a.k + lane);
                g = __ldg(a.dtopk_w + t * a.k + lane);
                if (uint32_t(e) >= uint32_t(a.E)) e = -1;
            }
            const float s = warp_sum(w * g);
            g = w * (g - s);
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
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < NV * 4; ++i) m = fmaxf(m, v[i]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        // all -infinity: no probabilities (a NaN among them is no maximum, but makes the sum NaN)
        if (m == -INFINITY) m = 0.f;
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < NV * 4; ++i) {
            v[i] = expf(v[i] - m);
            s += v[i];
        }
        s = warp_sum(s);
        const float inv = s == 0.f ? 0.f : 1.f / s;
        const float lse = s == 0.f ? 0.f : m + logf(s);
        z = fmaf(lse, lse, z);
        float sf = 0.f;
        each4([&](int i) {
            float f[4] = {};
            if (GRAD) {
                if (VEC) {
                    if (col(4 * i) < a.E) {
                        const float4 q = *reinterpret_cast<const float4 *>(s_f + col(4 * i));
                        f[0] = q.x, f[1] = q.y, f[2] = q.z, f[3] = q.w;
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) f[j] = col(4 * i + j) < a.E ? s_f[col(4 * i + j)] : 0.f;
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[4 * i + j] *= inv;
                acc[4 * i + j] += v[4 * i + j];
                if (GRAD) sf = fmaf(f[j], v[4 * i + j], sf);
            }
        });
        if (!GRAD) continue;
        const float base = fmaf(-cb, warp_sum(sf), cz * lse);
        each4([&](int i) {
            float f[4] = {}, g[4] = {};
            if (VEC) {
                if (col(4 * i) < a.E) {
                    const float4 q = *reinterpret_cast<const float4 *>(s_f + col(4 * i));
                    f[0] = q.x, f[1] = q.y, f[2] = q.z, f[3] = q.w;
                    if (a.topk_w) {
                        const float4 r = *reinterpret_cast<const float4 *>(mine + col(4 * i));
                        g[0] = r.x, g[1] = r.y, g[2] = r.z, g[3] = r.w;
                    }
                }
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (col(4 * i + j) < a.E) {
                        f[j] = s_f[col(4 * i + j)];
                        g[j] = mine[col(4 * i + j)];
                    }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) v[4 * i + j] = fmaf(v[4 * i + j], fmaf(cb, f[j], base), g[j]);
        });
        store();
        if (a.topk_w) {
            __syncwarp();
            if (lane < a.k) {
                const int e = __ldg(a.idx + t * a.k + lane);
                if (uint32_t(e) < uint32_t(a.E)) mine[e] = 0.f;
            }
            __syncwarp();
        }
    }
    // the block's sums
#pragma unroll
    for (int i = 0; i < NV * 4; ++i)
        if (col(i) < a.E) mine[col(i)] = acc[i];
    if (lane == 0) s_z[warp] = z;
    __syncthreads();
    float *out = a.part + int64_t(blockIdx.x) * (a.E + 1);
    for (int e = threadIdx.x; e < a.E; e += kBlock) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v += s_row[w * Ep + e];
        out[e] = v;
    }
    if (threadIdx.x == 0) {
        float v = 0.f;
        for (int w = 0; w < kWarps; ++w) v += s_z[w];
        out[a.E] = v;
    }
}

// The blocks' sums added in order (within 16 strands, added in order), probs, and
// the losses.  One cluster: each CTA takes a share of the experts, rank 0 adds the
// shares of the loss.
constexpr int kFinalCtas = 8, kFinalWarps = 16;
__global__ void __cluster_dims__(kFinalCtas, 1, 1) __launch_bounds__(32 * kFinalWarps) k_balance_final(const BalanceArgs a, int blocks)
{
    __shared__ float s[kFinalWarps][33];
    __shared__ float s_loss[kFinalCtas];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rank = int(tc::cluster_rank());
    pdl_enter();
    const int tokens = *a.tokens;
    const float inv_n = tokens > 0 ? 1.f / float(tokens) : 0.f;
    const float scale = float(a.E) / float(a.k) * inv_n;
    float loss = 0.f;
    // column E holds the sums of lse^2
    for (int c0 = rank * 32; c0 <= a.E; c0 += kFinalCtas * 32) {
        const int c = c0 + lane;
        float v = 0.f;
        if (c <= a.E)
#pragma unroll 4
            for (int b = warp; b < blocks; b += kFinalWarps) v += a.part[int64_t(b) * (a.E + 1) + c];
        __syncthreads();
        s[warp][lane] = v;
        __syncthreads();
        if (warp == 0) {
            v = 0.f;
#pragma unroll
            for (int w = 0; w < kFinalWarps; ++w) v += s[w][lane];
            v *= inv_n;
            if (c < a.E) {
                a.probs[c] = v;
                loss = fmaf(float(a.counts[c]) * scale, v, loss);
            } else if (c == a.E) {
                a.loss[1] = v;
            }
        }
    }
    if (warp == 0) {
        loss = warp_sum(loss);
        if (lane == 0) tc::cluster_store_i32(tc::cluster_map(tc::smem_u32(&s_loss[rank]), 0), __float_as_int(loss));
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
cudaError_t rows(const BalanceArgs &a, unsigned grid, bool own, cudaStream_t st)
{
    const int Ep = (a.E + 3) & ~3;
    constexpr int kBlock = ROW_THREADS<NV>;
    const size_t smem = size_t(1 + kBlock / 32) * Ep * 4 + size_t(a.E + 1) * 4;
    auto *kern = k_balance_rows<NV, VEC, GRAD>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(grid), dim3(kBlock), smem, st, a, own);
}

template <int NV>
cudaError_t pick(const BalanceArgs &a, unsigned grid, bool own, cudaStream_t st)
{
    if (a.E % 4 == 0) return a.dlogits ? rows<NV, true, true>(a, grid, own, st) : rows<NV, true, false>(a, grid, own, st);
    return a.dlogits ? rows<NV, false, true>(a, grid, own, st) : rows<NV, false, false>(a, grid, own, st);
}

unsigned row_blocks(int64_t T)
{
    return unsigned(T < 152 ? (T > 0 ? T : 1) : 152);
}

size_t count_bytes(int64_t T, int E, int k)
{
    return T * k > kOwnCount ? size_t(round_up(int64_t(kCountBlocks) * (E + 1) * 4, 256)) : 0;
}

}  // namespace

// tokens (256 bytes) | counts of k_balance_count's blocks | sums of the row blocks
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
    const bool own = a.T * a.k <= kOwnCount;
    const unsigned grid = row_blocks(a.T);
    cudaError_t e = cudaSuccess;
    if (!own) e = launch_pdl(k_balance_count, dim3(kCountBlocks), dim3(1024), size_t(a.E + 1) * 4, st, a);
    if (e != cudaSuccess) return e;
    const int nv = int(ceil_div(a.E, 128));
    if (nv <= 2) e = pick<2>(a, grid, own, st);
    else if (nv <= 4) e = pick<4>(a, grid, own, st);
    else if (nv <= 7) e = pick<7>(a, grid, own, st);
    else e = pick<16>(a, grid, own, st);
    if (e != cudaSuccess) return e;
    return launch_pdl(k_balance_final, dim3(kFinalCtas), dim3(32 * kFinalWarps), 0, st, a, int(grid));
}

}  // namespace lmoe
