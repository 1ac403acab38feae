// Layer norm and its gradients.
//
//   m = mean(x),  s = rsqrt(mean((x - m)^2) + eps),  out = bf16( (x - m) s w + b )
//   h = (x - m) s,  g = dy w
//   dx = s (g - mean(g) - h mean(g h)) (+ add),   dw = sum_t dy h,   db = sum_t dy
//
// Forward: a row's elements stay in registers between the two statistics (the
// squares are those of the centred values), so x is read once and out written
// once.
//
// Backward: the sums over a row want the row's threads, the sums over the rows a
// thread that stays with its columns.  Persistent blocks do both in one pass: a
// warp (up to 512 columns) or a block (up to 8192) walks over rows, each thread
// always on the same 16 columns, whose w and shares of dw and db it keeps in
// registers; at the end each block writes its shares, and a second kernel adds the
// blocks' in order.  Wider rows take the column sums in a pass of their own.
//
// HBM bounds them where rows are many, but only with few instructions an element:
// packed fp32 arithmetic (two a lane), the two row sums reduced together, and rows on
// their way early (8192 bf16 rows of 7168 with add: a block a row without any of it
// 122 us; a ring of cp.async copies 118; w, h and g kept and packed arithmetic 113;
// four rows of ring 81, 5.9 TB/s, 86% of HBM; fp32 rows 143, 85%).  At few rows the two
// kernels' starts and ends are most of the time (64 rows of 7168: 8 us).
#include <algorithm>

#include "lmoe_internal.cuh"
#include "row_vec.cuh"

namespace lmoe {
namespace {

// Columns up to which a warp takes a row backward.  At 1024 its sums spill (8192 rows: 47 us, a
// block a row 29).  At 257 to 512 fp32 rows with add spill a little too (192 bytes at 128
// registers), and are ahead all the same: 8192 x 512 16.5 us, a block a row 25.4; 50000 x 512
// 74 and 82; bf16 rows 10.5 and 18.5, 46 and 51.
constexpr int kMaxWarpH = 512;
constexpr int kMaxFusedH = 8192;  // columns up to which one pass makes dx and the column sums

// Sum over a block of at most 16 warps, the same in every thread and in a fixed order.
// `part` is not used again before another block-wide barrier.
__device__ __forceinline__ float block_sum(float s, float *part)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    const int lane = threadIdx.x & 31;
    if (lane == 0) part[threadIdx.x >> 5] = s;
    __syncthreads();
    s = (lane & 15) < int(blockDim.x >> 5) ? part[lane & 15] : 0.f;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    return s;
}
// Two of them at once, half a warp each.
__device__ __forceinline__ float2 block_sum2(float a, float b, float (*part)[16])
{
    const int lane = threadIdx.x & 31, which = lane >> 4;
    float s = which ? b : a;
    s += __shfl_xor_sync(0xFFFFFFFFu, which ? a : b, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    if ((lane & 15) == 0) part[which][threadIdx.x >> 5] = s;
    __syncthreads();
    s = (lane & 15) < int(blockDim.x >> 5) ? part[which][lane & 15] : 0.f;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    return make_float2(__shfl_sync(0xFFFFFFFFu, s, 0), __shfl_sync(0xFFFFFFFFu, s, 16));
}

// R: x's type.  E8: eighths of a thread's elements.  WARP: a warp takes a row.
template <typename R, int E8, bool WARP>
__global__ void __launch_bounds__(E8 == 1 ? 1024 : 512) k_layer_norm(const LayerNormArgs p)
{
    constexpr int W = 16 / int(sizeof(R)), VPT = E8 * 8 / W;
    __shared__ float part[2][32];
    const int tid = WARP ? int(threadIdx.x & 31) : int(threadIdx.x);
    const int nt = WARP ? 32 : int(blockDim.x);
    const int64_t t = WARP ? int64_t(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5) : int64_t(blockIdx.x);
    pdl_enter();
    if (WARP && t >= p.T) return;
    const int nv = p.H / W;
    const int64_t row = t * p.H;
    const R *x = static_cast<const R *>(p.x) + row;
    Pack<R, W> r[VPT];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
        if (tid + i * nt < nv) r[i].load(x + (tid + i * nt) * W);
#pragma unroll
    for (int i = 0; i < VPT; ++i)
        if (tid + i * nt < nv) {
            float a[W];
            r[i].get(a);
#pragma unroll
            for (int j = 0; j < W; ++j) s += a[j];
        }
    const float m = row_sum<WARP>(s, part[0]) / float(p.H);
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
        if (tid + i * nt < nv) {
            float a[W];
            r[i].get(a);
#pragma unroll
            for (int j = 0; j < W; ++j) q = fmaf(a[j] - m, a[j] - m, q);
        }
    const float rs = __frsqrt_rn(row_sum<WARP>(q, part[1]) / float(p.H) + p.eps);
    if (p.mean && tid == 0) {
        p.mean[t] = m;
        p.rstd[t] = rs;
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = (tid + i * nt) * W;
        if (c >= p.H) continue;
        float v[W], a[W];
        r[i].get(v);
#pragma unroll
        for (int j = 0; j < W; ++j) v[j] = (v[j] - m) * rs;
        if (p.w) {
            Pack<float, W> w;
            w.load(p.w + c);
            w.get(a);
#pragma unroll
            for (int j = 0; j < W; ++j) v[j] *= a[j];
        }
        if (p.b) {
            Pack<float, W> b;
            b.load(p.b + c);
            b.get(a);
#pragma unroll
            for (int j = 0; j < W; ++j) v[j] += a[j];
        }
        Pack<uint16_t, W> o;
        o.set(v);
        o.store(p.out + row + c);
    }
}

// Many rows: a block walks over rows, its threads always on the same columns, so w and b
// stay in registers (fp32, they are four times a bf16 row's bytes: read again for every
// row they kept the first-level cache busy, 55 us at 8192 bf16 rows of 7168), and the next
// row's elements are on their way while this one's are worked on.
template <typename R, int E8>
__global__ void __launch_bounds__(512, 2) k_layer_norm_walk(const LayerNormArgs p)
{
    constexpr int W = 16 / int(sizeof(R)), VPT = E8 * 8 / W;
    __shared__ float part[2][16];
    const int tid = threadIdx.x, nt = blockDim.x;
    const float inv_h = 1.f / float(p.H);
    pdl_enter();
    Pack<R, W> r[VPT];
    auto load = [&](int64_t t) {
        if (t >= p.T) return;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if ((tid + i * nt) * W < p.H) r[i].load(static_cast<const R *>(p.x) + t * p.H + (tid + i * nt) * W);
    };
    load(blockIdx.x);
    F2 w[VPT][W / 2], b[VPT][W / 2];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = (tid + i * nt) * W;
#pragma unroll
        for (int j = 0; j < W / 2; ++j) {
            w[i][j] = p.w && c < p.H ? f2(p.w[c + 2 * j], p.w[c + 2 * j + 1]) : f2(1.f);
            b[i][j] = p.b && c < p.H ? f2(p.b[c + 2 * j], p.b[c + 2 * j + 1]) : f2(0.f);
        }
    }
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
        F2 v[VPT][W / 2], s = f2(0.f);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            pairs(r[i], v[i]);
            if ((tid + i * nt) * W < p.H)
#pragma unroll
                for (int j = 0; j < W / 2; ++j) s = s + v[i][j];
        }
        load(t + gridDim.x);
        const float m = block_sum(f2_sum(s), part[0]) * inv_h;
        F2 q = f2(0.f);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
#pragma unroll
            for (int j = 0; j < W / 2; ++j) v[i][j] = v[i][j] + f2(-m);
            if ((tid + i * nt) * W < p.H)
#pragma unroll
                for (int j = 0; j < W / 2; ++j) q = fma2(v[i][j], v[i][j], q);
        }
        const float rs = __frsqrt_rn(block_sum(f2_sum(q), part[1]) * inv_h + p.eps);
        if (p.mean && tid == 0) {
            p.mean[t] = m;
            p.rstd[t] = rs;
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (tid + i * nt) * W;
            if (c >= p.H) continue;
#pragma unroll
            for (int j = 0; j < W / 2; ++j) v[i][j] = fma2(v[i][j] * f2(rs), w[i][j], b[i][j]);
            Pack<uint16_t, W> o;
            set_pairs(o, v[i]);
            o.store(p.out + t * p.H + c);
        }
    }
}

template <typename R>
cudaError_t launch_fwd(const LayerNormArgs &a, cudaStream_t st)
{
    const int nv = a.H / 8;  // eights a row
    if (nv <= 128) {  // a warp holds a row
        const int warps = a.T >= 152 * 16 ? 4 : 1;
        const dim3 grid(unsigned(ceil_div(a.T, warps))), block(32 * warps);
        if (nv <= 32) return launch_pdl(k_layer_norm<R, 1, true>, grid, block, 0, st, a);
        if (nv <= 64) return launch_pdl(k_layer_norm<R, 2, true>, grid, block, 0, st, a);
        return launch_pdl(k_layer_norm<R, 4, true>, grid, block, 0, st, a);
    }
    const bool many = a.T > 8 * 152;
    // Many bf16 rows: as many blocks as an SM holds with the registers of 1024 threads.
    if constexpr (sizeof(R) == 2)
        if (a.H <= 8192 && many) {
            const unsigned threads = unsigned(round_up(ceil_div(nv, 2), 32));
            return launch_pdl(k_layer_norm_walk<R, 2>, dim3(152 * 2 * (512 / threads)), dim3(threads), 0, st, a);
        }
    // Else a block a row.  Few rows: eight elements a thread, the shortest way from load to
    // store.  Many fp32 rows, us, by eights a thread:
    //   8192 x 7168 (352 MB)  1: 78.5  2: 60.5  3: 60.7  4: 55.7 (6.3 TB/s)   walking 68.5
    //   8192 x 3584           1: 36.6  2: 30.6  3: 30.2  4: 29.4              walking 36.0
    //   8192 x 2048           1: 20.3  2: 17.4  3: 18.1  4: 18.3
    //   20000 x 1032          1: 27.5  2: 23.9  3: 24.0  4: 25.6
    // and of bf16 rows      8192 x 7168  1: 82.5  2: 56.1  3: 56.1  4: 55.1  walking 44.2 (5.3 TB/s)
    //                       8192 x 2048  1: 20.2  2: 16.1  3: 16.0  4: 16.5  walking 15.2
    const dim3 grid{unsigned(a.T)};
    int e8 = !many ? 1 : nv > 300 ? 4 : 2;  // (2: fp32 alone, such bf16 rows are walked over)
    if (e8 == 1 && nv > 1024) e8 = nv <= 1536 ? 3 : 4;
    if (nv > 2048) e8 = 8;
    const dim3 block(unsigned(round_up(ceil_div(nv, e8), 32)));
    if constexpr (sizeof(R) == 4)
        if (e8 == 2) return launch_pdl(k_layer_norm<R, 2, false>, grid, block, 0, st, a);
    switch (e8) {
    case 1: return launch_pdl(k_layer_norm<R, 1, false>, grid, block, 0, st, a);
    case 3: return launch_pdl(k_layer_norm<R, 3, false>, grid, block, 0, st, a);
    case 4: return launch_pdl(k_layer_norm<R, 4, false>, grid, block, 0, st, a);
    default: return launch_pdl(k_layer_norm<R, 8, false>, grid, block, 0, st, a);
    }
}

// ---- backward ------------------------------------------------------------------------

// Rows of at most 512 columns: a warp walks over rows, the next row on its way while this
// one is worked on.  SUMS: the column sums are kept, and written to part[block][2][H] at
// the end.
template <typename R, int E8, bool SUMS, bool ADD>
__global__ void __launch_bounds__(256, 2) k_layer_norm_warps(const LayerNormBackArgs p)
{
    constexpr int W = 16 / int(sizeof(R)), VPT = E8 * 8 / W, COLS = E8 * 256;
    extern __shared__ __align__(16) float s_cols[];  // SUMS: [8 warps][2][COLS]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const float inv_h = 1.f / float(p.H);
    const int64_t step = int64_t(gridDim.x) * 8;
    F2 w[VPT][W / 2], dw[SUMS ? VPT : 1][W / 2], db[SUMS ? VPT : 1][W / 2];
    Pack<R, W> x[VPT], ad[ADD ? VPT : 1];
    Pack<uint16_t, W> y[VPT];
    float m = 0.f, rs = 0.f;
    auto load = [&](int64_t t) {
        if (t >= p.T) return;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (lane + i * 32) * W;
            if (c >= p.H) continue;
            x[i].load(static_cast<const R *>(p.x) + t * p.H + c);
            y[i].load(p.dy + t * p.H + c);
            if (ADD) ad[i].load(static_cast<const R *>(p.add) + t * p.H + c);
        }
        m = __ldg(p.mean + t);
        rs = __ldg(p.rstd + t);
    };
    pdl_enter();
    int64_t t = int64_t(blockIdx.x) + int64_t(warp) * gridDim.x;
    load(t);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = (lane + i * 32) * W;
#pragma unroll
        for (int j = 0; j < W / 2; ++j) {
            w[i][j] = p.w && c < p.H ? f2(p.w[c + 2 * j], p.w[c + 2 * j + 1]) : f2(1.f);
            if (SUMS) dw[i][j] = db[i][j] = f2(0.f);
        }
    }
    for (; t < p.T; t += step) {
        F2 h[VPT][W / 2], g[VPT][W / 2], a[ADD ? VPT : 1][W / 2], s1 = f2(0.f), s2 = f2(0.f);
        const float r1 = rs;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if ((lane + i * 32) * W >= p.H) continue;
            pairs(x[i], h[i]);
            pairs(y[i], g[i]);
            if (ADD) pairs(ad[i], a[i]);
#pragma unroll
            for (int j = 0; j < W / 2; ++j) {
                h[i][j] = (h[i][j] + f2(-m)) * f2(r1);
                if (SUMS) {
                    dw[i][j] = fma2(g[i][j], h[i][j], dw[i][j]);
                    db[i][j] = db[i][j] + g[i][j];
                }
                g[i][j] = g[i][j] * w[i][j];
                s1 = s1 + g[i][j];
                s2 = fma2(g[i][j], h[i][j], s2);
            }
        }
        load(t + step);
        const float2 s = warp_sum2(f2_sum(s1), f2_sum(s2));
        // dx = rs g - rs mean(g) - h rs mean(g h)
        const F2 ca = f2(-r1 * (s.x * inv_h)), cb = f2(-r1 * (s.y * inv_h)), r2 = f2(r1);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (lane + i * 32) * W;
            if (c >= p.H) continue;
#pragma unroll
            for (int j = 0; j < W / 2; ++j) {
                h[i][j] = fma2(g[i][j], r2, fma2(h[i][j], cb, ca));
                if (ADD) h[i][j] = h[i][j] + a[i][j];
            }
            Pack<R, W> o;
            set_pairs(o, h[i]);
            o.store(static_cast<R *>(p.dx) + t * p.H + c);
        }
    }
    if (!SUMS) return;
    float *mine = s_cols + warp * 2 * COLS;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        Pack<float, W> q;
        set_pairs(q, dw[i]);
        q.store(mine + (lane + i * 32) * W);
        set_pairs(q, db[i]);
        q.store(mine + COLS + (lane + i * 32) * W);
    }
    __syncthreads();
    float *out = p.part + int64_t(blockIdx.x) * 2 * p.H;
    for (int c = threadIdx.x; c < 2 * p.H; c += 256) {
        const int at = c < p.H ? c : COLS + c - p.H;
        float v = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) v += s_cols[k * 2 * COLS + at];
        out[c] = v;
    }
}

// Rows too wide for a block to keep their column sums: dx alone, a block a row.
template <typename R, int E8>
__global__ void __launch_bounds__(512) k_layer_norm_dx(const LayerNormBackArgs p)
{
    constexpr int W = 16 / int(sizeof(R)), VPT = E8 * 8 / W;
    __shared__ float part[2][2][16];
    const int tid = threadIdx.x, nt = blockDim.x;
    const float inv_h = 1.f / float(p.H);
    pdl_enter();
    int turn = 0;
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x, turn ^= 1) {
        const int64_t row = t * p.H;
        const R *x = static_cast<const R *>(p.x) + row;
        Pack<R, W> r[VPT];
        Pack<uint16_t, W> y[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (tid + i * nt) * W;
            if (c < p.H) {
                r[i].load(x + c);
                y[i].load(p.dy + row + c);
            }
        }
        const float m = __ldg(p.mean + t), rs = __ldg(p.rstd + t);
        // h and g of a vector of columns
        auto value = [&](int i, int c, F2 (&h)[W / 2], F2 (&g)[W / 2]) {
            pairs(r[i], h);
            pairs(y[i], g);
#pragma unroll
            for (int j = 0; j < W / 2; ++j) h[j] = (h[j] + f2(-m)) * f2(rs);
            if (p.w) {
                Pack<float, W> q;
                F2 w[W / 2];
                q.load(p.w + c);
                pairs(q, w);
#pragma unroll
                for (int j = 0; j < W / 2; ++j) g[j] = g[j] * w[j];
            }
        };
        F2 s1 = f2(0.f), s2 = f2(0.f);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (tid + i * nt) * W;
            if (c >= p.H) continue;
            F2 h[W / 2], g[W / 2];
            value(i, c, h, g);
#pragma unroll
            for (int j = 0; j < W / 2; ++j) {
                s1 = s1 + g[j];
                s2 = fma2(g[j], h[j], s2);
            }
        }
        const float2 s = block_sum2(f2_sum(s1), f2_sum(s2), part[turn]);
        const F2 a = f2(-rs * (s.x * inv_h)), b = f2(-rs * (s.y * inv_h)), r2 = f2(rs);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (tid + i * nt) * W;
            if (c >= p.H) continue;
            F2 h[W / 2], g[W / 2];
            value(i, c, h, g);
#pragma unroll
            for (int j = 0; j < W / 2; ++j) h[j] = fma2(g[j], r2, fma2(h[j], b, a));
            if (p.add) {
                Pack<R, W> q;
                q.load(static_cast<const R *>(p.add) + row + c);
                pairs(q, g);
#pragma unroll
                for (int j = 0; j < W / 2; ++j) h[j] = h[j] + g[j];
            }
            Pack<R, W> o;
            set_pairs(o, h);
            o.store(static_cast<R *>(p.dx) + row + c);
        }
    }
}

// A block walks over rows, each thread's columns of the next rows on their way into a
// ring in shared memory (cp.async: a thread waits for its own copies, no barrier), read
// from there once for the sums and once for the output.
template <int BYTES>
__device__ __forceinline__ void copy_async(void *dst, const void *src)
{
    // 16 bytes go past the first-level cache, which the ring leaves too small for the copies in flight
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(uint32_t(__cvta_generic_to_shared(dst))), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(uint32_t(__cvta_generic_to_shared(dst))), "l"(src), "n"(BYTES)
                     : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <typename R, int S, bool SUMS, bool ADD>
__global__ void __launch_bounds__(512, 1) k_layer_norm_ring(const LayerNormBackArgs p)
{
    constexpr int W = 16 / int(sizeof(R)), VPT = 16 / W;
    __shared__ float part[2][2][16];
    extern __shared__ __align__(16) uint8_t ring[];  // [S] x row | dy row | add row
    const int tid = threadIdx.x, nt = blockDim.x;
    const int stage = p.H * (int(sizeof(R)) * (ADD ? 2 : 1) + 2);
    const float inv_h = 1.f / float(p.H);
    F2 w[VPT][W / 2], dw[SUMS ? VPT : 1][W / 2], db[SUMS ? VPT : 1][W / 2];
    auto xs = [&](int s) { return reinterpret_cast<R *>(ring + s * stage); };
    auto ys = [&](int s) { return reinterpret_cast<uint16_t *>(ring + s * stage + p.H * int(sizeof(R))); };
    auto as = [&](int s) { return reinterpret_cast<R *>(ring + s * stage + p.H * (int(sizeof(R)) + 2)); };
    auto fetch = [&](int64_t t, int s) {
        if (t < p.T) {
            const int64_t row = t * p.H;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int c = (tid + i * nt) * W;
                if (c < p.H) {
                    copy_async<16>(xs(s) + c, static_cast<const R *>(p.x) + row + c);
                    copy_async<2 * W>(ys(s) + c, p.dy + row + c);
                    if (ADD) copy_async<16>(as(s) + c, static_cast<const R *>(p.add) + row + c);
                }
            }
        }
        copy_commit();
    };
    pdl_enter();
#pragma unroll
    for (int s = 0; s < S - 1; ++s) fetch(int64_t(blockIdx.x) + int64_t(s) * gridDim.x, s);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = (tid + i * nt) * W;
#pragma unroll
        for (int j = 0; j < W / 2; ++j) {
            w[i][j] = p.w && c < p.H ? f2(p.w[c + 2 * j], p.w[c + 2 * j + 1]) : f2(1.f);
            if (SUMS) dw[i][j] = db[i][j] = f2(0.f);
        }
    }
    float m = 0.f, rs = 0.f;
    if (blockIdx.x < p.T) m = __ldg(p.mean + blockIdx.x), rs = __ldg(p.rstd + blockIdx.x);
    int turn = 0, slot = 0;
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x, turn ^= 1) {
        fetch(t + int64_t(S - 1) * gridDim.x, slot == 0 ? S - 1 : slot - 1);
        float nm = 0.f, nrs = 0.f;
        if (t + gridDim.x < p.T) nm = __ldg(p.mean + t + gridDim.x), nrs = __ldg(p.rstd + t + gridDim.x);
        copy_wait<S - 1>();
        F2 h[VPT][W / 2], g[VPT][W / 2], s1 = f2(0.f), s2 = f2(0.f);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (tid + i * nt) * W;
            if (c >= p.H) continue;
            Pack<R, W> x;
            Pack<uint16_t, W> y;
            x.load(xs(slot) + c);
            y.load(ys(slot) + c);
            pairs(x, h[i]);
            pairs(y, g[i]);
#pragma unroll
            for (int j = 0; j < W / 2; ++j) {
                h[i][j] = (h[i][j] + f2(-m)) * f2(rs);
                if (SUMS) {
                    dw[i][j] = fma2(g[i][j], h[i][j], dw[i][j]);
                    db[i][j] = db[i][j] + g[i][j];
                }
                g[i][j] = g[i][j] * w[i][j];
                s1 = s1 + g[i][j];
                s2 = fma2(g[i][j], h[i][j], s2);
            }
        }
        const float2 s = block_sum2(f2_sum(s1), f2_sum(s2), part[turn]);
        // dx = rs g - rs mean(g) - h rs mean(g h)
        const F2 a = f2(-rs * (s.x * inv_h)), b = f2(-rs * (s.y * inv_h)), r2 = f2(rs);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (tid + i * nt) * W;
            if (c >= p.H) continue;
            Pack<R, W> o;
            if (ADD) {
                F2 d[W / 2];
                o.load(as(slot) + c);
                pairs(o, d);
#pragma unroll
                for (int j = 0; j < W / 2; ++j) h[i][j] = fma2(g[i][j], r2, fma2(h[i][j], b, a)) + d[j];
            } else {
#pragma unroll
                for (int j = 0; j < W / 2; ++j) h[i][j] = fma2(g[i][j], r2, fma2(h[i][j], b, a));
            }
            set_pairs(o, h[i]);
            o.store(static_cast<R *>(p.dx) + t * p.H + c);
        }
        m = nm;
        rs = nrs;
        if (++slot == S) slot = 0;
    }
    copy_wait<0>();
    if (!SUMS) return;
    float *out = p.part + int64_t(blockIdx.x) * 2 * p.H;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = (tid + i * nt) * W;
        if (c >= p.H) continue;
        Pack<float, W> q;
        set_pairs(q, dw[i]);
        q.store(out + c);
        set_pairs(q, db[i]);
        q.store(out + p.H + c);
    }
}

// The column sums alone, for rows too wide for a block to keep them: a block takes
// 256 columns and every gridDim.y-th group of eight rows, a warp a row of it.
template <typename R>
__global__ void __launch_bounds__(256) k_layer_norm_cols(const LayerNormBackArgs p)
{
    __shared__ float s_cols[8][2][256];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = (int(blockIdx.x) * 32 + lane) * 8;
    float dw[8] = {}, db[8] = {};
    pdl_enter();
    if (c < p.H)
        for (int64_t t = int64_t(blockIdx.y) * 8 + warp; t < p.T; t += int64_t(gridDim.y) * 8) {
            Pack<R, 8> x;
            Pack<uint16_t, 8> y;
            x.load(static_cast<const R *>(p.x) + t * p.H + c);
            y.load(p.dy + t * p.H + c);
            const float m = __ldg(p.mean + t), rs = __ldg(p.rstd + t);
            float v[8], d[8];
            x.get(v);
            y.get(d);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                dw[j] = fmaf(d[j], (v[j] - m) * rs, dw[j]);
                db[j] += d[j];
            }
        }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        s_cols[warp][0][lane * 8 + j] = dw[j];
        s_cols[warp][1][lane * 8 + j] = db[j];
    }
    __syncthreads();
    const int col = int(blockIdx.x) * 256 + threadIdx.x;
    if (col >= p.H) return;
    float *out = p.part + int64_t(blockIdx.y) * 2 * p.H;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        float v = 0.f;
#pragma unroll
        for (int q = 0; q < 8; ++q) v += s_cols[q][k][threadIdx.x];
        out[k * p.H + col] = v;
    }
}

// The row splits of k_layer_norm_cols: enough blocks for four an SM.
int64_t cols_splits(int64_t T, int H)
{
    const int64_t want = ceil_div(152 * 4, ceil_div(H, 256)), most = ceil_div(T, 8);
    return want < most ? want : most;
}

// Blocks an SM, and in all, of the one-pass kernel.
int blocks_per_sm(int H)
{
    if (H <= kMaxWarpH) return 2;
    const int n = 512 / int(round_up(ceil_div(H, 16), 32));
    return n < 1 ? 1 : n > 6 ? 6 : n;  // (1024 columns, 8192 rows: two 26.0, four 19.8, six 19.6, eight 21.5 us)
}
// A block costs a row of partial sums, so it takes two rows from 304 blocks on, four from
// 608 on (fp32 rows, us: 1001 x 1024 8.3, 2000 x 1024 12.0, 500 x 2048 7.2, 1001 x 2048 12.7;
// a block a row up to the most: 12.4, 15.4, 8.5, 11.2).
int64_t fused_blocks(int64_t T, int H)
{
    const int64_t most = int64_t(152) * blocks_per_sm(H);
    if (H <= kMaxWarpH) return std::min(ceil_div(T, 8), most);
    return std::min(std::max({std::min<int64_t>(T, 304), std::min<int64_t>(T / 2, 608), T / 4}), most);
}

template <typename R, int E8>
cudaError_t warps(const LayerNormBackArgs &a, unsigned grid, cudaStream_t st)
{
    const bool sums = a.dw || a.db;
    const size_t smem = sums ? size_t(8) * 2 * E8 * 256 * 4 : 0;
    auto *kern = sums ? (a.add ? k_layer_norm_warps<R, E8, true, true> : k_layer_norm_warps<R, E8, true, false>)
                      : (a.add ? k_layer_norm_warps<R, E8, false, true> : k_layer_norm_warps<R, E8, false, false>);
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(grid), dim3(256), smem, st, a);
}

constexpr int64_t kRingBytes = 220 * 1024;  // of an SM's shared memory for the rings of its blocks
template <typename R, int S>
cudaError_t ring(const LayerNormBackArgs &a, unsigned grid, cudaStream_t st)
{
    const size_t smem = size_t(S) * a.H * (sizeof(R) * (a.add ? 2 : 1) + 2);
    const bool sums = a.dw || a.db;
    auto *kern = sums ? k_layer_norm_ring<R, S, true, true> : k_layer_norm_ring<R, S, false, true>;
    if constexpr (S == 4)  // (without add four stages always fit)
        if (!a.add) kern = sums ? k_layer_norm_ring<R, S, true, false> : k_layer_norm_ring<R, S, false, false>;
    // the most of any width: another host thread's narrower call does not lower it before this launch
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kRingBytes));
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(grid), dim3(unsigned(round_up(ceil_div(a.H / 8, 2), 32))), smem, st, a);
}

template <typename R>
cudaError_t launch_back(const LayerNormBackArgs &a, cudaStream_t st)
{
    const int nv = a.H / 8;
    const bool sums = a.dw || a.db;
    cudaError_t e;
    int64_t parts = 0;
    if (a.H <= kMaxFusedH) {
        const unsigned grid = unsigned(fused_blocks(a.T, a.H));
        parts = grid;
        if (nv <= 32) e = warps<R, 1>(a, grid, st);
        else if (nv <= 64) e = warps<R, 2>(a, grid, st);
        else {
            // stages of the ring: what the blocks of an SM have room for, four but for fp32 rows with add (the
            // blocks' rows have at most 8192 elements together: 10 bytes each there, else 6)
            const int64_t stages = kRingBytes / (int64_t(a.H) * 10 * blocks_per_sm(a.H));
            if (sizeof(R) == 2 || !a.add || stages >= 4) e = ring<R, 4>(a, grid, st);
            else if constexpr (sizeof(R) == 4) e = stages == 3 ? ring<R, 3>(a, grid, st) : ring<R, 2>(a, grid, st);
        }
    } else {
        const unsigned grid = unsigned(a.T < 152 * 2 ? a.T : 152 * 2);
        const int e8 = nv <= 2048 ? 4 : 8;
        const unsigned block = unsigned(round_up(ceil_div(nv, e8), 32));
        if (sums) {  // first: dx may be add, which it does not read
            parts = cols_splits(a.T, a.H);
            e = launch_pdl(k_layer_norm_cols<R>, dim3(unsigned(ceil_div(a.H, 256)), unsigned(parts)), dim3(256), 0, st, a);
            if (e != cudaSuccess) return e;
        }
        e = e8 == 4 ? launch_pdl(k_layer_norm_dx<R, 4>, dim3(grid), dim3(block), 0, st, a)
                    : launch_pdl(k_layer_norm_dx<R, 8>, dim3(grid), dim3(block), 0, st, a);
    }
    if (e != cudaSuccess || !sums) return e;
    return launch_col_sums(a.part, parts, a.H, 2, a.dw, a.db, st);
}

// out_k[c] = sum over g of part[g][k][c]: 32 columns a block, 16 strands of every 16th g,
// eight of a strand's loads in flight (one after another they took 20 us at 608 parts),
// the strands added in order.
constexpr int STRANDS = 16;
__global__ void __launch_bounds__(32 * STRANDS) k_col_sums(const float *part, int64_t G, int64_t C, int sets, float *out0, float *out1)
{
    __shared__ float s[STRANDS][33];
    const int lane = threadIdx.x & 31, strand = threadIdx.x >> 5;
    const int64_t c = int64_t(blockIdx.x) * 32 + lane;
    const int k = blockIdx.y;
    float *out = k ? out1 : out0;
    pdl_enter();
    if (!out) return;
    float v = 0.f;
    if (c < C) {
        const float *p = part + k * C + c;
        for (int64_t g = strand; g < G; g += 8 * STRANDS) {
            float q[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) q[i] = g + i * STRANDS < G ? p[(g + i * STRANDS) * sets * C] : 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) v += q[i];
        }
    }
    s[strand][lane] = v;
    __syncthreads();
    if (strand || c >= C) return;
#pragma unroll
    for (int q = 1; q < STRANDS; ++q) v += s[q][lane];
    out[c] = v;
}

}  // namespace

cudaError_t launch_layer_norm(const LayerNormArgs &a, cudaStream_t st)
{
    if (a.T == 0) return cudaSuccess;
    return a.x_fmt == LMOE_F32 ? launch_fwd<float>(a, st) : launch_fwd<uint16_t>(a, st);
}

size_t layer_norm_back_scratch_bytes(int64_t T, int H)
{
    if (T == 0) return 0;
    return size_t(H <= kMaxFusedH ? fused_blocks(T, H) : cols_splits(T, H)) * 2 * size_t(H) * 4;
}

cudaError_t launch_layer_norm_back(const LayerNormBackArgs &a, cudaStream_t st)
{
    if (a.T == 0) {
        cudaError_t e = cudaSuccess;
        for (float *o : {a.dw, a.db})
            if (o && e == cudaSuccess) e = cudaMemsetAsync(o, 0, size_t(a.H) * 4, st);
        return e;
    }
    return a.x_fmt == LMOE_F32 ? launch_back<float>(a, st) : launch_back<uint16_t>(a, st);
}

cudaError_t launch_col_sums(const float *part, int64_t G, int64_t C, int sets, float *out0, float *out1, cudaStream_t st)
{
    return launch_pdl(k_col_sums, dim3(unsigned(ceil_div(C, 32)), unsigned(sets)), dim3(32 * STRANDS), 0, st, part, G, C, sets,
                      out0, out1);
}

}  // namespace lmoe
