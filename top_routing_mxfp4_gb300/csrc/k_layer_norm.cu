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
// warp (up to 1024 columns) or a block (up to 8192) walks over rows, each thread
// always on the same columns, whose shares of dw and db it keeps in registers;
// at the end each block writes its shares, and a second kernel adds the blocks' in
// order.  Wider rows take the column sums in a pass of their own.
#include "lmoe_internal.cuh"
#include "row_vec.cuh"

namespace lmoe {
namespace {

constexpr int kMaxFusedH = 8192;  // columns up to which one pass makes dx and the column sums

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
    const dim3 grid{unsigned(a.T)};
    int e8 = 1;
    if (nv > 1024) e8 = nv <= 1536 ? 3 : nv <= 2048 ? 4 : 8;
    const dim3 block(unsigned(round_up(ceil_div(nv, e8), 32)));
    switch (e8) {
    case 1: return launch_pdl(k_layer_norm<R, 1, false>, grid, block, 0, st, a);
    case 3: return launch_pdl(k_layer_norm<R, 3, false>, grid, block, 0, st, a);
    case 4: return launch_pdl(k_layer_norm<R, 4, false>, grid, block, 0, st, a);
    default: return launch_pdl(k_layer_norm<R, 8, false>, grid, block, 0, st, a);
    }
}

// ---- backward ------------------------------------------------------------------------

// Two sums over a row's threads at once, the same in every thread, in a fixed
// order.  `part` is used by one call at a time and by none of the next one's:
// callers alternate between two.
template <bool WARP>
__device__ __forceinline__ float2 row_sum2(float a, float b, float2 *part)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
        b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
    }
    if (WARP) return make_float2(a, b);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = make_float2(a, b);
    __syncthreads();
    const int nw = int(blockDim.x) >> 5, lane = threadIdx.x & 31;
    const float2 v = lane < nw ? part[lane] : make_float2(0.f, 0.f);
    a = v.x, b = v.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
        b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
    }
    return make_float2(a, b);
}

// SUMS: the column sums are kept, and written to part[block][2][H] at the end.
template <typename R, int E8, bool WARP, bool SUMS>
__global__ void __launch_bounds__(WARP ? 256 : (E8 == 1 ? 1024 : 512)) k_layer_norm_back(const LayerNormBackArgs p)
{
    constexpr int W = 16 / int(sizeof(R)), VPT = E8 * 8 / W;
    __shared__ float2 part[2][32];
    extern __shared__ float s_cols[];  // WARP, SUMS: [warps][2][E8 * 256]
    const int tid = WARP ? int(threadIdx.x & 31) : int(threadIdx.x);
    const int nt = WARP ? 32 : int(blockDim.x);
    const int warps = int(blockDim.x >> 5), warp = int(threadIdx.x >> 5);
    const int64_t first = WARP ? int64_t(blockIdx.x) + int64_t(warp) * gridDim.x : int64_t(blockIdx.x);
    const int64_t step = WARP ? int64_t(gridDim.x) * warps : int64_t(gridDim.x);
    const float inv_h = 1.f / float(p.H);
    float dw[SUMS ? VPT : 1][W], db[SUMS ? VPT : 1][W];
    if (SUMS)
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int j = 0; j < W; ++j) dw[i][j] = db[i][j] = 0.f;
    pdl_enter();
    int turn = 0;
    for (int64_t t = first; t < p.T; t += step, turn ^= 1) {
        const int64_t row = t * p.H;
        const R *x = static_cast<const R *>(p.x) + row;
        Pack<R, W> r[VPT], ad[VPT];
        Pack<uint16_t, W> y[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (tid + i * nt) * W;
            if (c < p.H) {
                r[i].load(x + c);
                y[i].load(p.dy + row + c);
            }
        }
        if (p.add)
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int c = (tid + i * nt) * W;
                if (c < p.H) ad[i].load(static_cast<const R *>(p.add) + row + c);
            }
        const float m = __ldg(p.mean + t), rs = __ldg(p.rstd + t);
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (tid + i * nt) * W;
            if (c >= p.H) continue;
            float v[W], d[W], w[W];
            r[i].get(v);
            y[i].get(d);
            if (p.w) {
                Pack<float, W> q;
                q.load(p.w + c);
                q.get(w);
            }
#pragma unroll
            for (int j = 0; j < W; ++j) {
                const float h = (v[j] - m) * rs, g = p.w ? d[j] * w[j] : d[j];
                if (SUMS) {
                    dw[i][j] = fmaf(d[j], h, dw[i][j]);
                    db[i][j] += d[j];
                }
                s1 += g;
                s2 = fmaf(g, h, s2);
            }
        }
        const float2 s = row_sum2<WARP>(s1, s2, part[turn]);
        const float a = s.x * inv_h, b = s.y * inv_h;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (tid + i * nt) * W;
            if (c >= p.H) continue;
            float v[W], d[W], w[W];
            r[i].get(v);
            y[i].get(d);
            if (p.w) {
                Pack<float, W> q;
                q.load(p.w + c);
                q.get(w);
            }
#pragma unroll
            for (int j = 0; j < W; ++j) {
                const float h = (v[j] - m) * rs, g = p.w ? d[j] * w[j] : d[j];
                v[j] = rs * (g - a - h * b);
            }
            if (p.add) {
                ad[i].get(d);
#pragma unroll
                for (int j = 0; j < W; ++j) v[j] += d[j];
            }
            r[i].set(v);
            r[i].store(static_cast<R *>(p.dx) + row + c);
        }
    }
    if (!SUMS) return;
    float *out = p.part + int64_t(blockIdx.x) * 2 * p.H;
    if (!WARP) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (tid + i * nt) * W;
            if (c >= p.H) continue;
            Pack<float, W> q;
            q.set(dw[i]);
            q.store(out + c);
            q.set(db[i]);
            q.store(out + p.H + c);
        }
        return;
    }
    constexpr int COLS = E8 * 256;
    float *mine = s_cols + warp * 2 * COLS;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < W; ++j) {
            mine[(tid + i * nt) * W + j] = dw[i][j];
            mine[COLS + (tid + i * nt) * W + j] = db[i][j];
        }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * p.H; c += blockDim.x) {
        const int at = c < p.H ? c : COLS + c - p.H;
        float v = 0.f;
        for (int k = 0; k < warps; ++k) v += s_cols[k * 2 * COLS + at];
        out[c] = v;
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

// Blocks of the one-pass kernel.
int64_t fused_blocks(int64_t T, int H)
{
    const int64_t most = H <= 1024 ? 2 * 152 : 152;
    return T < most ? T : most;
}

template <typename R, int E8, bool WARP, bool SUMS>
cudaError_t back(const LayerNormBackArgs &a, unsigned grid, unsigned block, cudaStream_t st)
{
    const size_t smem = WARP && SUMS ? size_t(block / 32) * 2 * E8 * 256 * 4 : 0;
    auto *kern = k_layer_norm_back<R, E8, WARP, SUMS>;
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(kern, dim3(grid), dim3(block), smem, st, a);
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
        const unsigned block = a.H <= 1024 ? 256 : unsigned(round_up(nv, 32));
        parts = grid;
        if (nv <= 32) e = sums ? back<R, 1, true, true>(a, grid, block, st) : back<R, 1, true, false>(a, grid, block, st);
        else if (nv <= 64) e = sums ? back<R, 2, true, true>(a, grid, block, st) : back<R, 2, true, false>(a, grid, block, st);
        else if (nv <= 128) e = sums ? back<R, 4, true, true>(a, grid, block, st) : back<R, 4, true, false>(a, grid, block, st);
        else e = sums ? back<R, 1, false, true>(a, grid, block, st) : back<R, 1, false, false>(a, grid, block, st);
    } else {
        const unsigned grid = unsigned(a.T < 152 * 2 ? a.T : 152 * 2);
        const int e8 = nv <= 2048 ? 4 : 8;
        const unsigned block = unsigned(round_up(ceil_div(nv, e8), 32));
        if (sums) {  // first: dx may be add, which it does not read
            parts = cols_splits(a.T, a.H);
            e = launch_pdl(k_layer_norm_cols<R>, dim3(unsigned(ceil_div(a.H, 256)), unsigned(parts)), dim3(256), 0, st, a);
            if (e != cudaSuccess) return e;
        }
        e = e8 == 4 ? back<R, 4, false, false>(a, grid, block, st) : back<R, 8, false, false>(a, grid, block, st);
    }
    if (e != cudaSuccess || !sums) return e;
    return launch_col_sums(a.part, parts, a.H, 2, a.dw, a.db, st);
}

// out_k[c] = sum over g of part[g][k][c], in order of g within eight strands that are
// added in order: 32 columns a block, a warp of rows each.
__global__ void __launch_bounds__(256) k_col_sums(const float *part, int64_t G, int64_t C, int sets, float *out0, float *out1)
{
    __shared__ float s[8][33];
    const int lane = threadIdx.x & 31, strand = threadIdx.x >> 5;
    const int64_t c = int64_t(blockIdx.x) * 32 + lane;
    const int k = blockIdx.y;
    float *out = k ? out1 : out0;
    pdl_enter();
    if (!out) return;
    float v = 0.f;
    if (c < C)
        for (int64_t g = strand; g < G; g += 8) v += part[(g * sets + k) * C + c];
    s[strand][lane] = v;
    __syncthreads();
    if (strand || c >= C) return;
#pragma unroll
    for (int q = 1; q < 8; ++q) v += s[q][lane];
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
    return launch_pdl(k_col_sums, dim3(unsigned(ceil_div(C, 32)), unsigned(sets)), dim3(256), 0, st, part, G, C, sets,
                      out0, out1);
}

}  // namespace lmoe
