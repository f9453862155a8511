// Dense feed-forward operators: launches of the products by their plan, the products
// with short rows, and the elementwise half of the backward passes.
#include <algorithm>
#include <atomic>

#include "dense_launch.h"

namespace ecf {
namespace {

// Products whose operands have rows of under 8 elements, which the MFMA tiles'
// 16-byte chunks do not take, and fp32 products over under kShortK k, with fp32
// FMAs: a block owns a 64 x 64 tile of the output, stages 16 k of both operands in
// LDS as fp32 and each of its 256 threads sums a 4 x 4 patch (two, gated).
constexpr int TM = 64, TN = 64, TK = 16;

template <class E, bool GATED>
__global__ __launch_bounds__(256) void k_dense_short(DenseGemm g, int tiles_n)
{
    typedef typename E::raw R;
    __shared__ __attribute__((aligned(16))) float As[TK][TM + 4], Bs[GATED ? 2 : 1][TK][TN + 4];
    const int mt = (g.M + TM - 1) / TM, ty0 = (int)blockIdx.x / tiles_n;
    const int half = ty0 / mt;
    const int m0 = (ty0 % mt) * TM, n0 = ((int)blockIdx.x % tiles_n) * TN;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    float acc[GATED ? 2 : 1][4][4] = {};
    for (int s = 0; s < g.ksegs; ++s) {
        const R *pa = (const R *)g.a[g.mhalves == 2 ? half : s];
        for (int k0 = 0; k0 < g.K; k0 += TK) {
            for (int i = tid; i < TM * TK; i += 256) {
                const int m = g.a_t ? i % TM : i / TK, k = g.a_t ? i / TM : i % TK;
                const int64_t gm = m0 + m, gk = k0 + k;
                As[k][m] = gm < g.M && gk < g.K ? E::to_f(pa[g.a_t ? gk * g.lda + gm : gm * g.lda + gk]) : 0.f;
            }
            for (int i = tid; i < TN * TK; i += 256) {
                const int n = g.b_t ? i % TN : i / TK, k = g.b_t ? i / TN : i % TK;
                const int64_t gn = n0 + n, gk = k0 + k;
                const bool in = gn < g.N && gk < g.K;
                const int64_t at = g.b_t ? gk * g.ldb + gn : gn * g.ldb + gk;
                Bs[0][k][n] = in ? E::to_f(((const R *)g.b[GATED ? 0 : s])[at]) : 0.f;
                if (GATED)
                    Bs[GATED][k][n] = in ? E::to_f(((const R *)g.b[1])[at]) : 0.f;
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < TK; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        acc[0][i][j] += As[k][ty * 4 + i] * Bs[0][k][tx * 4 + j];
                        if (GATED)
                            acc[GATED][i][j] += As[k][ty * 4 + i] * Bs[GATED][k][tx * 4 + j];
                    }
            __syncthreads();
        }
    }
    const float mul = unscale_of<E, true>(g);
    for (int i = 0; i < 4; ++i) {
        const int64_t m = m0 + ty * 4 + i, n1 = n0 + tx * 4;
        void *out = g.out[half];
        if (m >= g.M || n1 >= g.N)
            continue;
        f32x4_t y4;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t n = min(n1 + j, (int64_t)g.N - 1);
            float z[2];
            for (int q = 0; q < (GATED ? 2 : 1); ++q) {
                z[q] = acc[q][i][j] * mul + (g.bias[q] ? E::to_f(((const R *)g.bias[q])[n]) : 0.f);
                if (g.save[q] && n1 + j < g.N)
                    ((R *)g.save[q])[m * g.ldsave + n] = E::from_f(z[q]);
            }
            float y = act_value(z[0], g.act);
            if (GATED)
                y *= z[1];
            else if (g.res)
                y += g.out_dtype == ECF_F32 ? ((const float *)g.res)[m * g.ldres + n]
                                            : E::to_f(((const R *)g.res)[m * g.ldres + n]);
            y4[j] = y;
        }
        if (!out)
            continue;
        if (g.out_dtype == ECF_F32 && n1 + 4 <= g.N) {
            ((any128x4 *)((float *)out + m * g.ldout + n1))->v = y4;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (n1 + j < g.N)
                    store_el(out, m * g.ldout + n1 + j, y4[j], g.out_dtype);
        }
    }
}

// dz = dout * act'(a) (linear) or da = dout * b * act'(a), db = dout * act(a)
// (gated), rounded once to the operands' type: they are operands of the two
// matrix products that follow, which the matrix cores take in that type.
// Bound by memory: reads dout, a and b, writes da and db (4096 x 1024 bf16: 9.6 us,
// 4.4 TB/s).  A block owns 64 columns
// of 64 rows (32 where that leaves CUs without two blocks): a thread takes 8
// columns (16-byte accesses) of every 32nd row, and the column sums (of the
// unrounded values) are joined over the 32 row lanes in LDS, always in the same
// order.  (256 columns and 8 row lanes: 14.6 us for 57 x 6272, a chain of eight rows.)
constexpr int kGradRows = 64, kGradCols = 64, kGradLanes = 32, kGradBlocks = 512;

// dz (da and db) of columns c .. c + 7 of row t, zeros where they end (n are left).
template <class E, class ED, bool GATED>
__device__ __forceinline__ void grad8(const DenseGrad &g, int64_t t, int c, int n, float out[GATED ? 2 : 1][8])
{
    constexpr int H = GATED ? 2 : 1;
    float d[8], a[8], b[8];
    load8<ED>(row_at<ED>(g.dout, t * g.lddout), c, n, d);
    if (g.a)
        load8<E>(row_at<E>(g.a, t * g.ldab), c, n, a);
    if constexpr (GATED)
        load8<E>(row_at<E>(g.b, t * g.ldab), c, n, b);
    with_act(g.act, [&](auto act) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float v = 0.f, s = 1.f;
            if constexpr (GATED || decltype(act)::value != ECF_ACT_NONE)
                act_both(a[j], decltype(act)::value, v, s);
            out[0][j] = GATED ? d[j] * b[j] * s : d[j] * s;
            if constexpr (GATED)
                out[H - 1][j] = d[j] * v;
        }
    });
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j >= n)
                out[h][j] = 0.f;
}

// The largest of `top` over the block's four waves; red: 4 words.
__device__ __forceinline__ uint32_t block_max(uint32_t top, uint32_t *red)
{
#pragma unroll
    for (int o = 32; o; o >>= 1)
        top = max(top, (uint32_t)__shfl_xor((int)top, o));
    if ((threadIdx.x & 63) == 0)
        red[threadIdx.x >> 6] = top;
    __syncthreads();
    return max(max(red[0], red[1]), max(red[2], red[3]));
}

// The largest finite |dz| that each block meets (as bits, which order as the values
// do), over the tiles of k_dense_grad.  A pass of its own, because every element's scale
// needs the largest of all; k_dense_grad then finds its inputs in the cache (777 x 1999,
// three inputs of odd width: 7.1 to 7.4 us, of which the launch and one load are most;
// linear 523 x 1411: 3.6 to 4.6).
template <class E, class ED, bool GATED>
__global__ __launch_bounds__(256) void k_dense_grad_top(DenseGrad g, int row_blocks, int rows, int tiles)
{
    __shared__ uint32_t red[4];
    const int cg = threadIdx.x & 7, rl = threadIdx.x >> 3;
    uint32_t top = 0;
    for (int tile = (int)blockIdx.x; tile < tiles; tile += (int)gridDim.x) {
        const int cb = tile / row_blocks, rb = tile - cb * row_blocks;
        const int c = cb * kGradCols + cg * 8, n = g.I - c, t1 = min(g.T, (rb + 1) * rows);
        if (n > 0)
            for (int64_t t = (int64_t)rb * rows + rl; t < t1; t += kGradLanes) {
                float out[GATED ? 2 : 1][8];
                grad8<E, ED, GATED>(g, t, c, n, out);
#pragma unroll
                for (int h = 0; h < (GATED ? 2 : 1); ++h)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint32_t u = __float_as_uint(out[h][j]) & 0x7fffffffu;
                        top = max(top, u < 0x7f800000u ? u : 0u);
                    }
            }
    }
    top = block_max(top, red);
    if (threadIdx.x == 0)
        g.tops[blockIdx.x] = top;
}

// The power of two that puts `top` (the bits of a finite value) at 2^14 to 2^15, as far as it and its
// inverse are normal numbers: 2^-113 to 2^126.
__device__ __forceinline__ int scale_exponent(uint32_t top)
{
    return top ? min(14 + 127 - (int)(top >> 23), 126) : 0;
}
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

template <class E, class ED, bool GATED>
__global__ __launch_bounds__(256) void k_dense_grad(DenseGrad g, int row_blocks, int rows, int n_tops)
{
    constexpr int H = GATED ? 2 : 1;
    constexpr bool SCALED = std::is_same<E, F16>::value;
    __shared__ float red[kGradLanes][H][kGradCols + 4];
    const int cb = (int)blockIdx.x / row_blocks, rb = (int)blockIdx.x - cb * row_blocks;
    const int cg = threadIdx.x & 7, rl = threadIdx.x >> 3;
    const int c = cb * kGradCols + cg * 8, n = g.I - c;
    const int t1 = min(g.T, (rb + 1) * rows);
    float sum[H][8] = {}, scale = 1.f;
    int64_t t = (int64_t)rb * rows + rl;
    auto take = [&](float out[H][8]) __attribute__((always_inline)) {
#pragma unroll
        for (int h = 0; h < H; ++h) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                sum[h][j] += out[h][j];
                if (SCALED)
                    out[h][j] *= scale;
            }
            if (g.dz)
                store8<E>(row_at<E>(g.dz, ((int64_t)h * g.T + t) * g.pitch), c, 8, out[h]);
        }
        t += kGradLanes;
    };
    if (SCALED && n_tops) {
        // the blocks' largest values travel together with the first row
        __shared__ uint32_t red4[4];
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < kDenseTops; i += 256)
            top = max(top, g.tops[min(i + (int)threadIdx.x, n_tops - 1)]);
        float out[H][8];
        const bool in = n > 0 && t < t1;
        if (in)
            grad8<E, ED, GATED>(g, t, c, n, out);
        const int e = scale_exponent(block_max(top, red4));
        scale = power_of_two(e);
        if (blockIdx.x == 0 && threadIdx.x == 0)
            *g.unscale = power_of_two(-e);
        if (in)
            take(out);
    }
    if (n > 0) {
#pragma unroll 2
        while (t < t1) {
            float out[H][8];
            grad8<E, ED, GATED>(g, t, c, n, out);
            take(out);
        }
    }
    if (!g.want_sums)
        return;
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
        for (int j = 0; j < 8; ++j)
            red[rl][h][cg * 8 + j] = sum[h][j];
    __syncthreads();
    if (threadIdx.x >= kGradCols * H)
        return;
    const int h = threadIdx.x / kGradCols, lc = threadIdx.x % kGradCols;
    const int64_t col = (int64_t)cb * kGradCols + lc;
    if (col < g.I) {
        float s = 0.f;
#pragma unroll
        for (int r = 0; r < kGradLanes; ++r)
            s += red[r][h][lc];
        if (row_blocks > 1)
            g.partial[((int64_t)rb * H + h) * g.I + col] = s;
        else if (g.sums[h])
            store_el(g.sums[h], col, s, g.sums_dtype);
    }
}

__global__ __launch_bounds__(256) void k_dense_colsum(DenseColsum s)
{
    __shared__ float red[4 * 64];
    colsum_block(s, (int)blockIdx.x, red);
}

}  // namespace

namespace {

// CUs of the current device, asked once per device.
int cu_count(int *out)
{
    static std::atomic<int> known[64];
    int dev = 0;
    ECF_HIP_CHECK(hipGetDevice(&dev));
    const bool slot = dev >= 0 && dev < 64;
    if (slot && (*out = known[dev].load(std::memory_order_relaxed)) > 0)
        return ECF_OK;
    ECF_HIP_CHECK(hipDeviceGetAttribute(out, hipDeviceAttributeMultiprocessorCount, dev));
    if (slot)
        known[dev].store(*out, std::memory_order_relaxed);
    return ECF_OK;
}

// Outputs of half the 256 MiB memory-side cache and more are stored past the caches:
// 8192 x 16384 bf16 of K 4096 907 -> 879 us, 8192 x 2048 (32 MiB) within 1%, and there
// the next operator finds the output in the cache.
constexpr int64_t kStreamBytes = (int64_t)128 << 20;

DenseGrid grid_of(const DenseGemm &g, const DenseTile &t, int splits, void *ws)
{
    const int bn = g.gated ? t.bn / 2 : t.bn;
    DenseGrid gr{};
    gr.half_tiles = (g.M + t.bm - 1) / t.bm;
    gr.tiles_m = gr.half_tiles * g.mhalves;
    gr.tiles_n = (g.N + bn - 1) / bn;
    gr.splits = splits;
    gr.partial = (float *)ws;
    gr.np = (g.N + 7) / 8 * 8;
    return gr;
}

}  // namespace

int launch_dense_gemm(const DenseGemm &gin, void *ws, size_t room, hipStream_t st)
{
    DenseGemm g = gin;
    g.stream_out = (int64_t)g.M * g.N * (int64_t)dense_esize(g.out_dtype) >= kStreamBytes;
    ProfScope p(g.gated ? "dense_gated" : g.a_t ? "dense_gemm_tn" : g.b_t ? "dense_gemm_nn" : "dense_gemm_nt", st);
    int cus = 0;
    const int rc = cu_count(&cus);
    if (rc != ECF_OK)
        return rc;
    const DenseChoice c = choose_gemm(g, cus, room);
    if (c.kind == DenseChoice::kFew)
        return launch_dense_few(g, c.few, st);
    if (c.kind == DenseChoice::kShort) {
        const int tiles_n = (g.N + TN - 1) / TN;
        const dim3 grid((unsigned)tiles_n * ((g.M + TM - 1) / TM) * g.mhalves);
        auto go = [&](auto e) {
            using E = decltype(e);
            if (g.gated)
                hipLaunchKernelGGL((k_dense_short<E, true>), grid, dim3(256), 0, st, g, tiles_n);
            else
                hipLaunchKernelGGL((k_dense_short<E, false>), grid, dim3(256), 0, st, g, tiles_n);
        };
        if (g.dtype == ECF_F32)
            go(F32{});
        else if (g.dtype == ECF_BF16)
            go(BF16{});
        else
            go(F16{});
        ECF_HIP_CHECK(hipGetLastError());
        return ECF_OK;
    }
    const DensePlan &plan = c.tiles;
    const DenseGrid gr = grid_of(g, dense_tile(g.dtype, plan.dma, plan.tile), plan.splits, ws);
    return g.gated ? launch_gemm_gated(g, plan, gr, st)
           : g.a_t ? launch_gemm_tn(g, plan, gr, st)
           : g.b_t ? launch_gemm_nn(g, plan, gr, st)
                   : launch_gemm_nt(g, plan, gr, st);
}

int launch_dense_backward(const DenseGemm *gx, const DenseGemm *gw, const DenseColsum &sums, void *ws, size_t room,
                          hipStream_t st)
{
    if (gx && gw) {
        int cus = 0;
        const int rc = cu_count(&cus);
        if (rc != ECF_OK)
            return rc;
        DensePair p;
        if (choose_pair(*gx, *gw, cus, room, &p)) {
            ProfScope scope("dense_gemm_pair", st);
            const DenseTile t = dense_tile(gx->dtype, p.x.dma, p.x.tile);
            return launch_gemm_pair(*gx, grid_of(*gx, t, p.x.splits, ws), *gw,
                                    grid_of(*gw, t, p.splits_w, (char *)ws + p.at_w), sums, p.x, st);
        }
    }
    if (sums.blocks) {
        ProfScope p("dense_colsum", st);
        hipLaunchKernelGGL(k_dense_colsum, dim3(sums.blocks), dim3(256), 0, st, sums);
        ECF_HIP_CHECK(hipGetLastError());
    }
    if (gx) {
        const int rc = launch_dense_gemm(*gx, ws, room, st);
        if (rc != ECF_OK)
            return rc;
    }
    return gw ? launch_dense_gemm(*gw, ws, room, st) : ECF_OK;
}

int64_t dense_grad_max_row_blocks(int64_t T) { return (T + kGradLanes - 1) / kGradLanes; }

int launch_dense_grad(const DenseGrad &g, DenseColsum *left, hipStream_t st)
{
    const int64_t cols = (g.I + kGradCols - 1) / kGradCols;
    // rows per block; all of a short batch in one block saves the launch that joins the sums
    const bool few = ((int64_t)g.T + kGradRows - 1) / kGradRows * cols < kGradBlocks;
    const int per = few && !(g.want_sums && g.T <= kGradRows) ? kGradLanes : kGradRows;
    const int rows = (g.T + per - 1) / per;
    if (rows > 0) {
        ProfScope p("dense_grad", st);
        const dim3 grid((unsigned)(cols * rows)), block(256);
        const int tiles = (int)(cols * rows), n_tops = g.tops ? std::min(tiles, kDenseTops) : 0;
        auto go = [&](auto e, auto ed) {
            using E = decltype(e);
            using ED = decltype(ed);
            if constexpr (std::is_same<E, F16>::value) {
                if (n_tops && g.gated)
                    hipLaunchKernelGGL((k_dense_grad_top<E, E, true>), dim3(n_tops), block, 0, st, g, rows, per, tiles);
                else if (n_tops)
                    hipLaunchKernelGGL((k_dense_grad_top<E, ED, false>), dim3(n_tops), block, 0, st, g, rows, per, tiles);
            }
            if (g.gated)  // dout is of the operands' type
                hipLaunchKernelGGL((k_dense_grad<E, E, true>), grid, block, 0, st, g, rows, per, n_tops);
            else
                hipLaunchKernelGGL((k_dense_grad<E, ED, false>), grid, block, 0, st, g, rows, per, n_tops);
        };
        if (g.dtype == ECF_F32)
            go(F32{}, F32{});
        else if (g.dtype == ECF_BF16)
            g.dout_dtype == ECF_F32 ? go(BF16{}, F32{}) : go(BF16{}, BF16{});
        else
            g.dout_dtype == ECF_F32 ? go(F16{}, F32{}) : go(F16{}, F16{});
        ECF_HIP_CHECK(hipGetLastError());
    }
    if (g.want_sums && rows != 1) {
        const int n = g.gated ? 2 : 1;
        *left = DenseColsum{g.partial, rows, g.I, n, g.sums_dtype, {g.sums[0], g.sums[1]},
                            (int)(((int64_t)n * g.I + 63) / 64)};
    }
    return ECF_OK;
}

}  // namespace ecf
