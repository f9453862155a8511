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
    for (int i = 0; i < 4; ++i) {
        const int64_t m = m0 + ty * 4 + i, n1 = n0 + tx * 4;
        const float mul = unscale_of<E, true>(g, half, m);
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

// The bits of |v| where v is finite: they order as the values do.
__device__ __forceinline__ uint32_t finite_bits(float v)
{
    const uint32_t u = __float_as_uint(v) & 0x7fffffffu;
    return u < 0x7f800000u ? u : 0u;
}
// The power of two that puts `top` (such bits) at 2^14 to 2^15, as far as it and its
// inverse are normal numbers: 2^-113 to 2^126.
__device__ __forceinline__ int scale_exponent(uint32_t top)
{
    return top ? min(14 + 127 - (int)(top >> 23), 126) : 0;
}
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// The largest finite |dz| of each row and column of a tile of k_dense_grad.  A pass of
// its own, because every element's scales need the largest of its whole row and column;
// k_dense_grad then finds its inputs in the cache (777 x 1999, three inputs of odd
// width: 7.4 us, of which the launch and one load are most; linear 523 x 1411: 4.2 to 5.0).
template <class E, class ED, bool GATED>
__global__ __launch_bounds__(256) void k_dense_grad_top(DenseGrad g, int row_blocks, int rows)
{
    constexpr int H = GATED ? 2 : 1;
    __shared__ uint32_t red[kGradLanes][H][kGradCols + 4];
    const int cb = (int)blockIdx.x / row_blocks, rb = (int)blockIdx.x - cb * row_blocks;
    const int cg = threadIdx.x & 7, rl = threadIdx.x >> 3;
    const int c = cb * kGradCols + cg * 8, n = g.I - c, t1 = min(g.T, (rb + 1) * rows);
    uint32_t col[H][8] = {};
    for (int64_t t = (int64_t)rb * rows + rl; t < t1; t += kGradLanes) {
        uint32_t row = 0;
        if (n > 0) {
            float out[H][8];
            grad8<E, ED, GATED>(g, t, c, n, out);
#pragma unroll
            for (int h = 0; h < H; ++h)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint32_t u = finite_bits(out[h][j]);
                    col[h][j] = max(col[h][j], u);
                    row = max(row, u);
                }
        }
#pragma unroll
        for (int o = 4; o; o >>= 1)  // the row's eight lanes
            row = max(row, (uint32_t)__shfl_xor((int)row, o));
        if (g.dz && cg == 0)
            g.row_tops[(int64_t)cb * g.T + t] = row;
    }
    if (!g.dz_w)
        return;
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
        for (int j = 0; j < 8; ++j)
            red[rl][h][cg * 8 + j] = col[h][j];
    __syncthreads();
    const int h = threadIdx.x / kGradCols, lc = threadIdx.x % kGradCols;
    const int64_t i = (int64_t)cb * kGradCols + lc;
    if (h >= H || i >= g.I)
        return;
    uint32_t top = 0;
#pragma unroll
    for (int r = 0; r < kGradLanes; ++r)
        top = max(top, red[r][h][lc]);
    g.col_tops[((int64_t)rb * H + h) * g.I + i] = top;
}

template <class E, class ED, bool GATED>
__global__ __launch_bounds__(256) void k_dense_grad(DenseGrad g, int row_blocks, int rows, int col_blocks)
{
    constexpr int H = GATED ? 2 : 1;
    constexpr bool F16S = std::is_same<E, F16>::value;  // may be scaled
    __shared__ float red[kGradLanes][H][kGradCols + 4];
    __shared__ float row_scale[F16S ? kGradRows : 1], col_scale[H][F16S ? kGradCols : 1];
    const int cb = (int)blockIdx.x / row_blocks, rb = (int)blockIdx.x - cb * row_blocks;
    const int cg = threadIdx.x & 7, rl = threadIdx.x >> 3;
    const int c = cb * kGradCols + cg * 8, n = g.I - c;
    const int64_t t0 = (int64_t)rb * rows;
    const int t1 = min(g.T, (rb + 1) * rows);
    float sum[H][8] = {};
    int64_t t = t0 + rl;
    auto take = [&](const float out[H][8]) __attribute__((always_inline)) {
#pragma unroll
        for (int h = 0; h < H; ++h) {
            const int64_t at = ((int64_t)h * g.T + t) * g.pitch;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                sum[h][j] += out[h][j];
            if (!F16S || !g.scaled) {
                if (g.dz)
                    store8<E>(row_at<E>(g.dz, at), c, 8, out[h]);
                continue;
            }
            float q[8];
            if (g.dz) {
                const float by = row_scale[F16S ? t - t0 : 0];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    q[j] = out[h][j] * by;
                store8<E>(row_at<E>(g.dz, at), c, 8, q);
            }
            if (g.dz_w) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    q[j] = out[h][j] * col_scale[h][F16S ? cg * 8 + j : 0];
                store8<E>(row_at<E>(g.dz_w, at), c, 8, q);
            }
        }
        t += kGradLanes;
    };
    if (F16S && g.scaled) {
        // the tiles' largest values, four (or two) lanes per row and column, travel
        // together with the first row
        constexpr int CL = kGradCols * H;
        __shared__ uint32_t tops[2][256];
        const int tid = threadIdx.x;
        constexpr int FIRST = 16;  // loads of each kind at once (more are needed beyond 64 blocks)
        const int64_t i = (int64_t)cb * kGradCols + tid % kGradCols;  // its column, of half tid / 64 % H
        const int64_t hi = (int64_t)(tid % CL / kGradCols) * g.I + min(i, (int64_t)g.I - 1);
        const uint32_t *pr = g.row_tops + min(t0 + tid % kGradRows, (int64_t)g.T - 1), *pc = g.col_tops + hi;
        auto fetch = [&](const uint32_t *p, int64_t ld, int from, int step, int n, uint32_t v[FIRST])
                         __attribute__((always_inline)) {
#pragma unroll
            for (int u = 0; u < FIRST; ++u)
                v[u] = p[min(from + u * step, n - 1) * ld];
        };
        auto most = [](uint32_t top, const uint32_t v[FIRST]) __attribute__((always_inline)) {
#pragma unroll
            for (int u = 0; u < FIRST; ++u)
                top = max(top, v[u]);
            return top;
        };
        constexpr int RS = 256 / kGradRows, CS = 256 / CL;
        uint32_t vr[FIRST] = {}, vc[FIRST] = {}, row = 0, col = 0;
        if (g.dz)
            fetch(pr, g.T, tid / kGradRows, RS, col_blocks, vr);
        if (g.dz_w)
            fetch(pc, (int64_t)H * g.I, tid / CL, CS, row_blocks, vc);
        float out[H][8];
        const bool in = n > 0 && t < t1;
        if (in)
            grad8<E, ED, GATED>(g, t, c, n, out);
        row = most(row, vr);
        col = most(col, vc);
        if (g.dz)
            for (int b = tid / kGradRows + FIRST * RS; b < col_blocks; b += FIRST * RS) {
                fetch(pr, g.T, b, RS, col_blocks, vr);
                row = most(row, vr);
            }
        if (g.dz_w)
            for (int b = tid / CL + FIRST * CS; b < row_blocks; b += FIRST * CS) {
                fetch(pc, (int64_t)H * g.I, b, CS, row_blocks, vc);
                col = most(col, vc);
            }
        tops[0][tid] = row;
        tops[1][tid] = col;
        __syncthreads();
        if (tid < kGradRows) {
#pragma unroll
            for (int b = kGradRows; b < 256; b += kGradRows)
                row = max(row, tops[0][tid + b]);
            const int e = scale_exponent(row);
            row_scale[tid] = power_of_two(e);
            if (g.dz && cb == 0 && t0 + tid < t1)
                g.row_inverse[t0 + tid] = power_of_two(-e);
        }
        if (tid < CL) {
#pragma unroll
            for (int b = CL; b < 256; b += CL)
                col = max(col, tops[1][tid + b]);
            const int e = scale_exponent(col);
            col_scale[tid / kGradCols][tid % kGradCols] = power_of_two(e);
            if (g.dz_w && rb == 0 && i < g.I)
                g.col_inverse[hi] = power_of_two(-e);
        }
        __syncthreads();
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

int64_t dense_grad_col_blocks(int64_t I) { return (I + kGradCols - 1) / kGradCols; }
int64_t dense_grad_max_row_blocks(int64_t T) { return (T + kGradLanes - 1) / kGradLanes; }

int launch_dense_grad(const DenseGrad &g, DenseColsum *left, hipStream_t st)
{
    const int64_t cols = dense_grad_col_blocks(g.I);
    // rows per block; all of a short batch in one block saves the launch that joins the sums
    const bool few = ((int64_t)g.T + kGradRows - 1) / kGradRows * cols < kGradBlocks;
    const int per = few && !(g.want_sums && g.T <= kGradRows) ? kGradLanes : kGradRows;
    const int rows = (g.T + per - 1) / per;
    if (rows > 0) {
        ProfScope p("dense_grad", st);
        const dim3 grid((unsigned)(cols * rows)), block(256);
        auto go = [&](auto e, auto ed) {
            using E = decltype(e);
            using ED = decltype(ed);
            if constexpr (std::is_same<E, F16>::value) {
                if (g.scaled && g.gated)
                    hipLaunchKernelGGL((k_dense_grad_top<E, E, true>), grid, block, 0, st, g, rows, per);
                else if (g.scaled)
                    hipLaunchKernelGGL((k_dense_grad_top<E, ED, false>), grid, block, 0, st, g, rows, per);
            }
            if (g.gated)  // dout is of the operands' type
                hipLaunchKernelGGL((k_dense_grad<E, E, true>), grid, block, 0, st, g, rows, per, (int)cols);
            else
                hipLaunchKernelGGL((k_dense_grad<E, ED, false>), grid, block, 0, st, g, rows, per, (int)cols);
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
