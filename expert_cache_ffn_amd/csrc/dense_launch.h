// Launches of the products for one pair of operand layouts.
#pragma once

#include "dense_gemm.h"

namespace ecf {

template <class E, bool AT, bool BT, bool GATED, bool DMA, int BM, int BN, int WM, int WN, int BK, int NS, int KW = 1>
void launch_gemm(const DenseGemm &g, const DenseGrid &gr, hipStream_t st)
{
    hipLaunchKernelGGL((k_gemm<E, AT, BT, GATED, DMA, BM, BN, WM, WN, BK, NS, KW>), dim3(gr.blocks()),
                       dim3(64 * WM * WN * KW), 0, st, g, gr);
}

template <class E, bool GATED>
void launch_join(const DenseGemm &g, const DenseGrid &gr, hipStream_t st)
{
    const int64_t n = gr.np / 8 * g.M * g.mhalves;
    hipLaunchKernelGGL((k_dense_join<E, GATED>), dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st, g, gr);
}

template <class E, bool AT, bool BT, bool GATED, bool DMA>
int pick_gemm(const DenseGemm &g, const DensePlan &p, const DenseGrid &gr, hipStream_t st)
{
    // the order of the launcher's tables
    if constexpr (std::is_same<E, F32>::value) {
        switch (p.tile) {
        case 0: launch_gemm<E, AT, BT, GATED, false, 128, 128, 4, 2, 32, 1>(g, gr, st); break;
        case 1: launch_gemm<E, AT, BT, GATED, false, 64, 128, 2, 4, 64, 1>(g, gr, st); break;
        default: launch_gemm<E, AT, BT, GATED, false, 64, 64, 2, 2, 64, 1, 2>(g, gr, st); break;
        }
    } else {
        switch (p.tile) {
        case 0: launch_gemm<E, AT, BT, GATED, DMA, 256, 256, 2, 4, 64, DMA ? 2 : 1>(g, gr, st); break;
        case 1: launch_gemm<E, AT, BT, GATED, DMA, 128, 256, 2, 4, 64, DMA ? 3 : 2>(g, gr, st); break;
        case 2: launch_gemm<E, AT, BT, GATED, DMA, 128, 128, 2, 2, 64, DMA ? 2 : 1>(g, gr, st); break;
        case 3: launch_gemm<E, AT, BT, GATED, DMA, 64, DMA ? 128 : 64, 2, 2, 64, DMA ? 3 : 1>(g, gr, st); break;
        default:
            if constexpr (DMA)
                launch_gemm<E, AT, BT, GATED, true, 64, 64, 2, 2, 64, 3>(g, gr, st);
        }
    }
    if (gr.splits > 1)
        launch_join<E, GATED>(g, gr, st);
    ECF_HIP_CHECK(hipGetLastError());
    return ECF_OK;
}

template <class E, bool DMA, int BM, int BN, int WM, int WN, int BK, int NS, int KW = 1>
void launch_pair(const DenseGemm &gx, const DenseGrid &grx, const DenseGemm &gw, const DenseGrid &grw,
                 const DenseColsum &sums, hipStream_t st)
{
    const int x_first = (int64_t)gx.K * gx.ksegs / grx.splits >= gw.K / grw.splits;
    hipLaunchKernelGGL((k_gemm_pair<E, DMA, BM, BN, WM, WN, BK, NS, KW>), dim3(grx.blocks() + grw.blocks() + sums.blocks),
                       dim3(64 * WM * WN * KW), 0, st, gx, grx, gw, grw, sums, x_first);
}

template <class E, bool DMA>
int pick_pair(const DenseGemm &gx, const DenseGrid &grx, const DenseGemm &gw, const DenseGrid &grw,
              const DenseColsum &sums, const DensePlan &p, hipStream_t st)
{
    if constexpr (std::is_same<E, F32>::value) {
        switch (p.tile) {
        case 0: launch_pair<E, false, 128, 128, 4, 2, 32, 1>(gx, grx, gw, grw, sums, st); break;
        case 1: launch_pair<E, false, 64, 128, 2, 4, 64, 1>(gx, grx, gw, grw, sums, st); break;
        default: launch_pair<E, false, 64, 64, 2, 2, 64, 1, 2>(gx, grx, gw, grw, sums, st); break;
        }
    } else {
        switch (p.tile) {
        case 2: launch_pair<E, DMA, 128, 128, 2, 2, 64, DMA ? 2 : 1>(gx, grx, gw, grw, sums, st); break;
        case 3: launch_pair<E, DMA, 64, DMA ? 128 : 64, 2, 2, 64, DMA ? 3 : 1>(gx, grx, gw, grw, sums, st); break;
        default:
            if constexpr (DMA)
                launch_pair<E, true, 64, 64, 2, 2, 64, 3>(gx, grx, gw, grw, sums, st);
        }
    }
    if (grx.splits > 1)
        launch_join<E, false>(gx, grx, st);
    if (grw.splits > 1)
        launch_join<E, false>(gw, grw, st);
    ECF_HIP_CHECK(hipGetLastError());
    return ECF_OK;
}

template <bool AT, bool BT, bool GATED>
int run_gemm(const DenseGemm &g, const DensePlan &p, const DenseGrid &gr, hipStream_t st)
{
    if (g.dtype == ECF_F32)
        return pick_gemm<F32, AT, BT, GATED, false>(g, p, gr, st);
    if (g.dtype == ECF_BF16)
        return p.dma ? pick_gemm<BF16, AT, BT, GATED, true>(g, p, gr, st)
                     : pick_gemm<BF16, AT, BT, GATED, false>(g, p, gr, st);
    return p.dma ? pick_gemm<F16, AT, BT, GATED, true>(g, p, gr, st)
                 : pick_gemm<F16, AT, BT, GATED, false>(g, p, gr, st);
}

int launch_gemm_gated(const DenseGemm &g, const DensePlan &p, const DenseGrid &gr, hipStream_t st);
int launch_gemm_nt(const DenseGemm &g, const DensePlan &p, const DenseGrid &gr, hipStream_t st);
int launch_gemm_nn(const DenseGemm &g, const DensePlan &p, const DenseGrid &gr, hipStream_t st);
int launch_gemm_tn(const DenseGemm &g, const DensePlan &p, const DenseGrid &gr, hipStream_t st);

int launch_gemm_pair(const DenseGemm &gx, const DenseGrid &grx, const DenseGemm &gw, const DenseGrid &grw,
                     const DenseColsum &sums, const DensePlan &p, hipStream_t st);

}  // namespace ecf
