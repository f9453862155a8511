// Products of the dense operators: both products of a backward pass in one launch.
#include "dense_launch.h"

namespace ecf {

int launch_gemm_pair(const DenseGemm &gx, const DenseGrid &grx, const DenseGemm &gw, const DenseGrid &grw,
                     const DenseColsum &sums, const DensePlan &p, hipStream_t st)
{
    if (gx.dtype == ECF_F32)
        return pick_pair<F32, false>(gx, grx, gw, grw, sums, p, st);
    if (gx.dtype == ECF_BF16)
        return p.dma ? pick_pair<BF16, true>(gx, grx, gw, grw, sums, p, st)
                     : pick_pair<BF16, false>(gx, grx, gw, grw, sums, p, st);
    return p.dma ? pick_pair<F16, true>(gx, grx, gw, grw, sums, p, st)
                 : pick_pair<F16, false>(gx, grx, gw, grw, sums, p, st);
}

}  // namespace ecf
