// Products of the dense operators: the gated projection (x and both weights k-contiguous).
#include "dense_launch.h"

namespace ecf {

int launch_gemm_gated(const DenseGemm &g, const DensePlan &p, const DenseGrid &gr, hipStream_t st)
{
    return run_gemm<false, false, true>(g, p, gr, st);
}

}  // namespace ecf
