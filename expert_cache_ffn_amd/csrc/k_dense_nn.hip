// Products of the dense operators: B n-contiguous (dz W).
#include "dense_launch.h"

namespace ecf {

int launch_gemm_nn(const DenseGemm &g, const DensePlan &p, const DenseGrid &gr, hipStream_t st)
{
    return run_gemm<false, true, false>(g, p, gr, st);
}

}  // namespace ecf
