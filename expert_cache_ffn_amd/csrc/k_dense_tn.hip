// Products of the dense operators: both m/n-contiguous (dz^T x).
#include "dense_launch.h"

namespace ecf {

int launch_gemm_tn(const DenseGemm &g, const DensePlan &p, const DenseGrid &gr, hipStream_t st)
{
    return run_gemm<true, true, false>(g, p, gr, st);
}

}  // namespace ecf
