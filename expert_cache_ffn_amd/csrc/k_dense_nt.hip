// Products of the dense operators: both operands k-contiguous (x W^T).
#include "dense_launch.h"

namespace ecf {

int launch_gemm_nt(const DenseGemm &g, const DensePlan &p, const DenseGrid &gr, hipStream_t st)
{
    return run_gemm<false, false, false>(g, p, gr, st);
}

}  // namespace ecf
