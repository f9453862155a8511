// 16-bit products of the dense operators: both m/n-contiguous (dz^T x).
#include "dense_launch16.h"

namespace ecf {

int launch_gemm16_tn(const DenseGemm &g, const DensePlan &p, const DenseGrid &gr, hipStream_t st)
{
    return run_gemm16<true, true, false>(g, p, gr, st);
}

}  // namespace ecf
