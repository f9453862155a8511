// 16-bit products of the dense operators: the gated projection (x and both weights k-contiguous).
#include "dense_launch16.h"

namespace ecf {

int launch_gemm16_gated(const DenseGemm &g, const DensePlan &p, const DenseGrid &gr, hipStream_t st)
{
    return run_gemm16<false, false, true>(g, p, gr, st);
}

}  // namespace ecf
