// 16-bit products of the dense operators: B n-contiguous (dz W).
#include "dense_launch16.h"

namespace ecf {

int launch_gemm16_nn(const DenseGemm &g, const DensePlan &p, const DenseGrid &gr, hipStream_t st)
{
    return run_gemm16<false, true, false>(g, p, gr, st);
}

}  // namespace ecf
