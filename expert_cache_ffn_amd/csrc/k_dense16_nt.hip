// 16-bit products of the dense operators: both operands k-contiguous (x W^T).
#include "dense_launch16.h"

namespace ecf {

int launch_gemm16_nt(const DenseGemm &g, const DensePlan &p, const DenseGrid &gr, hipStream_t st)
{
    return run_gemm16<false, false, false>(g, p, gr, st);
}

}  // namespace ecf
