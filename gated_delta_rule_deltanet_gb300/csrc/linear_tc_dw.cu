// linear_tc_dw.cu -- the tensor-core product of the gradient dz^T x: both operands MN-major.
#include "linear_tc.cuh"

namespace kda {

cudaError_t launch_gemm_tc_dw(const Gemm& g, int planes, cudaStream_t st) {
  return launch_shape<true, true>(g, planes, st);
}

}  // namespace kda
