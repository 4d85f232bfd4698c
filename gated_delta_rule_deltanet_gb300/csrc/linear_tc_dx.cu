// linear_tc_dx.cu -- the tensor-core product of the gradient dz w: A = w^T MN-major, B = dz K-major.
#include "linear_tc.cuh"

namespace kda {

cudaError_t launch_gemm_tc_dx(const Gemm& g, int planes, cudaStream_t st) {
  return launch_shape<true, false>(g, planes, st);
}

}  // namespace kda
