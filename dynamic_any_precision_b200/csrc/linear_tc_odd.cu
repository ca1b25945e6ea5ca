// The dense products' tensor-memory kernel for output rows that are not whole groups of 8 features.
#include "linear_tc.cuh"

namespace dpa {

template cudaError_t launch_linear_variant<false>(const LinearArgs&, const LinearLaunch&, cudaStream_t);

}  // namespace dpa
