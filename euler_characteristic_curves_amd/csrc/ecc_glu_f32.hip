// The gated pair of projections, elements of type float.
#include "ecc_glu_kernels.hpp"

namespace ecc {
template hipError_t launch_glu_fwd<float>(const GluArgs&, hipStream_t);
template hipError_t launch_glu_bwd<float>(const GluArgs&, hipStream_t);
}  // namespace ecc
