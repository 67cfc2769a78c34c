// The gated pair of projections, elements of type f16.
#include "ecc_glu_kernels.hpp"

namespace ecc {
template hipError_t launch_glu_fwd<f16>(const GluArgs&, hipStream_t);
template hipError_t launch_glu_bwd<f16>(const GluArgs&, hipStream_t);
}  // namespace ecc
