// Group norm kernels for f16 features (ecc_norm_kernels.hpp).
#include "ecc_norm_kernels.hpp"

namespace ecc {
template hipError_t norm_launch_fwd<f16>(const NormArgs&, hipStream_t);
template hipError_t norm_launch_bwd<f16>(const NormArgs&, hipStream_t);
}  // namespace ecc
