// Group norm kernels for f32 features (ecc_norm_kernels.hpp).
#include "ecc_norm_kernels.hpp"

namespace ecc {
template hipError_t norm_launch_fwd<float>(const NormArgs&, hipStream_t);
template hipError_t norm_launch_bwd<float>(const NormArgs&, hipStream_t);
}  // namespace ecc
