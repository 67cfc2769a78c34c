// Group norm kernels for bf16 features (ecc_norm_kernels.hpp).
#include "ecc_norm_kernels.hpp"

namespace ecc {
template hipError_t norm_launch_fwd<bf16>(const NormArgs&, hipStream_t);
template hipError_t norm_launch_bwd<bf16>(const NormArgs&, hipStream_t);
}  // namespace ecc
