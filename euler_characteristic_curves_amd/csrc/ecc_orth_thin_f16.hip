// Orthogonalisation of thin f16 matrices (ecc_orth_thin_kernels.hpp).
#include "ecc_orth_thin_kernels.hpp"

namespace ecc {
template hipError_t launch_orth_thin<f16>(const OrthArgs&, hipStream_t);
}  // namespace ecc
