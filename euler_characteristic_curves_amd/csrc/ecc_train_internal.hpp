// Internal declarations of the training operators (include/ecc_train.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace ecc {

// Records the message ecc_last_error() returns (ecc_api.cpp).
void set_error(const char* message);

constexpr int kTF32 = 0, kTF16 = 1, kTBF16 = 2;  // ECC_T_*
inline int elem_bytes(int dtype) { return dtype == kTF32 ? 4 : 2; }

// ------------------------------------------------------------ group norm
struct NormArgs {
  const void* x;
  int64_t B, S, C, G;  // samples, voxels, channels, groups
  const void* weight;  // null: 1
  const void* bias;    // null: 0
  const void* readout;
  const void* offset;  // null: 0
  int pdtype;
  int act;
  float eps;
  void* y;         // features (norm) or null
  float* field;    // grid (readout) or null
  float* stats;    // [B][G][2]
  const void* gy;  // gradient of y, or of the field (float32)
  void* gx;
  void *gw, *gb, *gr, *go;  // parameter gradients, each may be null
  void* ws;
};

// Workgroups per sample of the passes over the features.  A workgroup has at
// least 4096 elements, and a launch about 8 workgroups per CU of 256.
inline int64_t norm_blocks(int64_t B, int64_t S, int64_t C) {
  int64_t nb = (S * C + 4095) / 4096, most = (2048 + B - 1) / B;
  nb = nb < most ? nb : most;
  nb = nb < S ? nb : S;
  return nb < 1 ? 1 : nb;
}

// Workspace: [partials: B x blocks rows | sums per sample: B rows | 2 floats
// per group and sample]; a row is 3 float64 per channel and one more.
inline size_t norm_row(int64_t C) { return (size_t)(3 * C + 1); }
inline size_t norm_workspace_bytes(int64_t B, int64_t S, int64_t C, int64_t G) {
  const size_t rows = (size_t)B * (size_t)(norm_blocks(B, S, C) + 1);
  return rows * norm_row(C) * sizeof(double) + (size_t)B * (size_t)G * 2 * sizeof(float) + 256;
}

template <class T>
hipError_t norm_launch_fwd(const NormArgs& a, hipStream_t stream);
template <class T>
hipError_t norm_launch_bwd(const NormArgs& a, hipStream_t stream);

}  // namespace ecc
