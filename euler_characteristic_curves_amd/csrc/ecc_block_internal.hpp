// Internal declarations of the operators of a residual block (include/ecc_train.h):
// norms around a block, the gated pair of projections, the gated recurrence.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace ecc {

// --------------------------------------------------- norms around a block
struct ResArgs {
  const void* x;
  const void* branch;  // null: y is scale x, and is not written
  int xdtype, dtype;   // of x, y, and of branch, z
  int64_t batch, inner, channels;
  const void* gate;    // null: 1
  int64_t gate_stride;  // channels where every sample has gates of its own, else 0
  const void* weight;   // null: 1
  const void* branch_weight;  // null: 1
  int pdtype;
  bool norm_branch;
  float scale, eps;
  void* y;
  void* z;
  float* stats;     // [rows][2]: 1 / rms of the branch, of y
  const void* gy;   // null: 0
  const void* gz;   // null: 0
  void *gx, *gbranch, *ggate, *gweight, *gbranch_weight;  // each may be null
  void* ws;
};

// How a row is laid over lanes: vectors of V elements, K of them a lane, L lanes
// (a power of two), in workgroups of `threads`.
struct RowShape {
  int V, K, L, threads;
};
inline RowShape res_shape(int64_t channels, bool half) {
  RowShape best{};
  const int vec = half ? 8 : 4, most = half ? 2 : 4;  // 16 elements a lane at most: the backward pass holds ten of each
  if (channels < vec) {
    best.V = best.K = 1;
    for (best.L = 1; best.L < channels; best.L *= 2) {
    }
  } else {
    const int64_t vectors = (channels + vec - 1) / vec;
    int64_t least = INT64_MAX;
    for (int K = 1; K <= most; ++K) {
      int64_t L = 1;
      while (L * K < vectors) L *= 2;
      // as few idle lanes as can be; of those, rows within one wave
      if (L <= 512 && (L * K < least || (L * K == least && best.L > 64))) {
        least = L * K;
        best.V = vec;
        best.K = K;
        best.L = (int)L;
      }
    }
  }
  best.threads = best.L > 256 ? best.L : 256;
  return best;
}

// Workgroups per sample (samples are one where gates are shared), `total` in a
// launch and more where a thread would get more than kResRows rows: their sums
// are float32.
constexpr int64_t kResRows = 256;
inline int64_t res_blocks(int64_t samples, int64_t rows, int slots, int64_t total) {
  const int64_t most = (rows + slots - 1) / slots;
  int64_t nb = (total + samples - 1) / samples;
  const int64_t least = (rows + slots * kResRows - 1) / (slots * kResRows);
  nb = nb > least ? nb : least;
  return nb < most ? nb : most;
}
constexpr int64_t kResSums = 1024, kResApply = 2048;

// Workspace of the backward pass: a partial row of 3 float32 per channel for
// every workgroup.  The layout does not depend on types, its bound neither.
inline size_t res_workspace_bytes(int64_t batch, int64_t inner, int64_t channels, bool sample_gates) {
  const int64_t samples = sample_gates ? batch : 1, rows = sample_gates ? inner : batch * inner;
  size_t most = 0;
  for (int half = 0; half < 2; ++half) {
    const RowShape s = res_shape(channels, half);
    const size_t bytes = (size_t)samples * (size_t)res_blocks(samples, rows, s.threads / s.L, kResSums) *
                         (size_t)(3 * channels) * sizeof(float);
    most = bytes > most ? bytes : most;
  }
  return most + 256;
}

hipError_t launch_residual_fwd(const ResArgs& a, hipStream_t stream);
hipError_t launch_residual_bwd(const ResArgs& a, hipStream_t stream);

}  // namespace ecc
