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

// -------------------------------------------------------- gated recurrence
struct RecArgs {
  const void* x;
  const void* gate;
  int64_t batch, steps, channels;
  const float* state;       // null: 0
  const int64_t* lengths;   // null: all steps
  void* h;
  float* last;
  float* saved;       // [batch][tiles][channels]: the state before every tile; null: not kept
  const void* gh;     // null: 0
  const float* glast;  // null: 0
  void *gx, *ggate;
  float* gstate;      // null: not wanted
  void* ws;
};

// A workgroup of 256 threads has L lanes of V channels and G = 256 / L groups of
// them, each with R steps of a tile, and takes `per` tiles one after the other.
struct RecShape {
  int V, R, L, G;
  int64_t blocks;       // workgroups across the channels
  int64_t tiles, per, segments;
};
inline RecShape rec_shape(int64_t batch, int64_t steps, int64_t channels, bool half) {
  RecShape s{};
  s.V = channels >= 2 ? 2 : 1;
  s.R = steps <= 4 ? 1 : (half ? 16 : 8);
  // lanes that leave few idle ones over the channels, wide where two are alike
  int64_t least = INT64_MAX;
  for (int L = 64; L >= 8; L /= 2) {
    const int64_t across = (int64_t)L * s.V, blocks = (channels + across - 1) / across;
    if (blocks * across < least) {
      least = blocks * across;
      s.L = L;
      s.blocks = blocks;
    }
  }
  s.G = 256 / s.L;
  const int64_t tile = (int64_t)s.G * s.R, base = batch * s.blocks;
  s.tiles = (steps + tile - 1) / tile;
  // with a workgroup for every CU a sequence is taken whole; with fewer, its
  // parts are summed up in a pass of their own and then run side by side
  const int64_t want = base >= 256 ? 1 : (1024 + base - 1) / base;
  s.per = (s.tiles + want - 1) / want;
  s.segments = (s.tiles + s.per - 1) / s.per;
  return s;
}
// Workspace: 3 float32 per channel for every part.
inline size_t rec_workspace_bytes(int64_t batch, int64_t steps, int64_t channels, bool half) {
  const RecShape s = rec_shape(batch, steps, channels, half);
  return s.segments > 1 ? (size_t)(batch * s.segments * 3 * channels) * sizeof(float) + 256 : 256;
}

template <class T>
hipError_t launch_recurrence_fwd(const RecArgs& a, hipStream_t stream);
template <class T>
hipError_t launch_recurrence_bwd(const RecArgs& a, hipStream_t stream);

}  // namespace ecc
