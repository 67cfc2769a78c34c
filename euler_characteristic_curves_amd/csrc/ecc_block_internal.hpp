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
inline RowShape res_shape(int64_t channels, bool half, bool backward) {
  RowShape best{};
  const int vec = half ? 8 : 4;
  if (channels < vec) {
    best.V = best.K = 1;
    for (best.L = 1; best.L < channels; best.L *= 2) {
    }
  } else {
    const int64_t vectors = (channels + vec - 1) / vec;
    // 16 elements a lane at most, 8 in the backward pass, which holds ten numbers
    // of each, unless a row would need more than 512 lanes
    int most = 16 / vec;
    if (backward && vectors <= 512 * (8 / vec)) most = 8 / vec;
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
    const RowShape s = res_shape(channels, half, true);
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
  // (8 steps of 16 bits: 64 x 256 x 1024 30 us forward and 50 backward, with 16
  // 30 and 45; 12 x 8192 x 201 37 and 54, with 16 33 and 62, and its parts 27 for
  // 25.  With 64 channels a workgroup at most besides: 29 and 52, 41 and 64.)
  s.R = steps <= 4 ? 1 : (half ? 16 : 8);
  // lanes across the channels: few idle ones, and long runs of a row, as the
  // lines at a run's ends are fetched for others too (12 x 8192 x 201, float16,
  // forward and backward: 394 us with runs of 32 bytes)
  double least = 0.0;
  for (int L = 64; L >= 8; L /= 2) {
    const int64_t across = (int64_t)L * s.V, blocks = (channels + across - 1) / across;
    const double cost = (double)(blocks * across) * (1.0 + 64.0 / (double)(across * (half ? 2 : 4)));
    if (L == 64 || cost <= least) {
      least = cost;
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
// Sequences of one launch: HIP counts its threads in 32 bits.  (Parts are for
// fewer than 256 workgroups.)
inline int64_t rec_run(const RecShape& s) { return s.segments > 1 ? INT64_MAX : UINT32_MAX / 256 / s.blocks; }
// Workspace: 3 float32 per channel for every part, and its first state.
inline size_t rec_workspace_bytes(int64_t batch, int64_t steps, int64_t channels, bool half) {
  const RecShape s = rec_shape(batch, steps, channels, half);
  return s.segments > 1 ? (size_t)(batch * s.segments * 4 * channels) * sizeof(float) + 256 : 256;
}

template <class T>
hipError_t launch_recurrence_fwd(const RecArgs& a, hipStream_t stream);
template <class T>
hipError_t launch_recurrence_bwd(const RecArgs& a, hipStream_t stream);

// ------------------------------------------- gated pair of projections
struct GluArgs {
  const void* x;          // [rows][channels]
  const void *wg, *wu;    // [hidden][channels]
  const void *bg, *bu;    // [hidden], null: 0
  int act;
  int64_t rows, channels, hidden;
  void* h;                // [rows][hidden]
  const void* gh;         // [rows][hidden]
  void *gx, *gwg, *gwu, *gbg, *gbu;  // each may be null
  void* ws;
};

// A product's workgroups: tiles of 64 FM x 64 FN results, each shared by
// `splits` workgroups along the summed axis.
struct GluShare {
  int FM, FN;
  int64_t tiles_m, tiles_n;
  int splits;
};
// Rows that one float32 sum of dW runs over, at most.  (dx's sums, like the
// projections', end with a matrix's side.)
constexpr int64_t kGluRun = 16384;
// m x n results of sums over k; `both` counts the matrices of the launch.  Large
// tiles where there are enough of them (or of their shares) for the card.  least:
// shares of a sum, 0 where it cannot be shared.
inline GluShare glu_share(int64_t m, int64_t n, int64_t k, int both, int step, int64_t least) {
  GluShare s{};
  const auto tiles = [&](int fm, int fn) { return ((m + 64 * fm - 1) / (64 * fm)) * ((n + 64 * fn - 1) / (64 * fn)) * both; };
  const int64_t steps = (k + step - 1) / step;
  const int64_t shares = least ? (steps / 16 > 1 ? steps / 16 : 1) : 1;
  const bool large = tiles(4, 2) * (shares < 64 ? shares : 64) >= 192 && m > 128;
  s.FM = large ? 4 : 1;
  s.FN = 2;
  s.tiles_m = (m + 64 * s.FM - 1) / (64 * s.FM);
  s.tiles_n = (n + 64 * s.FN - 1) / (64 * s.FN);
  int64_t splits = 1;
  if (least) {
    const int64_t all = s.tiles_m * s.tiles_n * both, most = steps / 8 > 1 ? steps / 8 : 1;
    splits = all < 512 ? 512 / all : 1;
    splits = splits < most ? splits : most;
    splits = splits > least ? splits : least;
  }
  s.splits = (int)splits;
  return s;
}
inline size_t glu_part_bytes(const GluShare& s, int both) {
  return s.splits > 1 ? (size_t)(s.tiles_m * s.tiles_n * both * s.splits) * (size_t)(64 * s.FM * 64 * s.FN) * sizeof(float) : 0;
}

// Up to so many rows the weights are read once, straight to registers.
constexpr int64_t kGluFew = 64;

// Workspace: x and both weights with rows of whole steps, where theirs are not
// whole 16-byte chunks (`packed`); in the backward pass the gradients of both
// projections (rows of 2 x pitch elements, of 4 where they have 16 bits and are
// kept in two parts), partial sums of the bias gradients and shares of products.
struct GluPlan {
  bool packed;
  bool pairs;     // gradients of the projections in two parts
  int64_t wide;   // elements of a packed row
  int64_t walkers;  // workgroups that share the rows of a narrow product, or 0
  int64_t pitch;  // elements from the gate's gradients to the other's
  GluShare gates, input, weight;
  size_t at_x, at_wg, at_wu, at_dab, at_bias, at_part, bytes;
};
inline GluPlan glu_plan(int64_t rows, int64_t channels, int64_t hidden, int elem, bool backward) {
  GluPlan p{};
  const int step = 64 / elem;  // elements of a step along the summed axis
  p.pitch = (hidden + 63) / 64 * 64;
  p.pairs = elem == 2;
  p.gates = glu_share(rows, 2 * hidden, channels, 1, step, 0);
  p.gates.tiles_n = (hidden + 63) / 64;  // 64 of both projections a tile
  p.input = glu_share(rows, channels, (p.pairs ? 4 : 2) * hidden, 1, step, 1);
  p.weight = glu_share(hidden, channels, (p.pairs ? 2 : 1) * rows, 2, step, (rows + kGluRun - 1) / kGluRun);
  size_t at = 0;
  const auto take = [&at](size_t bytes) {
    at = (at + 255) & ~(size_t)255;
    const size_t here = at;
    at += bytes;
    return here;
  };
  // chunks that are not whole go through registers element by element, which
  // costs a large product more than copying its operands once (1999 x 333 to
  // 877, float32, forward and backward: 174 us so)
  p.packed = channels * elem % 16 != 0 && rows > kGluFew;
  p.wide = (channels + step - 1) / step * step;
  // sums of up to four steps: a workgroup keeps its weights and walks over the
  // rows, 64 at a time, 64 times at most (its sums of the bias gradients are
  // float32).  About three workgroups a CU, a multiple of eight to each of the 64
  // units, so that those of one tile of rows run on one die.
  const int64_t row_tiles = (rows + 63) / 64, units = (hidden + 63) / 64;
  if (p.wide <= 4 * step && row_tiles >= 64) {
    p.walkers = (768 + units - 1) / units;
    if (p.walkers * 64 < row_tiles) p.walkers = (row_tiles + 63) / 64;
    p.walkers = (p.walkers + 7) / 8 * 8;
  }
  if (p.packed) {
    p.at_x = take((size_t)(rows * p.wide) * elem);
    p.at_wg = take((size_t)(hidden * p.wide) * elem);
    p.at_wu = take((size_t)(hidden * p.wide) * elem);
  }
  if (backward) {
    p.at_dab = take((size_t)rows * (p.pairs ? 4 : 2) * p.pitch * elem);
    const int64_t sums = p.walkers > p.gates.tiles_m ? p.walkers : p.gates.tiles_m;
    p.at_bias = take((size_t)sums * 2 * p.pitch * sizeof(float));
    const size_t a = glu_part_bytes(p.input, 1), b = glu_part_bytes(p.weight, 2);
    p.at_part = take(a > b ? a : b);
  }
  p.bytes = (at + 255) & ~(size_t)255;
  if (!p.bytes) p.bytes = 256;
  return p;
}

// Whether every launch of a pass has fewer than 2^32 threads, as HIP counts them
// in 32 bits: tiles and their shares in workgroups of 256, joins in 1024.
// `aligned`: x and the weights are (their rows are where they are packed).
inline bool glu_launches(const GluPlan& p, bool backward, bool aligned) {
  const auto fits = [](int64_t blocks, int64_t threads) { return blocks <= (int64_t)(UINT32_MAX / threads); };
  const auto product = [&](const GluShare& s, int both) {
    const int64_t tiles = s.tiles_m * s.tiles_n * both;
    return fits(tiles, s.splits > 1 ? 1024 : 256) && fits(tiles * s.splits, 256);
  };
  if (p.walkers && (aligned || p.packed) ? !fits(p.walkers * p.gates.tiles_n, 256) : !product(p.gates, 1)) return false;
  return !backward || (product(p.input, 1) && product(p.weight, 2));
}

template <class T>
hipError_t launch_glu_fwd(const GluArgs& a, hipStream_t stream);
template <class T>
hipError_t launch_glu_bwd(const GluArgs& a, hipStream_t stream);

}  // namespace ecc
