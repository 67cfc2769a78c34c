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
  float* stats;    // [B][G][3]
  const void* gy;  // gradient of y, or of the field (float32)
  void* gx;
  void *gw, *gb, *gr, *go;  // parameter gradients, each may be null
  void* ws;
};

// Workgroups per sample of a pass over the features, `total` in a launch.  Each
// has at least 4096 elements, or 8192 where it leaves partial sums, which the
// next pass has to read (256 x 256 x 64 float32 forward: 18.9 us, 20.3 with
// 4096).  Passes that hold sums or both gradients leave a partial row each and
// have some 4 workgroups a CU resident: 1024 (2 x 128^3 x 64, bfloat16: 803 us a
// training pass, 838 with 2048).  (They need 54 to 130 registers with one vector
// a lane, 4 to 8 workgroups a CU, 76 to 168 with two, 3 to 6, and float32 with four
// 130 to 251, 2 or 3.)  The forward's second pass fits 6 to 8 a CU with one
// vector: 2048 (read-out of 256^3 x 32: 226 us, 250 with 1024).
constexpr int64_t kNormSums = 1024, kNormApply = 2048;
inline int64_t norm_blocks(int64_t B, int64_t S, int64_t C, int64_t total) {
  const int64_t least = total == kNormSums ? 8192 : 4096;
  int64_t nb = (S * C + least - 1) / least, most = (total + B - 1) / B;
  nb = nb < most ? nb : most;
  nb = nb < S ? nb : S;
  return nb < 1 ? 1 : nb;
}

// Rows per sample that more partial rows than that can be folded to before they
// are joined.
constexpr int kNormFolded = 32;
inline int64_t norm_folded(int64_t blocks) { return blocks > kNormFolded ? kNormFolded : 0; }

// Workspace: [partials: B x blocks rows | sums per sample: B rows | folded
// partials: B x norm_folded rows | 2 floats per group and sample]; a row is 3
// float64 per channel and one more.
inline size_t norm_row(int64_t C) { return (size_t)(3 * C + 1); }
inline size_t norm_workspace_bytes(int64_t B, int64_t S, int64_t C, int64_t G) {
  const int64_t blocks = norm_blocks(B, S, C, kNormSums);
  const size_t rows = (size_t)B * (size_t)(blocks + 1 + norm_folded(blocks));
  return rows * norm_row(C) * sizeof(double) + (size_t)B * (size_t)G * 2 * sizeof(float) + 256;
}

template <class T>
hipError_t norm_launch_fwd(const NormArgs& a, hipStream_t stream);
template <class T>
hipError_t norm_launch_bwd(const NormArgs& a, hipStream_t stream);

// ------------------------------------------------- orthogonalised updates
struct OrthArgs {
  const void* g;  // gradient, [batch][rows][cols]
  int gdtype;
  int64_t batch, rows, cols;
  void* out;      // orthogonalised matrix, or the parameter when buffer is set
  int odtype;
  float* buffer;  // momentum, or null
  float momentum, blend;  // blend = 1 - momentum
  int nesterov;
  float keep, rate;  // parameter <- keep parameter - rate orthogonal
  int steps;
  float eps, a, b, c;
  // bounds of the iteration (orth_bounds): ||X|| <= min(growth^k, cap), and
  // the scales of the pairs that hold A = X X^T and P
  float growth, cap, sa, sp;
  double amplify;  // what an error of X_0 X_0^T may grow by when it is not formed anew
  float sq;        // scale of the pairs that hold the product of all steps' P
  void* ws;
  // set by the launcher
  double* squares;
  int square_blocks;
  float* scales;  // [batch][steps + 1]: 2^s of X before each step
};

// What the coefficients do to singular values in [0, 1]: fills growth, cap,
// sa, sp.  False where they leave [-16, 16] or are not finite.
bool orth_bounds(OrthArgs& o);

// What the lower half of a pair is multiplied by (ecc_orth.hip).
constexpr float kPairStep = 2048.0f;

inline int64_t orth_pad(int64_t n) { return n <= 64 ? 64 : (n + 127) / 128 * 128; }

// How a product of `batch` matrices of `rows` x `cols` (padded) results is
// shared out: workgroups of `pair` tiles, `tiles` of them a matrix, `whole`
// of which compute theirs alone and the `rest` with `splits` shares each.
struct OrthShare {
  int64_t tile, pair, tiles, whole, rest;
  int splits;
  bool deep;  // four stages in place of two, one workgroup a CU
};
inline OrthShare orth_share(int64_t rows, int64_t cols, int64_t batch, bool sym, int ksteps) {
  OrthShare w{};
  const auto count = [&](int64_t t) {
    const int64_t tm = rows / t, tn = cols / t;
    return sym ? tm * (tm + 1) / 2 : tm * tn;
  };
  w.tile = 64;
  w.pair = 1;
  if (rows >= 128 && cols >= 128 && count(128) * batch * (ksteps >= 16 ? ksteps / 8 : 1) >= 192) w.tile = 128;
  w.tiles = count(w.tile);
  int64_t slots = 512;  // two a CU
  // two tiles a workgroup read fewer columns and have a stage more, but leave
  // one workgroup a CU: better once the sums are long (2000 x 8000: 1.81 ms,
  // 2.22 with one; 1500 x 1500: 475 and 507 us), worse before (12 x 700 x 1000:
  // 746 and 693), and where single tiles come out in whole rounds (4096 x 4096:
  // 4.00 and 3.90 ms)
  const bool even = w.tiles * batch >= 512 && w.tiles * batch % 512 * 16 <= w.tiles * batch;
  if (w.tile == 128 && rows % 256 == 0 && ksteps >= 44 && !even) {
    const int64_t tm = rows / 256;
    w.pair = 2;
    w.tiles = sym ? tm * (tm + 1) : tm * (cols / 128);
    slots = 256;
  }
  const int64_t all = w.tiles * batch;
  // between half a round of one workgroup a CU and a whole one, sharing would
  // leave CUs idle or too much to join (12 x 700 x 1000: 699 us, 714 without)
  w.deep = w.tile == 128 && w.pair == 1 && all > 128 && all <= 256;
  if (w.deep) slots = 256;
  w.whole = all / slots * slots;
  w.rest = all - w.whole;
  w.splits = 1;
  // a share keeps 8 steps, and shares cost a launch more, some 4 us, which is 8 to 16 steps
  if (w.rest && ksteps >= 24) {
    int64_t s = slots / w.rest;
    s = s < ksteps / 8 ? s : ksteps / 8;
    w.splits = s < 1 ? 1 : (int)s;
  }
  if (w.splits == 1) {
    w.whole = all;
    w.rest = 0;
  }
  return w;
}
inline size_t orth_part_bytes(int64_t rows, int64_t cols, int64_t batch, bool sym, int64_t k) {
  const OrthShare w = orth_share(rows, cols, batch, sym, (int)((k + 31) / 32));
  return w.splits > 1 ? (size_t)(w.rest * w.splits * w.pair * w.tile * w.tile) * sizeof(float) : 0;
}

// Workspace: offsets in bytes.
struct OrthPlan {
  int64_t m, n, mpad, npad;
  int square_blocks;
  size_t at_squares, at_scales, at_x0, at_x1, at_xt0, at_xt1, at_a, at_p, at_part, bytes;
};
inline OrthPlan orth_plan(int64_t batch, int64_t rows, int64_t cols) {
  OrthPlan w{};
  w.m = rows < cols ? rows : cols;
  w.n = rows < cols ? cols : rows;
  w.mpad = orth_pad(w.m);
  w.npad = orth_pad(w.n);
  int64_t sb = (w.m * w.n + 8191) / 8192, most = (1024 + batch - 1) / batch;
  w.square_blocks = (int)(sb < most ? sb : most);
  size_t at = 0;
  auto take = [&at](size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) & ~(size_t)255;
    return here;
  };
  const size_t x = (size_t)batch * w.mpad * w.npad * 4, mm = (size_t)batch * w.mpad * w.mpad * 4;
  w.at_squares = take((size_t)batch * w.square_blocks * sizeof(double));
  w.at_scales = take((size_t)batch * 65 * sizeof(float));
  w.at_x0 = take(x);
  w.at_x1 = take(x);
  w.at_xt0 = take(x);
  w.at_xt1 = take(x);
  w.at_a = take(mm);
  w.at_p = take(mm);
  const size_t g = orth_part_bytes(w.mpad, w.mpad, batch, true, w.n);
  const size_t q = orth_part_bytes(w.mpad, w.mpad, batch, true, w.m);
  const size_t u = orth_part_bytes(w.mpad, w.npad, batch, false, w.m);
  const size_t part = g > q ? (g > u ? g : u) : (q > u ? q : u);
  w.at_part = take(part);
  w.bytes = at;
  return w;
}

// Matrices with a short side of at most kThin that are carried through their
// steps by the short side's matrix alone (ecc_orth_thin_kernels.hpp).
constexpr int64_t kThin = 64;
constexpr double kMaxAmplify = 67108864.0;  // 2^26: leaves float64 2^-27
struct ThinPlan {
  int64_t per;  // columns of a workgroup of the first pass, a multiple of 16
  int splits;
  size_t at_part, at_q, at_pow2, bytes;
};
inline ThinPlan thin_plan(int64_t batch, int64_t rows, int64_t cols) {
  ThinPlan w{};
  const int64_t n = rows < cols ? cols : rows;
  // a column costs a workgroup 17 ns of float64 products, a partial sum the
  // one that joins them 0.2 us: balanced at sqrt(n / 12) parts, if a workgroup
  // keeps 128 columns and the launch does not pass the 256 CUs, of which each
  // holds one
  int64_t s = 1;
  while (12 * (s + 1) * (s + 1) <= n) ++s;
  const int64_t fill = batch < 256 ? 256 / batch : 1, most = (n + 127) / 128;
  s = s < fill ? s : fill;
  s = s < most ? s : most;
  w.per = ((n + s - 1) / s + 15) / 16 * 16;
  w.splits = (int)((n + w.per - 1) / w.per);
  size_t at = 0;
  auto take = [&at](size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) & ~(size_t)255;
    return here;
  };
  w.at_part = take((size_t)batch * w.splits * 10 * 256 * sizeof(double));
  w.at_q = take((size_t)batch * 64 * 64 * sizeof(float));
  w.at_pow2 = take((size_t)batch * sizeof(float));
  w.bytes = at;
  return w;
}
inline bool orth_is_thin(const OrthArgs& o) {
  return (o.rows <= kThin || o.cols <= kThin) && o.amplify <= kMaxAmplify;
}

// Long matrices: the same for longer short sides (ecc_orth_long.hip), after
// the direct way's preparation and before its last product, whose pair matrix
// X^T stays where orth_plan puts it; the rest lies behind.
struct LongPlan {
  int64_t m, npad, per;
  int splits;
  size_t square_bytes, at_x, at_part, at_square, bytes;
};
inline LongPlan long_plan(int64_t batch, int64_t rows, int64_t cols) {
  LongPlan w{};
  const OrthPlan d = orth_plan(batch, rows, cols);
  w.m = d.mpad;
  w.npad = d.npad;
  const int64_t b = w.m / 64, tiles = b * (b + 1) / 2 * batch, most = (w.npad + 127) / 128;
  int64_t s = tiles < 256 ? 256 / tiles : 1;  // a workgroup for every CU
  s = s < most ? s : most;
  w.per = ((w.npad + s - 1) / s + 127) / 128 * 128;
  w.splits = (int)((w.npad + w.per - 1) / w.per);
  w.square_bytes = (size_t)batch * w.m * w.m * sizeof(double);
  w.at_x = d.bytes;
  w.at_part = w.at_x + (size_t)batch * w.m * w.npad * sizeof(double);
  w.at_square = w.at_part + (size_t)tiles * w.splits * 4096 * sizeof(double);
  w.bytes = w.at_square + 5 * w.square_bytes;
  return w;
}
// Its float64 products cost some 14 m^3 + m^2 n at a fifth of the direct way's
// rate for 5 m^3 + 15 m^2 n, and few launches less.  Where launches are most
// of it, it gains from n = 2 m on (256 x 512: 113 us, direct 127); where the
// products are, from about 8 m (512 x 4096: 211 and 254; 512 x 1024: 181 and
// 176) or 24 m (4 x 512 x 16384: 1.2 and 1.4 ms; 1024 x 8192: 0.93 and 0.65).
// Nearer to square the two are alike, and Q's rounding would show.
inline bool orth_shape_is_long(int64_t batch, int64_t rows, int64_t cols) {
  const int64_t m = rows < cols ? rows : cols, n = rows < cols ? cols : rows, p = orth_pad(m);
  const double cube = (double)batch * (double)p * (double)p * (double)p;
  const int64_t ratio = cube <= 3.4e7 ? 2 : (cube <= 1.4e8 ? 8 : 24);
  return m > kThin && n >= ratio * m;
}
inline bool orth_is_long(const OrthArgs& o) {
  return orth_shape_is_long(o.batch, o.rows, o.cols) && o.amplify <= kMaxAmplify;
}
// Workspace of whichever way (the coefficients, which decide too, come with the call).
inline size_t orth_workspace_bytes(int64_t batch, int64_t rows, int64_t cols) {
  if (orth_shape_is_long(batch, rows, cols)) return long_plan(batch, rows, cols).bytes;
  const size_t direct = orth_plan(batch, rows, cols).bytes;
  if (rows > kThin && cols > kThin) return direct;
  const size_t thin = thin_plan(batch, rows, cols).bytes;
  return thin > direct ? thin : direct;
}

hipError_t launch_orth(const OrthArgs& o, hipStream_t stream);
// From X (float64, in the workspace, scaled by o.scales) to the pair matrix of
// Q, scaled by o.sq.
hipError_t launch_orth_long(const OrthArgs& o, void* q, void* ws, hipStream_t stream);
template <class GT>
hipError_t launch_orth_thin(const OrthArgs& o, hipStream_t stream);

}  // namespace ecc
