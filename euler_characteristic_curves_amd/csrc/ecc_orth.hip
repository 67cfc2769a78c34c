// Newton-Schulz orthogonalisation and the momentum update built on it
// (contract: include/ecc_train.h).
//
// With X (m x n, m <= n; a tall matrix is transposed on the way in and out)
// scaled to Frobenius norm below 1, a step is
//   A = X X^T,   P = a I + b A + c A A,   X <- P X,
// an odd polynomial of the singular values.  A and P are symmetric: only their
// lower triangle of tiles is computed, and written twice.
//
// Arithmetic.  gfx950's float32 matrix instructions run at a sixteenth of the
// float16 ones, so every operand is held as a pair of float16 numbers, x 2^s =
// hi + 2^-11 lo, 22 bits and a sign together, and a product is three float16
// matrix products, hi hi' + 2^-11 (hi lo' + lo hi'), its two parts summed in
// float32 apart (the dropped lo lo' is below 2^-24).  The exponent s comes from
// a bound of the matrix's entries, so that nothing overflows: per matrix and
// step for X, per call for A and P.  lo has a scale of its own so that it
// reaches as far down as hi does: a pair keeps its 22 bits to 2^-27 of the bound
// and ends at 2^-50, and rows and columns have float32's accuracy of their own
// norm down to 1e-5 of the largest.  (With lo in hi's scale, which saves
// nothing but the second sum, a pair ended at 2^-39: a row at 1e-5 of the others
// was off by 4e-5 to 4e-4 of itself, one at 1e-7 by 0.4 to 5 %; 4096 x 4096 took
// 3.97 ms, 4.01 so.)
//
// What bounds the products of large matrices: the clock, which falls from 2.4 to
// 1.73 GHz under them, and the waits of a step, for its loads and the other
// waves, 23 % of the waves' cycles.  4096 x 4096 takes 4.0 ms, 1.02e15 float16
// operations a second (a library's product of that size in float16: 1.16e15);
// the matrix unit is busy 60 (X X^T) to 63 % (P X) of the cycles that are left.
// Of smaller ones: short sums, the pipeline's start and the launches.  Matrices
// up to 64 across, and long ones, take other ways (orth_is_thin, orth_is_long).
//
// Layout.  A pair matrix keeps blocks of 32 columns one after the other, in
// each its rows of 32 hi and 32 lo, 128 bytes: what a tile loads per step of
// the long axis is one piece, as is the 32 x 32 block a wave writes, and a
// load needs a scalar base and constants only (with rows one after the other,
// 64-bit addresses per lane: 4096 x 4096 4.19 ms, 4.00 then).  Both
// operands of a product lie along the summed axis, so X is kept twice, as X
// and as X^T.  Rows and columns are padded with zeros to the tile, and stay
// zero, so no product checks a bound.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "ecc_act.hpp"
#include "ecc_internal.hpp"
#include "ecc_train_internal.hpp"

namespace ecc {
namespace {

constexpr int kNT = 256;
typedef f16 f16x8 __attribute__((ext_vector_type(8)));
typedef f16 f16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// Offset of element (row, col) of a pair matrix of `rows` rows.
__device__ __forceinline__ int64_t pair_at(int64_t row, int64_t col, int64_t rows) {
  return ((col >> 5) * rows + row) * 64 + (col & 31);
}

// ------------------------------------------------------------- preparation
// The matrix to be orthogonalised, element i of one matrix: the gradient, or
// the momentum buffer after its update, or both mixed (Nesterov).
template <class GT>
__device__ __forceinline__ float update_value(const OrthArgs& p, const GT* g, const float* buf, int64_t i) {
  if (!buf) return (float)g[i];
  const float b = buf[i];  // already the new buffer
  return p.nesterov ? fmaf(p.momentum, b, p.blend * (float)g[i]) : b;
}

// Sums of squares, float64, one slot per workgroup; the momentum buffer is
// updated on the way.
template <class GT>
__global__ __launch_bounds__(kNT) void orth_square_kernel(OrthArgs p) {
  __shared__ double lds[kNT / 64];
  const int64_t n = p.rows * p.cols, off = (int64_t)blockIdx.y * n;
  const GT* g = reinterpret_cast<const GT*>(p.g) + off;
  float* buf = p.buffer ? p.buffer + off : nullptr;
  double s = 0.0;
  const int64_t stride = (int64_t)gridDim.x * kNT;
  const auto add = [&](float gv, float& bv) {
    float u = gv;
    if (buf) {
      bv = fmaf(p.momentum, bv, p.blend * gv);
      u = p.nesterov ? fmaf(p.momentum, bv, p.blend * gv) : bv;
    }
    s = fma((double)u, (double)u, s);
  };
  const int64_t first = (int64_t)blockIdx.x * kNT + threadIdx.x;
#pragma unroll 2
  for (int64_t i = first; i < n / 4; i += stride) {  // four neighbours at a time
    Vec<GT, 4> gv;
    Vec<float, 4> bv = {};
    load_vec(g + i * 4, gv);
    if (buf) load_vec(buf + i * 4, bv);
#pragma unroll
    for (int j = 0; j < 4; ++j) add((float)gv.v[j], bv.v[j]);
    if (buf) store_vec(buf + i * 4, bv);
  }
  if (first < n % 4) {
    const int64_t i = n / 4 * 4 + first;
    float bv = buf ? buf[i] : 0.0f;
    add((float)g[i], bv);
    if (buf) buf[i] = bv;
  }
  for (int d = 1; d < 64; d *= 2) s += __shfl_xor(s, d);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) p.squares[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = (lds[0] + lds[1]) + (lds[2] + lds[3]);
}

// 1 / (norm + eps) of this workgroup's matrix, and the bound of ||X|| that
// follows, from the slots above (every thread gets both).
__device__ __forceinline__ double inverse_norm(const OrthArgs& p, int batch, double* lds, double& bound) {
  double s = 0.0;
  for (int i = threadIdx.x; i < p.square_blocks; i += kNT) s += p.squares[(int64_t)batch * p.square_blocks + i];
  for (int d = 1; d < 64; d *= 2) s += __shfl_xor(s, d);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = s;
  __syncthreads();
  const double norm = sqrt((lds[0] + lds[1]) + (lds[2] + lds[3]));
  const double inv = 1.0 / (norm + (double)p.eps);
  bound = norm * inv;
  return inv;
}

// 2^s for a matrix of entries up to `bound`: the largest entry lands in (2^13, 2^14].
__device__ __forceinline__ float pair_scale(float bound) {
  int e;
  frexpf(fmaxf(bound, 1e-30f), &e);  // bound <= 2^e
  return ldexpf(1.0f, 14 - e);
}

__device__ __forceinline__ void split(float v, f16& hi, f16& lo) {
  hi = (f16)v;
  lo = (f16)((v - (float)hi) * kPairStep);
}

// X and X^T as pairs from a 64 x 64 tile of the input, and the scales of the
// steps.  P1 has the input's orientation, P2 the other.  D, where given, takes
// the place of X (which is the other orientation where rows > cols), in float64.
template <class GT>
__global__ __launch_bounds__(kNT) void orth_prepare_kernel(OrthArgs p, f16* P1, f16* P2, double* D, int64_t rpad, int64_t cpad) {
  __shared__ float tile[64][65];
  __shared__ double lds[kNT / 64];
  const int batch = blockIdx.z;
  double bound;
  const double inv = inverse_norm(p, batch, lds, bound);
  const float sc = pair_scale((float)bound);
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) {
    float r = (float)bound;
    for (int k = 0; k <= p.steps; ++k) {
      p.scales[(int64_t)batch * (p.steps + 1) + k] = pair_scale(r);
      r = fminf(r * p.growth, p.cap);
    }
  }
  const int64_t n = p.rows * p.cols, off = (int64_t)batch * n;
  const GT* g = reinterpret_cast<const GT*>(p.g) + off;
  const float* buf = p.buffer ? p.buffer + off : nullptr;
  const int64_t r0 = (int64_t)blockIdx.y * 64, c0 = (int64_t)blockIdx.x * 64;
  const int tx = threadIdx.x & 63, ty = threadIdx.x >> 6;
#pragma unroll 4
  for (int i = ty; i < 64; i += 4) {
    const int64_t r = r0 + i, c = c0 + tx;
    float v = 0.0f;
    if (r < p.rows && c < p.cols) v = (float)((double)update_value(p, g, buf, r * p.cols + c) * inv) * sc;
    tile[i][tx] = v;
  }
  __syncthreads();
  f16* out1 = P1 + (int64_t)batch * rpad * 2 * cpad;
  f16* out2 = P2 + (int64_t)batch * rpad * 2 * cpad;
  const bool tall = p.rows > p.cols;
  if (D) {
    D += (int64_t)batch * rpad * cpad;
    for (int i = ty; i < 64; i += 4) {
      if (tall)
        D[(c0 + i) * rpad + r0 + tx] = (double)tile[tx][i];
      else
        D[(r0 + i) * cpad + c0 + tx] = (double)tile[i][tx];
    }
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int at = q * kNT + threadIdx.x, row = at >> 4, ch = at & 15;
    const int k = (ch >> 3) * 32 + (ch & 3) * 8;
    const bool low = (ch >> 2) & 1;
    f16x8 a, b;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      f16 hi, lo;
      split(tile[row][k + j], hi, lo);
      a[j] = low ? lo : hi;
      split(tile[k + j][row], hi, lo);
      b[j] = low ? lo : hi;
    }
    if (!D || tall) *reinterpret_cast<f16x8*>(out1 + pair_at(r0 + row, c0 + (ch >> 3) * 32, rpad) + (ch & 7) * 8) = a;
    if (!D || !tall) *reinterpret_cast<f16x8*>(out2 + pair_at(c0 + row, r0 + (ch >> 3) * 32, cpad) + (ch & 7) * 8) = b;
  }
}

// ----------------------------------------------------------------- products
enum Kind { kGram, kPoly, kUpdate, kLast };

// One product, out = A B^T over pair matrices, and what becomes of it.
struct Product {
  const f16 *A, *B;    // [batch][rows][2 kpad]
  int64_t sA, sB;      // batch strides, elements
  int64_t rowsA, rowsB;  // padded
  int ksteps;          // steps of 32 columns that are not all padding
  int tiles, tiles_n;  // workgroups of one matrix, column tiles
  int whole;           // workgroups, of all matrices, that one workgroup computes
  int splits;          // workgroups that share the columns of each of the others
  float* part;         // their float32 sums
  int step;
  float sa, sp;        // scales of A and of P
  f16 *out, *outT;     // pair matrices written (outT: the transpose, of kUpdate)
  int64_t sOut, out_rows, outT_rows;
  const f16* gram;     // kPoly: the matrix A itself
  OrthArgs o;
};

template <int T>
constexpr int kFrag = T / 64;  // 32 x 32 fragments per wave and axis (4 waves, 2 x 2, to T x T results)

// A workgroup computes R tiles of T x T that share their columns, four waves
// to each.  Row and column tile of the first one of workgroup `t`.  Symmetric
// products enumerate the lower triangle, row by row; with R = 2 the last block
// of a row ends in a tile above the diagonal, which is left out at the end.
template <int R>
__device__ __forceinline__ void tile_of(bool sym, int t, int tiles_n, int& ti, int& tj) {
  if (sym) {
    // rows of i + 1 tiles, or of 2 i + 2
    int i = R == 1 ? (int)((sqrtf(8.0f * (float)t + 1.0f) - 1.0f) * 0.5f) : (int)((sqrtf(4.0f * (float)t + 1.0f) - 1.0f) * 0.5f);
    const auto before = [](int k) { return R == 1 ? k * (k + 1) / 2 : k * (k + 1); };
    while (before(i + 1) <= t) ++i;
    while (before(i) > t) --i;
    ti = R * i;
    tj = t - before(i);
  } else {
    ti = t / tiles_n;
    tj = t - ti * tiles_n;
    ti *= R;
  }
}

// Four neighbouring results of the last step, columns i..i+3 of row j of the
// short side's view, in the caller's orientation.
template <class PT>
__device__ __forceinline__ void store_result(const OrthArgs& o, int64_t batch, int64_t i, int64_t j, const float* v) {
  PT* out = reinterpret_cast<PT*>(o.out) + batch * o.rows * o.cols;
  if (o.rows > o.cols) {  // row j, columns i..i+3: one access
    if (j >= o.rows) return;
    out += j * o.cols + i;
    if (i + 4 <= o.cols) {
      Vec<PT, 4> r;
      if (o.buffer) load_vec(out, r);
#pragma unroll
      for (int k = 0; k < 4; ++k) r.v[k] = (PT)(o.buffer ? fmaf((float)r.v[k], o.keep, -o.rate * v[k]) : v[k]);
      store_vec(out, r);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (i + k < o.cols) out[k] = (PT)(o.buffer ? fmaf((float)out[k], o.keep, -o.rate * v[k]) : v[k]);
    }
    return;
  }
  if (j >= o.cols) return;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (i + k >= o.rows) return;
    PT* at = out + (i + k) * o.cols + j;
    *at = (PT)(o.buffer ? fmaf((float)*at, o.keep, -o.rate * v[k]) : v[k]);
  }
}

// 32 x 32 values of a wave as pairs, through 4 KB of LDS of its own, so that
// they are written as one piece: a lane holds column lane % 32 of rows
// 8 q + 4 (lane / 32) + r.  TURN: the rows written are those columns.  `out`:
// where the block lies.  Chunks of 16 bytes are permuted by the row.
template <bool TURN>
__device__ __forceinline__ void store_block(f16* out, const f32x16& v, f16* lds) {
  const int lane = threadIdx.x & 63, c = lane & 31, h = lane >> 5;
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if constexpr (TURN) {
      f16x4 hi, lo;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        f16 a, b;
        split(v[q * 4 + r], a, b);
        hi[r] = a;
        lo[r] = b;
      }
      *reinterpret_cast<f16x4*>(lds + c * 64 + ((q ^ (c & 7)) << 3) + h * 4) = hi;
      *reinterpret_cast<f16x4*>(lds + c * 64 + (((q + 4) ^ (c & 7)) << 3) + h * 4) = lo;
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = q * 8 + h * 4 + r;
        f16 a, b;
        split(v[q * 4 + r], a, b);
        lds[row * 64 + (((c >> 3) ^ (row & 7)) << 3) + (c & 7)] = a;
        lds[row * 64 + ((((c >> 3) + 4) ^ (row & 7)) << 3) + (c & 7)] = b;
      }
    }
  }
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    const int row = n * 8 + (lane >> 3), ch = lane & 7;
    *reinterpret_cast<f16x8*>(out + row * 64 + ch * 8) =
        *reinterpret_cast<const f16x8*>(lds + row * 64 + ((ch ^ (row & 7)) << 3));
  }
}

// One fragment of a wave's results; lds: 4 KB of its own.
template <int T, int KIND, class PT>
__device__ __forceinline__ void epilogue(const Product& p, int batch, int ti, int tj, int fi, int fj, f32x16 v, f16* lds) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6 & 3;
  if ((KIND == kGram || KIND == kPoly) && ti < tj) return;
  const float* xs = p.o.scales + (int64_t)batch * (p.o.steps + 1) + p.step;
  float f;
  if constexpr (KIND == kGram)
    f = p.sa / (xs[0] * xs[0]);
  else if constexpr (KIND == kPoly)
    f = p.o.c * p.sp / (p.sa * p.sa);
  else if constexpr (KIND == kUpdate)
    f = xs[1] / (p.sp * xs[0]);
  else
    f = 1.0f / (p.sp * xs[0]);
  const int64_t j0 = (int64_t)tj * T + (wave & 1) * (T / 2) + fj * 32, i0 = (int64_t)ti * T + (wave >> 1) * (T / 2) + fi * 32;
  const int64_t j = j0 + (lane & 31);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int64_t i = i0 + q * 8 + (lane >> 5) * 4;
    float u[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) u[r] = v[q * 4 + r] * f;
    if constexpr (KIND == kPoly) {
      const f16* gp = p.gram + (int64_t)batch * p.sOut + pair_at(j, i, p.out_rows);
      const f16x4 gh = *reinterpret_cast<const f16x4*>(gp), gl = *reinterpret_cast<const f16x4*>(gp + 32);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        u[r] = fmaf(p.o.b * p.sp / p.sa, fmaf((float)gl[r], 1.0f / kPairStep, (float)gh[r]), u[r]);
        if (i + r == j) u[r] += p.o.a * p.sp;
      }
    }
    if constexpr (KIND == kLast) store_result<PT>(p.o, batch, i, j, u);
#pragma unroll
    for (int r = 0; r < 4; ++r) v[q * 4 + r] = u[r];
  }
  if constexpr (KIND == kLast) return;
  f16* out = p.out + (int64_t)batch * p.sOut;
  f16* turned = KIND == kUpdate ? p.outT + (int64_t)batch * p.sOut : out;
  store_block<true>(turned + pair_at(j0, i0, KIND == kUpdate ? p.outT_rows : p.out_rows), v, lds);
  if (KIND == kUpdate || ti != tj) store_block<false>(out + pair_at(i0, j0, p.out_rows), v, lds);
}

// Loads one step (32 columns, T rows, 128 bytes a row) of an operand to LDS.
// A wave's load covers 8 rows; the 16-byte chunk a lane fetches is permuted
// within its row by half the row's number, so that the 16 lanes a fragment's
// read serves at a time, 16 rows at one chunk, meet every bank once: two rows
// fill the banks, and eight pairs of rows have eight chunks.
// `step`: where the step's rows begin, the same for every lane, so that a load
// has a scalar base, a register of offsets (in_step; its bit 6 turns in every
// second load) and a constant, which the hardware adds to both addresses.
template <int ROWS, int WAVES>
__device__ __forceinline__ uint32_t in_step() {
  static_assert(ROWS / WAVES % 16 == 0, "the permutation repeats after 16 rows");
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane >> 3;
  return (uint32_t)(wave * (ROWS / WAVES) * 128 + r * 128 + ((lane & 7) ^ (r >> 1)) * 16);
}
template <int N>
__device__ __forceinline__ void load_rows(const char* even, const char* odd, f16* dst) {
  if constexpr (N > 1) load_rows<N - 1>(even, odd, dst);
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(N % 2 ? even : odd),
                                   (__attribute__((address_space(3))) void*)dst, 16, (N - 1) * 1024, 0);
}
template <int ROWS, int WAVES>
__device__ __forceinline__ void load_step(const f16* step, uint32_t offset, f16* lds) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const char* base = reinterpret_cast<const char*>(step);
  load_rows<ROWS / 8 / WAVES>(base + offset, base + (offset ^ 64), lds + wave * (ROWS / WAVES) * 64);
}

template <int T>
__device__ __forceinline__ f16x8 fragment(const f16* lds, int row, int chunk) {
  return *reinterpret_cast<const f16x8*>(lds + row * 64 + ((chunk ^ (row >> 1 & 7)) << 3));
}

// The first products' fragments are read, then one more with every product.
template <int T>
__device__ __forceinline__ void multiply_step(const f16* la, const f16* lb, f32x16 (&acc)[kFrag<T>][kFrag<T>],
                                              f32x16 (&low)[kFrag<T>][kFrag<T>]) {
  constexpr int F = kFrag<T>;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int ra = (wave >> 2) * T + (wave >> 1 & 1) * (T / 2) + (lane & 31), rb = (wave & 1) * (T / 2) + (lane & 31);
  f16x8 ah[2][F], al[2][F], bh[2][F], bl[2][F];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int ch = s * 2 + (lane >> 5);
#pragma unroll
    for (int i = 0; i < F; ++i) {
      ah[s][i] = fragment<T>(la, ra + i * 32, ch);
      bh[s][i] = fragment<T>(lb, rb + i * 32, ch);
    }
#pragma unroll
    for (int i = 0; i < F; ++i) {
      bl[s][i] = fragment<T>(lb, rb + i * 32, ch + 4);
      al[s][i] = fragment<T>(la, ra + i * 32, ch + 4);
    }
  }
#pragma unroll
  for (int s = 0; s < 2; ++s) {
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
      for (int j = 0; j < F; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(ah[s][i], bh[s][j], acc[i][j], 0, 0, 0);
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
      for (int j = 0; j < F; ++j)
        low[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(ah[s][i], bl[s][j], low[i][j], 0, 0, 0);
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
      for (int j = 0; j < F; ++j)
        low[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(al[s][i], bh[s][j], low[i][j], 0, 0, 0);
  }
  __builtin_amdgcn_sched_group_barrier(0x100, 2 * F, 0);
#pragma unroll
  for (int i = 0; i < 6 * F; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
  }
  __builtin_amdgcn_sched_group_barrier(0x008, 6 * F * F - 6 * F, 0);
}

// Waits for all but the newest N steps' loads of this wave and for what it has
// read of LDS, then for the other waves.  (A workgroup fence would wait for
// every load; one block, and ordered with memory, so that no read of LDS is
// still on its way when another wave's loads overwrite it.)
template <int T, int R, int N>
__device__ __forceinline__ void wait_step() {
  constexpr int vm = N * (T / 32 + T / 32 / R);  // loads a wave issues per step
  __builtin_amdgcn_s_waitcnt((vm & 15) | 0x0070 | ((vm >> 4) << 14));  // the same, known to the compiler
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(vm) : "memory");
}

// R tiles of a product, or a share of their columns.  S: steps of the long
// axis that are in LDS or on their way to it, the one in use counted.
template <int T, int R, int S, int KIND, class PT>
__global__ __launch_bounds__(kNT * R, T == 128 && S == 4 ? 1 : 2) void product_kernel(Product p) {
  constexpr int F = kFrag<T>, A = T * R * 64, B = T * 64;
  // arrays of their own, so that a read of one is known not to wait for another's loads
  __shared__ __align__(16) f16 a0[A], b0[B], a1[A], b1[B];
  __shared__ __align__(16) f16 a2[S > 2 ? A : 8], b2[S > 2 ? B : 8], a3[S > 3 ? A : 8], b3[S > 3 ? B : 8];
  const int rest = (int)blockIdx.x - p.whole;
  const int all = rest < 0 ? (int)blockIdx.x : p.whole + rest / p.splits, sp = rest < 0 ? 0 : rest % p.splits;
  const int batch = all / p.tiles;
  int ti, tj;
  tile_of<R>(KIND == kGram || KIND == kPoly, all - batch * p.tiles, p.tiles_n, ti, tj);
  ti = __builtin_amdgcn_readfirstlane(ti);
  tj = __builtin_amdgcn_readfirstlane(tj);
  const int per = rest < 0 ? p.ksteps : (p.ksteps + p.splits - 1) / p.splits;
  const int k0 = sp * per, k1 = k0 + per < p.ksteps ? k0 + per : p.ksteps;
  const f16* Ap = p.A + batch * p.sA + (int64_t)ti * T * 64;
  const f16* Bp = p.B + batch * p.sB + (int64_t)tj * T * 64;
  const uint32_t offA = in_step<T * R, 4 * R>(), offB = in_step<T, 4 * R>();
  f32x16 acc[F][F], low[F][F];
#pragma unroll
  for (int i = 0; i < F; ++i)
#pragma unroll
    for (int j = 0; j < F; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = low[i][j][r] = 0.0f;
  const auto load = [&](int k, f16* la, f16* lb) {
    if (k < k1) {
      load_step<T * R, 4 * R>(Ap + k * p.rowsA * 64, offA, la);
      load_step<T, 4 * R>(Bp + k * p.rowsB * 64, offB, lb);
    }
  };
  // step k, whose loads are complete, and the loads of step k + S - 1 into the
  // buffer that step k - 1 has left
  const auto step = [&](int k, f16* la, f16* lb, f16* na, f16* nb) {
    if (k >= k1) return;
    const int newer = k1 - 1 - k;
    if (newer >= S - 2)
      wait_step<T, R, S - 2>();
    else if (S > 3 && newer == 1)
      wait_step<T, R, 1>();
    else
      wait_step<T, R, 0>();
    load(k + S - 1, na, nb);
    multiply_step<T>(la, lb, acc, low);
  };
  load(k0, a0, b0);
  if constexpr (S == 2) {
    for (int k = k0; k < k1; k += 2) {
      step(k, a0, b0, a1, b1);
      step(k + 1, a1, b1, a0, b0);
    }
  } else if constexpr (S == 3) {
    load(k0 + 1, a1, b1);
    for (int k = k0; k < k1; k += 3) {
      step(k, a0, b0, a2, b2);
      step(k + 1, a1, b1, a0, b0);
      step(k + 2, a2, b2, a1, b1);
    }
  } else {
    load(k0 + 1, a1, b1);
    load(k0 + 2, a2, b2);
    for (int k = k0; k < k1; k += 4) {
      step(k, a0, b0, a3, b3);
      step(k + 1, a1, b1, a0, b0);
      step(k + 2, a2, b2, a1, b1);
      step(k + 3, a3, b3, a2, b2);
    }
  }
#pragma unroll
  for (int i = 0; i < F; ++i)
#pragma unroll
    for (int j = 0; j < F; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = fmaf(low[i][j][r], 1.0f / kPairStep, acc[i][j][r]);
  const int half = threadIdx.x / kNT;
  if (rest >= 0 && p.splits > 1) {
    float* out = p.part + ((int64_t)rest * R + half) * (T * T) + threadIdx.x % kNT * 4;
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
      for (int j = 0; j < F; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          f32x4 v;
#pragma unroll
          for (int r = 0; r < 4; ++r) v[r] = acc[i][j][q * 4 + r];
          *reinterpret_cast<f32x4*>(out + ((i * F + j) * 4 + q) * (4 * kNT)) = v;
        }
    return;
  }
  wait_step<T, R, 0>();  // the stages are free: 4 KB of the first ones for each wave
  f16* mine = R == 1 ? (threadIdx.x < kNT / 2 ? a0 : b0) + (threadIdx.x >> 6 & 1) * 2048 : a0 + (threadIdx.x >> 6) * 2048;
#pragma unroll
  for (int i = 0; i < F; ++i)
#pragma unroll
    for (int j = 0; j < F; ++j) epilogue<T, KIND, PT>(p, batch, ti + half, tj, i, j, acc[i][j], mine);
}

// Joins the shares of a tile, in order, and finishes it: blockIdx.y is the
// fragment of each of the four waves.
template <int T, int R, int KIND, class PT>
__global__ __launch_bounds__(kNT) void finish_kernel(Product p) {
  constexpr int F = kFrag<T>;
  constexpr int64_t next = (int64_t)R * T * T;  // from one share to the next
  __shared__ __align__(16) f16 lds[4 * 2048];
  const int block = (int)blockIdx.x / R, half = (int)blockIdx.x % R;
  const int all = p.whole + block, batch = all / p.tiles;
  int ti, tj;
  tile_of<R>(KIND == kGram || KIND == kPoly, all - batch * p.tiles, p.tiles_n, ti, tj);
  const float* in = p.part + block * p.splits * next + half * (T * T) + (int64_t)blockIdx.y * (16 * kNT) + threadIdx.x * 4;
  f32x4 s[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) s[q] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  int k = 0;
  for (; k + 3 <= p.splits; k += 3) {
    f32x4 v[3][4];
#pragma unroll
    for (int u = 0; u < 3; ++u)
#pragma unroll
      for (int q = 0; q < 4; ++q) v[u][q] = *reinterpret_cast<const f32x4*>(in + (k + u) * next + q * (4 * kNT));
#pragma unroll
    for (int u = 0; u < 3; ++u)
#pragma unroll
      for (int q = 0; q < 4; ++q) s[q] += v[u][q];
  }
  for (; k < p.splits; ++k)
#pragma unroll
    for (int q = 0; q < 4; ++q) s[q] += *reinterpret_cast<const f32x4*>(in + k * next + q * (4 * kNT));
  f32x16 v;
#pragma unroll
  for (int q = 0; q < 4; ++q)
#pragma unroll
    for (int r = 0; r < 4; ++r) v[q * 4 + r] = s[q][r];
  epilogue<T, KIND, PT>(p, batch, ti + half, tj, (int)blockIdx.y / F, (int)blockIdx.y % F, v, lds + (threadIdx.x >> 6) * 2048);
}

template <int T, int R, int S, int KIND, class PT>
hipError_t launch_product_t(Product p, const OrthShare& w, int64_t cols, hipStream_t s) {
  p.tiles = (int)w.tiles;
  p.tiles_n = (int)(cols / T);
  p.whole = (int)w.whole;
  p.splits = w.splits;
  hipLaunchKernelGGL((product_kernel<T, R, S, KIND, PT>), dim3((unsigned)(w.whole + w.rest * w.splits)), dim3(kNT * R), 0, s,
                     p);
  if (w.splits > 1)
    hipLaunchKernelGGL((finish_kernel<T, R, KIND, PT>), dim3((unsigned)(w.rest * R), kFrag<T> * kFrag<T>), dim3(kNT), 0, s,
                       p);
  return hipGetLastError();
}

template <int KIND, class PT>
hipError_t launch_product(const Product& p, int64_t rows, int64_t cols, int64_t batch, hipStream_t s) {
  const OrthShare w = orth_share(rows, cols, batch, KIND == kGram || KIND == kPoly, p.ksteps);
  if (w.tile == 64) return launch_product_t<64, 1, 4, KIND, PT>(p, w, cols, s);
  if (w.pair == 2) return launch_product_t<128, 2, 3, KIND, PT>(p, w, cols, s);
  if (w.deep) return launch_product_t<128, 1, 4, KIND, PT>(p, w, cols, s);
  return launch_product_t<128, 1, 2, KIND, PT>(p, w, cols, s);
}

template <class GT, class PT>
hipError_t run(const OrthArgs& o, hipStream_t s) {
  const OrthPlan w = orth_plan(o.batch, o.rows, o.cols);
  OrthArgs a = o;
  char* ws = reinterpret_cast<char*>(o.ws);
  a.squares = reinterpret_cast<double*>(ws + w.at_squares);
  a.scales = reinterpret_cast<float*>(ws + w.at_scales);
  a.square_blocks = w.square_blocks;
  f16* X[2] = {reinterpret_cast<f16*>(ws + w.at_x0), reinterpret_cast<f16*>(ws + w.at_x1)};
  f16* XT[2] = {reinterpret_cast<f16*>(ws + w.at_xt0), reinterpret_cast<f16*>(ws + w.at_xt1)};
  f16* A = reinterpret_cast<f16*>(ws + w.at_a);
  f16* P = reinterpret_cast<f16*>(ws + w.at_p);
  float* part = reinterpret_cast<float*>(ws + w.at_part);

  hipLaunchKernelGGL((orth_square_kernel<GT>), dim3((unsigned)w.square_blocks, (unsigned)a.batch), dim3(kNT), 0, s, a);
  const bool tall = a.rows > a.cols;
  const int64_t rpad = tall ? w.npad : w.mpad, cpad = tall ? w.mpad : w.npad;
  hipLaunchKernelGGL((orth_prepare_kernel<GT>), dim3((unsigned)(cpad / 64), (unsigned)(rpad / 64), (unsigned)a.batch),
                     dim3(kNT), 0, s, a, tall ? XT[0] : X[0], tall ? X[0] : XT[0],
                     orth_is_long(a) ? reinterpret_cast<double*>(ws + long_plan(a.batch, a.rows, a.cols).at_x) : nullptr,
                     rpad, cpad);
  const int64_t sx = w.mpad * w.npad * 2, sm = w.mpad * w.mpad * 2;
  if (orth_is_long(a)) {
    const hipError_t e = launch_orth_long(a, P, a.ws, s);
    if (e != hipSuccess) return e;
    Product p{};
    p.o = a;
    p.sp = a.sq;
    p.part = part;
    p.A = P;
    p.sA = sm;
    p.B = XT[0];
    p.sB = sx;
    p.rowsA = w.mpad;
    p.rowsB = w.npad;
    p.ksteps = (int)((w.m + 31) / 32);
    return launch_product<kLast, PT>(p, w.mpad, w.npad, a.batch, s);
  }
  for (int k = 0; k < a.steps; ++k) {
    const int in = k & 1, on = 1 - in;
    Product p{};
    p.o = a;
    p.step = k;
    p.sa = a.sa;
    p.sp = a.sp;
    p.part = part;
    p.A = p.B = X[in];
    p.sA = p.sB = sx;
    p.rowsA = p.rowsB = w.mpad;
    p.ksteps = (int)((w.n + 31) / 32);
    p.out = A;
    p.sOut = sm;
    p.out_rows = w.mpad;
    hipError_t e = launch_product<kGram, float>(p, w.mpad, w.mpad, a.batch, s);
    if (e != hipSuccess) return e;
    p.A = p.B = p.gram = A;
    p.sA = p.sB = sm;
    p.ksteps = (int)((w.m + 31) / 32);
    p.out = P;
    e = launch_product<kPoly, float>(p, w.mpad, w.mpad, a.batch, s);
    if (e != hipSuccess) return e;
    p.A = P;
    p.B = XT[in];
    p.sB = sx;
    p.rowsB = w.npad;
    p.out = X[on];
    p.outT = XT[on];
    p.sOut = sx;
    p.outT_rows = w.npad;
    e = k + 1 < a.steps ? launch_product<kUpdate, float>(p, w.mpad, w.npad, a.batch, s)
                        : launch_product<kLast, PT>(p, w.mpad, w.npad, a.batch, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <class GT>
hipError_t run_out(const OrthArgs& o, int odtype, hipStream_t s) {
  if (odtype == kTF32) return run<GT, float>(o, s);
  if (odtype == kTF16) return run<GT, f16>(o, s);
  return run<GT, bf16>(o, s);
}

}  // namespace

hipError_t launch_orth(const OrthArgs& o, hipStream_t s) {
  if (orth_is_thin(o)) {
    if (o.gdtype == kTF32) return launch_orth_thin<float>(o, s);
    if (o.gdtype == kTF16) return launch_orth_thin<f16>(o, s);
    return launch_orth_thin<bf16>(o, s);
  }
  if (o.gdtype == kTF32) return run_out<float>(o, o.odtype, s);
  if (o.gdtype == kTF16) return run_out<f16>(o, o.odtype, s);
  return run_out<bf16>(o, o.odtype, s);
}

}  // namespace ecc
