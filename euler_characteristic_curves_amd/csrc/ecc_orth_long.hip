// The steps of a Newton-Schulz orthogonalisation on the short side's matrix
// alone, for matrices whose long side is many times their short side, of more
// than 64 (shorter ones: ecc_orth_thin_kernels.hpp, which has the mathematics
// and the reason for float64; the other products: ecc_orth.hip).
//
// X comes as a float64 matrix, and Q leaves as a pair matrix, so that what is
// left of X's products is A_0 = X X^T here and the last product of the direct
// iteration, with Q for P.  For m x n that is m^2 n + 14 m^3 operations in float64 (symmetric
// products, 5 steps) in place of 15 m^2 n + 5 m^3, each three float16 products;
// the float64 matrix rate is a fifth of what those three reach, so the long
// side has to be several times the short one (orth_is_long).
//
// What bounds it: A_0, the float64 matrix rate (512 x 16384: 83 to 87 us, 4.8e9
// operations, 55e12 a second; a library's 4096^3 product in float64 68e12);
// the 14 products of the short side, their launches and L2's latency, 5 to 9 us
// each.  In all 330 us of a momentum step of 512 x 16384, 483 by the direct way.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ecc_act.hpp"
#include "ecc_internal.hpp"
#include "ecc_train_internal.hpp"

namespace ecc {
namespace {

constexpr int kNT = 512;
constexpr int kNW = kNT / 64;
typedef double f64x2 __attribute__((ext_vector_type(2)));
typedef double f64x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ void triangle(int t, int& i, int& j) {
  i = (int)((sqrtf(8.0f * (float)t + 1.0f) - 1.0f) * 0.5f);
  while ((i + 1) * (i + 2) / 2 <= t) ++i;
  while (i * (i + 1) / 2 > t) --i;
  j = t - i * (i + 1) / 2;
}

struct Long {
  OrthArgs o;
  const double* x;  // [batch][m][npad]
  double* part;    // [batch][pairs of 64 rows][splits][64 x 64], tile order
  int64_t m, npad;  // m: padded
  int64_t pairs;    // tiles of 64 x 64, lower triangle
  int64_t per;     // columns of a share, a multiple of 128
  int splits;
};

// A 64 x 64 tile of X X^T over a share of the columns.  A wave takes 8
// columns: a lane has 2 of row 16 I + lane % 16 of each of the eight tile
// rows, and the next 8 on their way.  The float64 matrix instructions keep the
// vector unit to themselves, so the loop has next to nothing else for it (X in
// pairs, converted here, or chunks whose registers overflow into the
// accumulation file: 102 to 113 us of 512 x 16384).  Workgroups go to the
// eight dies in turn, so that numbers eight apart share an L2: those get the
// tiles of one share, which read the same columns.
__global__ __launch_bounds__(kNT) void long_gram_kernel(Long t) {
  __shared__ double lds[kNW * 4 * 256];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15, q = lane >> 4;
  const int64_t slot = (int64_t)(blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3);
  if (slot >= t.pairs * t.splits * t.o.batch) return;
  const int64_t pair = slot % t.pairs, share = slot / t.pairs % t.splits, batch = slot / t.pairs / t.splits;
  int bi, bj;
  triangle((int)pair, bi, bj);
  const double* x = t.x + batch * t.m * t.npad + r * t.npad + q * 2;
  const double* row[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) row[i] = x + ((i < 4 ? bi : bj) * 64 + (i & 3) * 16) * t.npad;
  const int64_t c0 = share * t.per, c1 = c0 + t.per < t.npad ? c0 + t.per : t.npad;
  f64x4 acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f64x4{0.0, 0.0, 0.0, 0.0};
  const auto fetch = [&](int64_t c, f64x2 (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = *reinterpret_cast<const f64x2*>(row[i] + c);
  };
  const auto use = [&](const f64x2 (&v)[8]) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f64_16x16x4f64(v[i][k], v[4 + j][k], acc[i][j], 0, 0, 0);
  };
  // a share is a multiple of 128 columns: an even number of chunks for each
  // wave, so the loop needs no condition (which costs it copies of the sums);
  // the last chunk is loaded once too often
  constexpr int64_t step = kNW * 8;
  f64x2 u[8], v[8];
  fetch(c0 + wave * 8, u);
  for (int64_t c = c0 + wave * 8; c < c1; c += 2 * step) {
    fetch(c + step, v);
    use(u);
    fetch(c + 2 * step < c1 ? c + 2 * step : c, u);
    use(v);
  }
  double* out = t.part + ((batch * t.pairs + pair) * t.splits + share) * 4096;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) lds[(wave * 4 + j) * 256 + k * 64 + lane] = acc[i][j][k];
    __syncthreads();
#pragma unroll
    for (int e = threadIdx.x; e < 1024; e += kNT) {
      double s = 0.0;
#pragma unroll
      for (int w = 0; w < kNW; ++w) s += lds[w * 1024 + e];
      out[i * 1024 + e] = s;
    }
  }
}

// The shares of a tile, in order, to A, both triangles, without X's scale.
// blockIdx.x: quarter of the tile; .y: tile; .z: matrix.
__global__ __launch_bounds__(256) void long_join_kernel(Long t, double* A) {
  int bi, bj;
  triangle(blockIdx.y, bi, bj);
  const double* in = t.part + ((int64_t)blockIdx.z * gridDim.y + blockIdx.y) * t.splits * 4096;
  const double sc = (double)t.o.scales[(int64_t)blockIdx.z * (t.o.steps + 1)], inv = 1.0 / (sc * sc);
  double* a = A + (int64_t)blockIdx.z * t.m * t.m;
  double s[4] = {0.0, 0.0, 0.0, 0.0};
  int k = 0;
  for (; k + 4 <= t.splits; k += 4) {
    double v[4][4];
#pragma unroll
    for (int w = 0; w < 4; ++w)
#pragma unroll
      for (int u = 0; u < 4; ++u) v[w][u] = in[(int64_t)(k + w) * 4096 + blockIdx.x * 1024 + u * 256 + threadIdx.x];
#pragma unroll
    for (int u = 0; u < 4; ++u) s[u] += (v[0][u] + v[1][u]) + (v[2][u] + v[3][u]);
  }
  for (; k < t.splits; ++k)
#pragma unroll
    for (int u = 0; u < 4; ++u) s[u] += in[(int64_t)k * 4096 + blockIdx.x * 1024 + u * 256 + threadIdx.x];
#pragma unroll
  for (int u = 0; u < 4; ++u) {  // u: column tile
    const int row = bi * 64 + (int)blockIdx.x * 16 + 4 * (threadIdx.x >> 6) + ((threadIdx.x >> 4) & 3);
    const int col = bj * 64 + u * 16 + (threadIdx.x & 15);
    a[(int64_t)row * t.m + col] = s[u] * inv;
    if (bi != bj) a[(int64_t)col * t.m + row] = s[u] * inv;
  }
}

// Products of commuting symmetric matrices [batch][m][m]: C = X Y, or the
// polynomial c X X + b X + a I (poly), or X Y as a pair matrix times `scale`.
// blockIdx.x: 32 x 32 tile of the lower triangle; .y: one of up to two products.
// A tile below the diagonal is written twice; one on it is whole by itself, and
// its two halves, which differ in their last bits, each have one writer.
struct Square {
  const double* x[2];
  const double* y[2];
  double* out[2];
  f16* pair;
  double a, b, c, scale;
  int poly;
  int64_t m;
};

__global__ __launch_bounds__(kNT) void long_square_kernel(Square p) {
  __shared__ double lds[kNW * 1024];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, q = lane >> 4;
  int bi, bj;
  triangle(blockIdx.x, bi, bj);
  const int64_t off = (int64_t)blockIdx.z * p.m * p.m;
  const int second = blockIdx.y;
  const double* X = (second ? p.x[1] : p.x[0]) + off;
  const double* Y = (second ? p.y[1] : p.y[0]) + off;
  // a wave sums an eighth of the rows; a lane's two columns are neighbours, so
  // element a of tile I is 2 a + I
  const int64_t rows = p.m / kNW, k0 = wave * rows;
  const double* xp = X + (k0 + q) * p.m + bi * 32 + r * 2;
  const double* yp = Y + (k0 + q) * p.m + bj * 32 + r * 2;
  f64x4 acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = f64x4{0.0, 0.0, 0.0, 0.0};
  for (int64_t k = 0; k < rows; k += 16) {  // m is a multiple of 128
    f64x2 xv[4], yv[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      xv[u] = *reinterpret_cast<const f64x2*>(xp + (k + 4 * u) * p.m);
      yv[u] = *reinterpret_cast<const f64x2*>(yp + (k + 4 * u) * p.m);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f64_16x16x4f64(xv[u][i], yv[u][j], acc[i][j], 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) lds[wave * 1024 + (i * 2 + j) * 256 + k * 64 + lane] = acc[i][j][k];
  __syncthreads();
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int e = u * kNT + threadIdx.x, i = e >> 9, j = (e >> 8) & 1;
    double s = 0.0;
#pragma unroll
    for (int w = 0; w < kNW; ++w) s += lds[w * 1024 + e];
    const int64_t row = bi * 32 + 2 * (4 * ((e >> 6) & 3) + ((e >> 4) & 3)) + i, col = bj * 32 + 2 * (e & 15) + j;
    if (p.poly) {
      s = fma(p.c, s, p.b * X[row * p.m + col]);
      if (row == col) s += p.a;
    }
    if (p.pair) {
      const float v = (float)(s * p.scale);
      const f16 hi = (f16)v, lo = (f16)((v - (float)hi) * kPairStep);
      f16* out = p.pair + off * 2;
      const int64_t at = ((col >> 5) * p.m + row) * 64 + (col & 31), to = ((row >> 5) * p.m + col) * 64 + (row & 31);
      out[at] = hi;
      out[at + 32] = lo;
      if (bi != bj) {
        out[to] = hi;
        out[to + 32] = lo;
      }
    } else {
      double* out = (second ? p.out[1] : p.out[0]) + off;
      out[row * p.m + col] = s;
      if (bi != bj) out[col * p.m + row] = s;
    }
  }
}

}  // namespace

hipError_t launch_orth_long(const OrthArgs& o, void* q_pairs, void* ws, hipStream_t s) {
  f16* q = reinterpret_cast<f16*>(q_pairs);
  const LongPlan w = long_plan(o.batch, o.rows, o.cols);
  char* base = reinterpret_cast<char*>(ws);
  double* buf[5];
  for (int i = 0; i < 5; ++i) buf[i] = reinterpret_cast<double*>(base + w.at_square + (size_t)i * w.square_bytes);
  double *A = buf[0], *W = buf[1], *P = buf[2], *Q = buf[3], *Q1 = buf[4];
  Long t{};
  t.o = o;
  t.x = reinterpret_cast<const double*>(base + w.at_x);
  t.part = reinterpret_cast<double*>(base + w.at_part);
  t.m = w.m;
  t.npad = w.npad;
  t.per = w.per;
  t.splits = w.splits;
  const unsigned b64 = (unsigned)(w.m / 64), pairs = b64 * (b64 + 1) / 2, batch = (unsigned)o.batch;
  t.pairs = pairs;
  hipLaunchKernelGGL(long_gram_kernel, dim3((unsigned)((t.pairs * w.splits * batch + 7) / 8 * 8)), dim3(kNT), 0, s, t);
  hipLaunchKernelGGL(long_join_kernel, dim3(4, pairs, batch), dim3(256), 0, s, t, A);
  const unsigned b32 = (unsigned)(w.m / 32), tiles = b32 * (b32 + 1) / 2;
  Square p{};
  p.a = o.a;
  p.b = o.b;
  p.c = o.c;
  p.m = w.m;
  p.scale = o.sq;
  const auto go = [&](unsigned n) {
    hipLaunchKernelGGL(long_square_kernel, dim3(tiles, n, batch), dim3(kNT), 0, s, p);
  };
  for (int k = 0; k < o.steps; ++k) {
    const bool first = k == 0, last = k + 1 == o.steps;
    double* now = first ? Q : P;  // the first step's P is Q
    p.poly = 1;
    p.x[0] = p.y[0] = A;
    p.out[0] = now;
    p.pair = first && last ? q : nullptr;
    go(1);
    p.poly = 0;
    if (last) {
      if (first) break;
      p.x[0] = Q;
      p.y[0] = now;
      p.pair = q;
      go(1);
      break;
    }
    p.x[0] = A;
    p.y[0] = now;
    p.out[0] = W;
    p.x[1] = Q;
    p.y[1] = now;
    p.out[1] = Q1;
    go(first ? 1 : 2);
    if (!first) {
      double* z = Q;
      Q = Q1;
      Q1 = z;
    }
    p.x[0] = W;
    p.y[0] = now;
    p.out[0] = A;
    go(1);
  }
  return hipGetLastError();
}

}  // namespace ecc
