// Newton-Schulz orthogonalisation of matrices with a short side of at most 64
// (contract: include/ecc_train.h; longer ones: ecc_orth.hip).
//
// Every X_k is Q_k X_0 with Q_k symmetric, and X_k X_k^T = A_k follows from A_0
// alone: with P = a I + b A + c A A,
//   A <- P A P,   Q <- Q P,
// all of them polynomials of A_0, so they commute and are symmetric.  The long
// side n is therefore passed twice only, for A_0 = X_0 X_0^T and for Q X_0,
// whatever the number of steps: 3 m^2 n products in place of 15 m^2 n.
//
// Precision.  A direction of singular value s is one of s^2 in A, and an error
// d of A grows with it, by p(s)^2 a step, where the direct iteration forms A
// anew.  In float32 that costs digits (relative error 5e-5 of a 64 x 66
// matrix, direct iteration 1e-6); in float64 it does not (1.1e-6, all of it
// the final product's), so A, P and Q are float64 throughout, on the float64
// matrix instructions; launch_orth leaves the cases whose growth would pass
// 2^26 to the direct iteration.  The final product is float32.
//
// What bounds it: the two passes, HBM and latency; the steps, one workgroup per
// matrix, the float64 matrix rate of a CU (64 cycles an instruction), 1.3 us
// per 64^3 product (lower triangle of tiles), 14 of them in 5 steps, and the
// strips each phase reads from LDS before it can multiply.  24 matrices of 64 x
// 1728 in float32, momentum step: 15 us for A_0, 40 for the steps, 19 for the
// result, 73 in all (three products a step on pairs: 267; floor of the bytes:
// 11).  27 x 64 in one launch: 13.5 us (17 launches: 64).
//
// Orientation.  m is the short side.  `tall` matrices (rows > cols) keep the
// short side contiguous; lanes then take MB consecutive short-side elements,
// so element a of tile I is a MB + I there and 16 I + a otherwise.

#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "ecc_act.hpp"
#include "ecc_internal.hpp"
#include "ecc_train_internal.hpp"

namespace ecc {
namespace {

constexpr int kNT = 512;
constexpr int kNW = kNT / 64;
typedef double f64x4 __attribute__((ext_vector_type(4)));
typedef double f64x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

template <int MB>
constexpr int kTiles = MB * (MB + 1) / 2;
// Place of an element in a matrix in LDS: rows are kept in pairs, so that one
// 16-byte read gives a lane its elements of two products' rows.
template <int MB>
__device__ __forceinline__ int at(int row, int col) {
  return (row >> 1) * (32 * MB) + col * 2 + (row & 1);
}

struct Thin {
  OrthArgs o;
  int m;
  int64_t n, per;  // columns of a workgroup
  int splits;
  double* part;  // [batch][splits][tiles][256]
  float* q;      // [batch][64 * 64]: Q / (norm + eps) 2^-t
  float* pow2;   // [batch]: 2^t
};

// N elements, of which `valid` lie inside.
template <int N, class T>
__device__ __forceinline__ void load_some(const T* p, int64_t valid, float (&v)[N]) {
  if (valid >= N) {
    Vec<T, N> r;
    load_vec(p, r);
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = (float)r.v[j];
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = j < valid ? (float)p[j] : 0.0f;
  }
}
template <int N, class T>
__device__ __forceinline__ void store_some(T* p, int64_t valid, const float (&v)[N]) {
  if (valid >= N) {
    Vec<T, N> r;
#pragma unroll
    for (int j = 0; j < N; ++j) r.v[j] = (T)v[j];
    store_vec(p, r);
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (j < valid) p[j] = (T)v[j];
  }
}

// N neighbouring elements of the gradient and the buffer, as stored.  Loads
// carry no condition, so that a wave has all of a chunk in flight: what lies
// past the end of a line (`count` elements from `line` on) is read from inside
// it and zeroed by `value`.  VEC: N divides count, or all N lie inside.
template <int N, class GT>
struct Raw {
  Vec<GT, N> g;
  Vec<float, N> b;
  template <bool VEC>
  __device__ __forceinline__ void load(const GT* gp, const float* buf, int64_t line, int first, int count, bool grad) {
    if constexpr (VEC) {
      const int64_t i = line + (first < count ? first : 0);
      if (grad) load_vec(gp + i, g);
      if (buf) load_vec(buf + i, b);
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const int64_t i = line + (first + j < count ? first + j : count - 1);
        if (grad) g.v[j] = gp[i];
        if (buf) b.v[j] = buf[i];
      }
    }
  }
  // The matrix that is orthogonalised.  The buffer is the old one where
  // `update` is set, and is brought forward.
  __device__ __forceinline__ void value(const OrthArgs& o, bool buf, bool update, int first, int count, float (&u)[N]) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      float x;
      if (buf) {
        if (update) b.v[j] = fmaf(o.momentum, b.v[j], o.blend * (float)g.v[j]);
        x = o.nesterov ? fmaf(o.momentum, b.v[j], o.blend * (float)g.v[j]) : b.v[j];
      } else {
        x = (float)g.v[j];
      }
      u[j] = first + j < count ? x : 0.0f;
    }
  }
};

// ------------------------------------------------------------------- A_0
// One k-step of the lower triangle of tiles; x[I]: this lane's element of tile I.
template <int MB>
__device__ __forceinline__ void gram_step(const float (&x)[MB], f64x4 (&acc)[kTiles<MB>]) {
  double d[MB];
#pragma unroll
  for (int i = 0; i < MB; ++i) d[i] = (double)x[i];
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j <= i; ++j)
      acc[i * (i + 1) / 2 + j] = __builtin_amdgcn_mfma_f64_16x16x4f64(d[i], d[j], acc[i * (i + 1) / 2 + j], 0, 0, 0);
}

// U U^T over columns [c0, c1) of the workgroup's matrix.  out: tile order,
// tiles x 256 doubles.  lds: kNW x 5 x 256 doubles.
template <int MB, bool TALL, class GT>
__device__ __forceinline__ void gram_part(const Thin& t, int64_t batch, int64_t c0, int64_t c1, double* lds,
                                          double* out) {
  const OrthArgs& o = t.o;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, q = lane >> 4;
  const int64_t off = batch * o.rows * o.cols;
  const GT* g = reinterpret_cast<const GT*>(o.g) + off;
  float* buf = o.buffer ? o.buffer + off : nullptr;
  f64x4 acc[kTiles<MB>];
#pragma unroll
  for (int i = 0; i < kTiles<MB>; ++i) acc[i] = f64x4{0.0, 0.0, 0.0, 0.0};
  // a wave's chunk of 16 columns; the next one is on its way while this one is multiplied
  constexpr int CH = 16, R = TALL ? CH / 4 : MB, E = TALL ? MB : 4;
  const int count = (int)(c1 - c0);
  typedef Raw<E, GT> Chunk[R];
  const auto fetch = [&](int64_t c, Chunk& x) {
    const auto go = [&](auto vec) {
      constexpr bool VEC = decltype(vec)::value;
#pragma unroll
      for (int s = 0; s < R; ++s) {
        if constexpr (TALL) {
          const int64_t j = c + s * 4 + q;
          x[s].template load<VEC>(g, buf, (j < c1 ? j : c1 - 1) * o.cols, r * MB, t.m, true);
        } else {
          const int row = s * 16 + r;
          x[s].template load<VEC>(g, buf, (row < t.m ? row : 0) * o.cols + c0, (int)(c - c0) + q * 4, count, true);
        }
      }
    };
    if (TALL ? t.m % MB == 0 : c + CH <= c1)
      go(std::true_type());
    else
      go(std::false_type());
  };
  const auto use = [&](int64_t c, Chunk& x) {
    float u[R][E];
#pragma unroll
    for (int s = 0; s < R; ++s) {
      if constexpr (TALL) {
        const int64_t j = c + s * 4 + q;
        x[s].value(o, buf, true, r * MB, j < c1 ? t.m : 0, u[s]);
        if (buf && j < c1 && r * MB < t.m) store_some<E>(buf + j * o.cols + r * MB, t.m - r * MB, x[s].b.v);
      } else {
        const int row = s * 16 + r, first = (int)(c - c0) + q * 4;
        x[s].value(o, buf, true, first, row < t.m ? count : 0, u[s]);
        if (buf && row < t.m && first < count) store_some<E>(buf + row * o.cols + c0 + first, count - first, x[s].b.v);
      }
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      float y[MB];
#pragma unroll
      for (int i = 0; i < MB; ++i) y[i] = TALL ? u[s][i] : u[i][s];
      gram_step<MB>(y, acc);
    }
  };
  int64_t c = c0 + wave * CH;
  if (c < c1) {
    Chunk x, next;
    fetch(c, x);
    for (; c < c1; c += kNW * CH) {
      const bool more = c + kNW * CH < c1;
      if (more) fetch(c + kNW * CH, next);
      use(c, x);
      if (more)
#pragma unroll
        for (int s = 0; s < R; ++s) x[s] = next[s];
    }
  }
  // the waves' sums, five tiles at a time, in order
#pragma unroll
  for (int t0 = 0; t0 < kTiles<MB>; t0 += 5) {
    const int nt = kTiles<MB> - t0 < 5 ? kTiles<MB> - t0 : 5;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 5; ++i)
      if (t0 + i < kTiles<MB>)
#pragma unroll
        for (int k = 0; k < 4; ++k) lds[(wave * 5 + i) * 256 + k * 64 + lane] = acc[t0 + i < kTiles<MB> ? t0 + i : 0][k];
    __syncthreads();
    for (int e = threadIdx.x; e < nt * 256; e += kNT) {
      double s = 0.0;
#pragma unroll
      for (int w = 0; w < kNW; ++w) s += lds[w * 5 * 256 + e];
      out[t0 * 256 + e] = s;
    }
  }
}

// ------------------------------------------------------------------ steps
// Tile (i, j), j <= i, of the lower triangle, at most four tiles a side.
__device__ __forceinline__ void tile_index(int tile, int& i, int& j) {
  i = tile >= 6 ? 3 : (tile >= 3 ? 2 : (tile >= 1 ? 1 : 0));
  j = tile - i * (i + 1) / 2;
}

// Row and column, within the matrix, of element e of tile-ordered storage.
template <int MB>
__device__ __forceinline__ void place(int e, bool tall, int& row, int& col) {
  int i, j;
  tile_index(e >> 8, i, j);
  const int a = 4 * ((e >> 6) & 3) + ((e >> 4) & 3), b = e & 15;
  row = tall ? a * MB + i : i * 16 + a;
  col = tall ? b * MB + j : j * 16 + b;
}

// One operand of tile row i: elements (row, 16 i + lane & 15) of four pairs of
// rows a step; the order of the rows is that of the other operand's.
template <int MB>
struct Strip {
  f64x2 v[2 * MB];
  __device__ __forceinline__ void load(const double* x, int i) {
    const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
#pragma unroll
    for (int k = 0; k < 2 * MB; ++k) v[k] = *reinterpret_cast<const f64x2*>(x + at<MB>(8 * k + 2 * q, i * 16 + r));
  }
};
// Tile of the product of two commuting symmetric matrices.
template <int MB>
__device__ __forceinline__ f64x4 tile_product(const Strip<MB>& x, const Strip<MB>& y) {
  f64x4 a = {0.0, 0.0, 0.0, 0.0};
#pragma unroll
  for (int k = 0; k < 2 * MB; ++k) {
    a = __builtin_amdgcn_mfma_f64_16x16x4f64(x.v[k][0], y.v[k][0], a, 0, 0, 0);
    a = __builtin_amdgcn_mfma_f64_16x16x4f64(x.v[k][1], y.v[k][1], a, 0, 0, 0);
  }
  return a;
}
template <int MB>
__device__ __forceinline__ void tile_store(double* z, int i, int j, f64x4 v) {
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int row = i * 16 + 4 * k + q, col = j * 16 + r;
    z[at<MB>(row, col)] = v[k];
    if (i != j) z[at<MB>(col, row)] = v[k];
  }
}
// From G = U U^T (tile order, `splits` partial sums apart by tiles x 256) to Q
// / (norm + eps) 2^-t in float32, row-major with 16 MB columns, at `q`; returns
// 2^t.  lds: 4 matrices and one double.
template <int MB>
__device__ __forceinline__ float thin_steps(const Thin& t, bool tall, const double* part, int splits, double* lds,
                                            float* q) {
  constexpr int N = 16 * MB, T = kTiles<MB>, SZ = N * N;
  const OrthArgs& o = t.o;
  double *A = lds, *P = lds + SZ, *W = lds + 2 * SZ, *Q = lds + 3 * SZ, *tr = lds + 4 * SZ;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  // the partial sums in order, every element of a thread's at once
  constexpr int E = (T * 256 + kNT - 1) / kNT;
  double sum[E];
#pragma unroll
  for (int u = 0; u < E; ++u) sum[u] = 0.0;
  for (int k = 0; k < splits; k += 8) {
    double v[8][E];
#pragma unroll
    for (int l = 0; l < 8; ++l)
#pragma unroll
      for (int u = 0; u < E; ++u) {
        const int e = threadIdx.x + u * kNT;
        v[l][u] = k + l < splits && e < T * 256 ? part[(int64_t)(k + l) * (T * 256) + e] : 0.0;
      }
#pragma unroll
    for (int u = 0; u < E; ++u) sum[u] += ((v[0][u] + v[1][u]) + (v[2][u] + v[3][u])) + ((v[4][u] + v[5][u]) + (v[6][u] + v[7][u]));
  }
#pragma unroll
  for (int u = 0; u < E; ++u) {
    const int e = threadIdx.x + u * kNT;
    if (e < T * 256) {
      int row, col;
      place<MB>(e, tall, row, col);
      A[at<MB>(row, col)] = sum[u];
      A[at<MB>(col, row)] = sum[u];
    }
  }
  __syncthreads();
  if (wave == 0) {
    double s = lane < N ? A[at<MB>(lane, lane)] : 0.0;
    for (int d = 1; d < 64; d *= 2) s += __shfl_xor(s, d);
    if (lane == 0) *tr = s;
  }
  __syncthreads();
  const double inv = 1.0 / (sqrt(*tr) + (double)o.eps);
  for (int e = threadIdx.x; e < SZ; e += kNT) A[e] = A[e] * inv * inv;
  __syncthreads();
  for (int s = 0; s < o.steps; ++s) {
    const bool first = s == 0, last = s + 1 == o.steps;
    const int r = lane & 15, q4 = lane >> 4;
    Strip<MB> x, y, z;
    for (int tile = wave; tile < T; tile += kNW) {
      int i, j;
      tile_index(tile, i, j);
      x.load(A, i);
      y.load(A, j);
      f64x4 v = tile_product(x, y);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int row = i * 16 + 4 * k + q4, col = j * 16 + r;
        v[k] = fma((double)o.c, v[k], (double)o.b * A[at<MB>(row, col)]);
        if (row == col) v[k] += (double)o.a;
      }
      tile_store<MB>(P, i, j, v);
      if (first) tile_store<MB>(Q, i, j, v);
    }
    __syncthreads();
    // W = A P and the new Q = Q P, tile by tile side by side: they share P's strip
    constexpr int kMine = (T + kNW - 1) / kNW;
    f64x4 held[kMine];
#pragma unroll
    for (int u = 0; u < kMine; ++u) {
      const int tile = wave + u * kNW;
      if (tile < T) {
        int i, j;
        tile_index(tile, i, j);
        y.load(P, j);
        if (!last) x.load(A, i);
        if (!first) z.load(Q, i);
        if (!last) tile_store<MB>(W, i, j, tile_product(x, y));
        if (!first) held[u] = tile_product(z, y);
      }
    }
    __syncthreads();
    if (!first)
#pragma unroll
      for (int u = 0; u < kMine; ++u) {
        const int tile = wave + u * kNW;
        if (tile < T) {
          int i, j;
          tile_index(tile, i, j);
          tile_store<MB>(Q, i, j, held[u]);
        }
      }
    if (!last)
      for (int tile = wave; tile < T; tile += kNW) {
        int i, j;
        tile_index(tile, i, j);
        x.load(W, i);
        y.load(P, j);
        tile_store<MB>(A, i, j, tile_product(x, y));
      }
    __syncthreads();
  }
  int e = 0;
  frexp(inv, &e);
  e = e < -126 ? -126 : (e > 126 ? 126 : e);
  if (!(inv < 1e300)) e = 0;
  const double f = inv * ldexp(1.0, -e);
  for (int k = threadIdx.x; k < N * N; k += kNT) q[k] = (float)(Q[at<MB>(k / N, k % N)] * f);
  return ldexpf(1.0f, e);
}

// ------------------------------------------------------------------ Q X_0
// N elements of the result or the parameter, as stored; the type is uniform,
// and one branch in a load or a store costs less than three copies of every
// kernel.
template <int N>
struct Out {
  float p[N];
  __device__ __forceinline__ void load(const OrthArgs& o, int64_t i, int64_t valid) {
    if (valid <= 0) return;
    if (o.odtype == kTF32)
      load_some<N>(reinterpret_cast<const float*>(o.out) + i, valid, p);
    else if (o.odtype == kTF16)
      load_some<N>(reinterpret_cast<const f16*>(o.out) + i, valid, p);
    else
      load_some<N>(reinterpret_cast<const bf16*>(o.out) + i, valid, p);
  }
  __device__ __forceinline__ void store(const OrthArgs& o, int64_t i, int64_t valid, float (&v)[N]) {
    if (valid <= 0) return;
    if (o.buffer)
#pragma unroll
      for (int j = 0; j < N; ++j) v[j] = fmaf(p[j], o.keep, -o.rate * v[j]);
    if (o.odtype == kTF32)
      store_some<N>(reinterpret_cast<float*>(o.out) + i, valid, v);
    else if (o.odtype == kTF16)
      store_some<N>(reinterpret_cast<f16*>(o.out) + i, valid, v);
    else
      store_some<N>(reinterpret_cast<bf16*>(o.out) + i, valid, v);
  }
};

// Columns [c0, c1) of the result; a wave takes 32 (wide) or 16 (tall) at a
// time and has read all of them before it writes, so the result may replace
// the input.  The summed axis is taken in the order that lets a lane read four
// of its factors of Q, symmetric, at once.  qm: Q in LDS, N x (N + 4); its padding is zero off the diagonal,
// so that what the loads find past the short side adds nothing.
template <int MB, bool TALL, class GT>
__device__ __forceinline__ void apply_part(const Thin& t, int64_t batch, int64_t c0, int64_t c1, int wave, int waves,
                                           const float* qm, float pow2) {
  constexpr int N = 16 * MB, LD = N + 4, CW = TALL ? 16 : 32;
  const OrthArgs& o = t.o;
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int64_t off = batch * o.rows * o.cols;
  const GT* g = reinterpret_cast<const GT*>(o.g) + off;
  const float* buf = o.buffer ? o.buffer + off : nullptr;
  const bool grad = !buf || o.nesterov;
  const auto block = [&](int64_t c, auto vec) {
    constexpr bool VEC = decltype(vec)::value;
    if constexpr (TALL) {
      Raw<4, GT> x[MB];
      Out<MB> p[4];
#pragma unroll
      for (int k = 0; k < MB; ++k)
        x[k].template load<VEC>(g, buf, (c + r < c1 ? c + r : c1 - 1) * o.cols, k * 16 + q * 4, t.m, grad);
      if (buf)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int64_t j = c + q * 4 + k;
          p[k].load(o, off + j * o.cols + r * MB, j < c1 ? t.m - r * MB : 0);
        }
      float u[MB][4];
#pragma unroll
      for (int k = 0; k < MB; ++k) {
        x[k].value(o, buf, false, k * 16 + q * 4, t.m, u[k]);
#pragma unroll
        for (int j = 0; j < 4; ++j) u[k][j] *= pow2;
      }
      f32x4 acc[MB];
#pragma unroll
      for (int i = 0; i < MB; ++i) acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int k = 0; k < MB; ++k) {
        f32x4 m[MB];
#pragma unroll
        for (int i = 0; i < MB; ++i) m[i] = *reinterpret_cast<const f32x4*>(qm + (r * MB + i) * LD + k * 16 + q * 4);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < MB; ++i) acc[i] = __builtin_amdgcn_mfma_f32_16x16x4f32(u[k][j], m[i][j], acc[i], 0, 0, 0);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int64_t j = c + q * 4 + k;
        float v[MB];
#pragma unroll
        for (int i = 0; i < MB; ++i) v[i] = acc[i][k];
        p[k].store(o, off + j * o.cols + r * MB, j < c1 ? t.m - r * MB : 0, v);
      }
    } else {
      Raw<2, GT> x[4 * MB];
      Out<2> p[MB][4];
      const int first = (int)(c - c0) + r * 2, count = (int)(c1 - c0);
#pragma unroll
      for (int k = 0; k < 4 * MB; ++k) {
        const int row = (k >> 2) * 16 + q * 4 + (k & 3);
        x[k].template load<VEC>(g, buf, (row < t.m ? row : 0) * o.cols + c0, first, count, grad);
      }
      if (buf)
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int row = i * 16 + q * 4 + k;
            p[i][k].load(o, off + row * o.cols + c0 + first, row < t.m ? count - first : 0);
          }
      float u[4 * MB][2];
#pragma unroll
      for (int k = 0; k < 4 * MB; ++k) {
        x[k].value(o, buf, false, first, count, u[k]);
#pragma unroll
        for (int j = 0; j < 2; ++j) u[k][j] *= pow2;
      }
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        f32x4 acc[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        f32x4 m[MB];
#pragma unroll
        for (int k = 0; k < MB; ++k) m[k] = *reinterpret_cast<const f32x4*>(qm + (i * 16 + r) * LD + k * 16 + q * 4);
#pragma unroll
        for (int k = 0; k < 4 * MB; ++k)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            acc[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(m[k >> 2][k & 3], u[k][j], acc[j], 0, 0, 0);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int row = i * 16 + q * 4 + k;
          float v[2] = {acc[0][k], acc[1][k]};
          p[i][k].store(o, off + row * o.cols + c0 + first, row < t.m ? count - first : 0, v);
        }
      }
    }
  };
  for (int64_t c = c0 + wave * CW; c < c1; c += waves * CW) {
    if (TALL ? t.m % 4 == 0 : c + CW <= c1)
      block(c, std::true_type());
    else
      block(c, std::false_type());
  }
}

// ---------------------------------------------------------------- kernels
constexpr int kGramLds = kNW * 5 * 256;  // doubles
template <int MB>
constexpr int kStepsLds = 4 * 256 * MB * MB + 2;
template <int MB>
constexpr int kWholeLds =
    kStepsLds<MB> > kGramLds + kTiles<MB> * 256 ? kStepsLds<MB> : kGramLds + kTiles<MB> * 256;

template <int MB, bool TALL, class GT>
__global__ __launch_bounds__(kNT) void thin_gram_kernel(Thin t) {
  __shared__ double lds[kGramLds];
  const int64_t c0 = (int64_t)blockIdx.x * t.per, c1 = c0 + t.per < t.n ? c0 + t.per : t.n;
  gram_part<MB, TALL, GT>(t, blockIdx.y, c0, c1, lds,
                          t.part + ((int64_t)blockIdx.y * t.splits + blockIdx.x) * (kTiles<MB> * 256));
}

template <int MB>
__global__ __launch_bounds__(kNT) void thin_steps_kernel(Thin t) {
  __shared__ __align__(16) double dyn[kStepsLds<MB>];
  const float p = thin_steps<MB>(t, t.o.rows > t.o.cols, t.part + (int64_t)blockIdx.x * t.splits * (kTiles<MB> * 256),
                                 t.splits, dyn, t.q + (int64_t)blockIdx.x * (64 * 64));
  if (threadIdx.x == 0) t.pow2[blockIdx.x] = p;
}

template <int MB, bool TALL, class GT>
__global__ __launch_bounds__(256) void thin_apply_kernel(Thin t) {
  constexpr int N = 16 * MB, COLS = TALL ? 64 : 128;
  __shared__ __align__(16) float qm[N * (N + 4)];
  const float* q = t.q + (int64_t)blockIdx.y * (64 * 64);
#pragma unroll
  for (int u = 0; u < (N * N + 1023) / 1024; ++u) {
    const int k = (u * 256 + threadIdx.x) * 4;
    if (N * N >= 1024 || k < N * N)
      *reinterpret_cast<f32x4*>(qm + (k / N) * (N + 4) + k % N) = *reinterpret_cast<const f32x4*>(q + k);
  }
  const float pow2 = t.pow2[blockIdx.y];
  __syncthreads();
  const int64_t c0 = (int64_t)blockIdx.x * COLS, c1 = c0 + COLS < t.n ? c0 + COLS : t.n;
  apply_part<MB, TALL, GT>(t, blockIdx.y, c0, c1, threadIdx.x >> 6, 4, qm, pow2);
}

// All of it, where one workgroup takes a whole matrix.
template <int MB, bool TALL, class GT>
__global__ __launch_bounds__(kNT) void thin_whole_kernel(Thin t) {
  constexpr int N = 16 * MB, SZ = N * N;
  __shared__ __align__(16) double dyn[kWholeLds<MB>];
  // the tile-ordered sums lie behind the waves' sums, where A is not
  double* g = dyn + kGramLds;
  gram_part<MB, TALL, GT>(t, blockIdx.x, 0, t.n, dyn, g);
  __syncthreads();
  float* q = reinterpret_cast<float*>(dyn);  // over A and P, free at the end
  const float pow2 = thin_steps<MB>(t, TALL, g, 1, dyn, q);
  __syncthreads();
  float* qm = reinterpret_cast<float*>(dyn + SZ * 2);
  for (int k = threadIdx.x; k < N * N; k += kNT) qm[(k / N) * (N + 4) + k % N] = q[k];
  __syncthreads();
  apply_part<MB, TALL, GT>(t, blockIdx.x, 0, t.n, threadIdx.x >> 6, kNW, qm, pow2);
}

template <int MB, bool TALL, class GT>
hipError_t thin_run(const Thin& t, hipStream_t s) {
  const unsigned batch = (unsigned)t.o.batch;
  if (t.splits == 1) {
    hipLaunchKernelGGL((thin_whole_kernel<MB, TALL, GT>), dim3(batch), dim3(kNT), 0, s, t);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((thin_gram_kernel<MB, TALL, GT>), dim3((unsigned)t.splits, batch), dim3(kNT), 0, s, t);
  hipLaunchKernelGGL((thin_steps_kernel<MB>), dim3(batch), dim3(kNT), 0, s, t);
  constexpr int64_t cols = TALL ? 64 : 128;
  hipLaunchKernelGGL((thin_apply_kernel<MB, TALL, GT>), dim3((unsigned)((t.n + cols - 1) / cols), batch), dim3(256), 0, s,
                     t);
  return hipGetLastError();
}

template <int MB, class GT>
hipError_t thin_side(const Thin& t, hipStream_t s) {
  return t.o.rows > t.o.cols ? thin_run<MB, true, GT>(t, s) : thin_run<MB, false, GT>(t, s);
}

}  // namespace

template <class GT>
hipError_t launch_orth_thin(const OrthArgs& o, hipStream_t s) {
  const ThinPlan w = thin_plan(o.batch, o.rows, o.cols);
  char* ws = reinterpret_cast<char*>(o.ws);
  Thin t{};
  t.o = o;
  t.m = (int)(o.rows < o.cols ? o.rows : o.cols);
  t.n = o.rows < o.cols ? o.cols : o.rows;
  t.per = w.per;
  t.splits = w.splits;
  t.part = reinterpret_cast<double*>(ws + w.at_part);
  t.q = reinterpret_cast<float*>(ws + w.at_q);
  t.pow2 = reinterpret_cast<float*>(ws + w.at_pow2);
  if (t.m <= 16) return thin_side<1, GT>(t, s);
  if (t.m <= 32) return thin_side<2, GT>(t, s);
  if (t.m <= 48) return thin_side<3, GT>(t, s);
  return thin_side<4, GT>(t, s);
}

}  // namespace ecc
