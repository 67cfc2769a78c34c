// Group norm with an activation over channels-last features, its read-out to
// a scalar grid, and the backward passes of both (contract: include/ecc_train.h).
//
// For sample b, group g of D = C/G channels and N = S D elements:
//   mean = sum x / N,  var = sum (x - mean)^2 / N,  rstd = 1/sqrt(var + eps)
//   u_c = (x_c - mean) a_c + bias_c,  a_c = rstd weight_c
//   y_c = act(u_c);   field = offset + sum_c r_c y_c
// and backwards, with q_c = dL/dy_c act'(u_c) (dL/dy_c = df r_c for the grid):
//   A1_c = sum q_c,  A2_c = sum q_c (x_c - mean)          per sample
//   dbias_c = sum_b A1,  dweight_c = sum_b rstd A2
//   m1 = sum_{c in g} weight_c A1_c / N,  m2 = sum_{c in g} weight_c rstd A2_c / N
//   dx_c = a_c q_c - rstd m1 - (x_c - mean) rstd^2 m2
//
// Every pass is a stream over the features and bound by HBM (or by the memory
// side cache when the features fit it); the statistics force two passes each
// way, so forward reads x twice and backward reads x and dy twice.  2 x 128^3 x
// 64 in bfloat16, a training pass: 0.83 ms, 8 times 537 MB at 5.2 TB/s (a copy
// of 1 GB: 5.0).  The read-out of 256^3 x 32: 1.12 to 1.16 ms, 5 times 1.07 GB;
// its passes with the activation are bound by issue as well, 13 to 16
// instructions an element beside two transcendental ones.  Mapping:
// a row of C channels is taken by L lanes of one wave, K vectors of V = 16
// bytes each, so a lane keeps its V K channels for the whole pass and holds
// their scale, shift and sums in registers; a wave has floor(64 / L) rows in
// flight per step.  A row that is not a multiple of V ends in a vector that
// overlaps the one before it; the overlap is left out of every sum (and
// stored twice with the same value).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "ecc_act.hpp"
#include "ecc_train_internal.hpp"

namespace ecc {
namespace {

constexpr int kNT = 256;
constexpr int kNW = kNT / 64;

// How a pass is laid out; filled by norm_geom on the host.
struct NormGeom {
  int64_t S, C;
  int NB;      // workgroups per sample
  int L;       // lanes per row
  int nv;      // vectors per row
  int chunks;  // column chunks of 64 vectors (rows of more than kMostK x 64)
  int runs;    // of kRun turns, of the workgroup that has most (passes that sum)
};

// A lane's columns, and its rows: the waves of a launch sweep the rows as one
// window, in which every wave has U neighbouring steps of floor(64 / L) rows,
// so that what is in flight lies close together in memory (a read of 1.07 GB
// took 175 us so, and 202 us with a wave's steps a window apart).
template <int V, int K>
struct Cols {
  int c[K];      // first channel of vector k
  int dup[K];    // leading elements that belong to another vector (V: none is its own)
  int64_t wave_id, waves;
  int l, sub, rows;
  __device__ Cols(const NormGeom& g) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    sub = lane / g.L;
    rows = 64 / g.L;
    l = lane - sub * g.L;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int v = (int)blockIdx.z * 64 + l + k * g.L;
      const int at = v * V, last = (int)g.C - V;
      if (v < g.nv) {
        c[k] = at < last ? at : last;
        dup[k] = at - c[k];
      } else {
        c[k] = last;
        dup[k] = V;
      }
    }
    wave_id = (int64_t)blockIdx.x * kNW + wave;
    waves = (int64_t)g.NB * kNW;
  }
  // The first of U rows, `rows` apart, of the first turn; past the end for lanes that have none.
  template <int U>
  __device__ __forceinline__ int64_t first(int64_t S) const {
    return sub < rows ? wave_id * (U * rows) + sub : S;
  }
};

// Rows a turn: of the passes over x and, with as many vectors in flight, of
// those over x and its gradient.
template <int K>
constexpr int kUnroll = K == 1 ? 4 : (K == 2 ? 2 : 1);
template <int K, bool READ>
constexpr int kSumsUnroll = READ ? kUnroll<K> : (kUnroll<K> + 1) / 2;

// Turns whose sums stay in float32.  A thread has as many turns as the features
// need, and one number added up over all of them is off by half a step of its
// sum each time, all one way where the terms are alike (1000 turns: 2e-5).  A
// turn's rows are added to each other first, so a sum is of kRun numbers at
// most, each of up to 4; then it goes to the workgroup's float64 sums.
constexpr int kRun = 32;

// Calls body(row...) for the rows of this lane from r on, which is left behind
// the last: U at a time while r is below `end`, and one by one where the rows
// end before.  body<N> gets an array of N row indexes.
template <int U, int V, int K, class Body>
__device__ __forceinline__ void for_rows(const Cols<V, K>& col, int64_t S, int64_t& r, int64_t end, Body body) {
  const int64_t step = col.waves * (U * col.rows), full = S - (U - 1) * col.rows, last = end < full ? end : full;
  for (; r < last; r += step) {
    int64_t rows[U];
#pragma unroll
    for (int i = 0; i < U; ++i) rows[i] = r + i * col.rows;
    body(rows, std::integral_constant<int, U>());
  }
  if constexpr (U > 1) {
    if (r < end)
      for (; r < S; r += col.rows) {
        int64_t rows[1] = {r};
        body(rows, std::integral_constant<int, 1>());
      }
  }
}
// All of this lane's rows.
template <int U, int V, int K, class Body>
__device__ __forceinline__ void for_rows(const Cols<V, K>& col, int64_t S, Body body) {
  int64_t r = col.template first<U>(S);
  for_rows<U>(col, S, r, S, body);
}
// The next run of them.
template <int U, int V, int K, class Body>
__device__ __forceinline__ void for_run(const Cols<V, K>& col, int64_t S, int64_t& r, Body body) {
  for_rows<U>(col, S, r, r + kRun * (col.waves * (U * col.rows)), body);
}

// Elements of a vector whose sums are joined at a time: few, so that the
// buffer does not limit how many workgroups a CU holds during the pass.
template <int V>
constexpr int kSumElems = V < 2 ? V : 2;

// Sums over the workgroup's rows of NV values per channel, in a fixed order
// and in float64, written to out[channel * NV + i], or added to it.  lds:
// kSumElems<V> NV kNT doubles.  P threads share one output and join by shuffles, P the largest
// power of two with P L kSumElems NV <= kNT (and at most 64).
template <int V, int K, int NV, class Value>
__device__ __forceinline__ void column_sums(const NormGeom& g, const Cols<V, K>& col, double* lds, double* out,
                                            bool more, Value value) {
  constexpr int E = kSumElems<V>;
  const int rows = 64 / g.L, L = g.L;
  const int nout = L * E * NV;
  int P = 1;
  while (P < 64 && 2 * P * nout <= kNT) P *= 2;
  const int p = threadIdx.x % P;
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int j0 = 0; j0 < V; j0 += E) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < E; ++j)
#pragma unroll
        for (int i = 0; i < NV; ++i) lds[(j * NV + i) * kNT + threadIdx.x] = value(k, j0 + j, i);
      __syncthreads();
      // every thread of a wave takes the same number of turns: the shuffles see whole waves
      for (int o0 = 0; o0 < nout; o0 += kNT / P) {
        const int o = o0 + threadIdx.x / P;
        const int l = o % L, ji = o / L;
        double s = 0.0;
        if (o < nout)
          for (int e = p; e < kNW * rows; e += P) s += lds[ji * kNT + (e / rows) * 64 + (e % rows) * L + l];
        for (int d = 1; d < P; d *= 2) s += __shfl_xor(s, d);
        const int v = (int)blockIdx.z * 64 + l + k * L;
        if (o < nout && p == 0 && v < g.nv) {
          const int at = v * V, last = (int)g.C - V, c = at < last ? at : last;
          const int j = j0 + ji / NV;
          double* to = out + (int64_t)(c + j) * NV + ji % NV;
          if (j >= at - c) *to = more ? *to + s : s;
        }
      }
    }
}

// Moments per channel, about the channel's value in the sample's first row: a
// value of the group itself, so that nothing cancels where the mean is many
// deviations off (moments about zero, in float64, lost the variance of values
// an ulp apart at 10^4).  A thread sums x - k and (x - k)^2 in float32, k the
// first value it meets of a run in that channel; float64 from there on.
template <class T, int V, int K>
__global__ __launch_bounds__(kNT) void norm_stats_kernel(NormGeom g, const T* x, double* part, int64_t row) {
  __shared__ double lds[kSumElems<V> * 2 * kNT];
  Cols<V, K> col(g);
  const T* xs = x + (int64_t)blockIdx.y * g.S * g.C;
  constexpr int U = kUnroll<K>;
  int64_t r = col.template first<U>(g.S);
  for (int run = 0; run < g.runs; ++run) {
    float piv[K][V], s1[K][V], s2[K][V];
    Vec<T, V> about[K];  // read again each run: the compiler would keep them as float64
#pragma unroll
    for (int k = 0; k < K; ++k) {
      load_vec(xs + col.c[k], about[k]);
      Vec<T, V> v = {};
      if (r < g.S) load_vec(xs + r * g.C + col.c[k], v);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        piv[k][j] = (float)v.v[j];
        s1[k][j] = s2[k][j] = 0.0f;
      }
    }
    int n = 0;
    for_run<U>(col, g.S, r, [&](const int64_t* rows, auto N) {
      Vec<T, V> v[N.value][K];
#pragma unroll
      for (int i = 0; i < N.value; ++i)
#pragma unroll
        for (int k = 0; k < K; ++k) load_vec(xs + rows[i] * g.C + col.c[k], v[i][k]);
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          float t1 = 0.0f, t2 = 0.0f;
#pragma unroll
          for (int i = 0; i < N.value; ++i) {
            const float d = (float)v[i][k].v[j] - piv[k][j];
            t1 = i ? t1 + d : d;
            t2 = i ? fmaf(d, d, t2) : d * d;
          }
          s1[k][j] += t1;
          s2[k][j] += t2;
        }
      n += N.value;
    });
    column_sums<V, K, 2>(g, col, lds, part + ((int64_t)blockIdx.y * g.NB + blockIdx.x) * row, run > 0,
                         [&](int k, int j, int i) {
      const double p = (double)piv[k][j] - (double)(float)about[k].v[j], a = (double)s1[k][j], m = (double)n;
      return i == 0 ? fma(m, p, a) : (double)s2[k][j] + p * (2.0 * a + m * p);
    });
  }
}

// Sums NV values of column q of the partial rows at, at + step, ..., below n.
template <int NV>
__device__ __forceinline__ void add_rows(const double* q, int64_t prow, int at, int step, int n, double (&s)[NV]) {
  int r = at;
  for (; r + 3 * step < n; r += 4 * step) {
    double v[4][NV];
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int i = 0; i < NV; ++i) v[u][i] = q[(int64_t)(r + u * step) * prow + i];
#pragma unroll
    for (int i = 0; i < NV; ++i) s[i] += (v[0][i] + v[1][i]) + (v[2][i] + v[3][i]);
  }
  for (; r < n; r += step)
#pragma unroll
    for (int i = 0; i < NV; ++i) s[i] += q[(int64_t)r * prow + i];
}

// From a channel's sums about its own first value to sums about the group's, `by` below it, of n values more.
__device__ __forceinline__ void shift_sums(double (&s)[2], double by, double n) {
  s[1] += by * (2.0 * s[0] + n * by);
  s[0] += n * by;
}

// A group's statistics: mean, 1 / sqrt(var + eps), and what float32 leaves of
// the mean, from sums about `pivot`.
constexpr int kStat = 3;
__device__ __forceinline__ void group_stats(double s1, double s2, double n, double pivot, float eps, float* st) {
  const double off = s1 / n, mean = pivot + off;
  double var = s2 / n - off * off;
  var = var < 0.0 ? 0.0 : var;
  st[0] = (float)mean;
  st[1] = (float)(1.0 / sqrt(var + (double)eps));
  st[2] = (float)(off + (pivot - (double)st[0]));
}

// Where a sample's partial rows are few (at most 64 KB), every
// workgroup of the second pass joins them itself, which costs less than a
// launch between the passes (3 to 4 us).  x: this sample's features.  Returns its
// statistics.
constexpr int kHereChannels = 512;
struct JoinLds {
  double sum[2][kHereChannels];
  float st[kStat * kHereChannels];
};
template <class T>
__device__ __forceinline__ const float* join_here(const NormArgs& p, const T* x, const double* part, int NB, int D,
                                                  int64_t prow, JoinLds& lds) {
  const int C = (int)p.C, G = (int)p.G, W = C < kNT ? C : kNT, parts = kNT / W;
  const int at = threadIdx.x % W, pt = threadIdx.x / W;
  const double* rows = part + (int64_t)blockIdx.y * NB * prow;
  if (pt < parts)
    for (int c = at; c < C; c += W) {
      double s[2] = {0.0, 0.0};
      const double by = (double)(float)x[c] - (double)(float)x[(unsigned)c / (unsigned)D * D];
      add_rows<2>(rows + (int64_t)c * 2, prow, pt, parts, NB, s);
      shift_sums(s, by, pt == 0 ? (double)p.S : 0.0);
      lds.sum[0][pt * C + c] = s[0];  // parts C <= kHereChannels: parts is 1 where C exceeds kNT
      lds.sum[1][pt * C + c] = s[1];
    }
  __syncthreads();
  int P = 1;  // threads of a group
  while (P < 64 && 2 * P * G <= kNT) P *= 2;
  const int q = threadIdx.x % P, n = D * parts;
  for (int g0 = 0; g0 < G; g0 += kNT / P) {
    const int g = g0 + threadIdx.x / P;
    double s1 = 0.0, s2 = 0.0;
    if (g < G)
      for (int e = q; e < n; e += P) {
        const int i = (e / D) * C + g * D + e % D;
        s1 += lds.sum[0][i];
        s2 += lds.sum[1][i];
      }
    for (int d = 1; d < P; d *= 2) {
      s1 += __shfl_xor(s1, d);
      s2 += __shfl_xor(s2, d);
    }
    if (g < G && q == 0) group_stats(s1, s2, (double)p.S * (double)D, (double)(float)x[g * D], p.eps, lds.st + kStat * g);
  }
  __syncthreads();
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < kStat * G; i += kNT) p.stats[(int64_t)blockIdx.y * G * kStat + i] = lds.st[i];
  return lds.st;
}

// What the passes after the statistics keep per channel.  Features are centred
// before they are scaled, 16-bit ones too: with the mean in the offset, u = x a
// + (bias - mean a), half a step of mean a stays, which is 1e-4 where a group
// is constant at 100 and the definition gives the bias exactly.  (The subtraction
// costs 1 to 2 %: 256^3 x 32 read-out, bfloat16, 1108 us a training pass, 1087
// without.)  x - mean is exact where it is small; what float32 left of the mean,
// half a step of it at most, is in the offset.
template <class T, int V, int K>
struct Affine {
  float mean[K][V], a[K][V], b[K][V];
  __device__ void load(const NormArgs& p, const Cols<V, K>& col, int D) {
    load(p, col, D, p.stats + (int64_t)blockIdx.y * p.G * kStat);
  }
  __device__ void load(const NormArgs& p, const Cols<V, K>& col, int D, const float* st) {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int c = col.c[k] + j, gr = (unsigned)c / (unsigned)D;
        mean[k][j] = st[kStat * gr];
        a[k][j] = st[kStat * gr + 1] * load_param(p.weight, p.pdtype, c, 1.0f);
        b[k][j] = fmaf(-st[kStat * gr + 2], a[k][j], load_param(p.bias, p.pdtype, c, 0.0f));
      }
  }
  // from d = x - mean, the mean as float32 has it
  __device__ __forceinline__ float u(int k, int j, float d) const { return fmaf(d, a[k][j], b[k][j]); }
};

template <class T, int V, int K, int ACT>
__global__ __launch_bounds__(kNT) void norm_apply_kernel(NormGeom g, NormArgs p, int D, const double* part, int NB,
                                                         int64_t prow) {
  __shared__ JoinLds lds;
  Cols<V, K> col(g);
  Affine<T, V, K> af;
  const int64_t base = (int64_t)blockIdx.y * g.S * g.C;
  const T* xs = reinterpret_cast<const T*>(p.x) + base;
  if (part)
    af.load(p, col, D, join_here(p, xs, part, NB, D, prow, lds));
  else
    af.load(p, col, D);
  T* ys = reinterpret_cast<T*>(p.y) + base;
  for_rows<kUnroll<K>>(col, g.S, [&](int64_t* rows, auto U) {
    Vec<T, V> v[U.value][K];
#pragma unroll
    for (int i = 0; i < U.value; ++i) {
      rows[i] = g.S - 1 - rows[i];  // what the statistics read last is read first
#pragma unroll
      for (int k = 0; k < K; ++k) load_vec(xs + rows[i] * g.C + col.c[k], v[i][k]);
    }
#pragma unroll
    for (int i = 0; i < U.value; ++i)
#pragma unroll
      for (int k = 0; k < K; ++k) {
        Vec<T, V> o;
#pragma unroll
        for (int j = 0; j < V; ++j) o.v[j] = (T)act_value<ACT>(af.u(k, j, (float)v[i][k].v[j] - af.mean[k][j]));
        if (col.dup[k] < V) store_vec(ys + rows[i] * g.C + col.c[k], o);
      }
  });
}

// Sum over the L lanes of a row, valid in its lane 0.
__device__ __forceinline__ float row_sum(float s, int l, int L) {
  for (int d = 1; d < L; d *= 2) {
    const float o = __shfl_down(s, d);
    s += l + d < L ? o : 0.0f;
  }
  return s;
}

template <class T, int V, int K, int ACT>
__global__ __launch_bounds__(kNT) void readout_apply_kernel(NormGeom g, NormArgs p, int D, const double* part, int NB,
                                                            int64_t prow) {
  __shared__ JoinLds lds;
  Cols<V, K> col(g);
  Affine<T, V, K> af;
  const T* xs = reinterpret_cast<const T*>(p.x) + (int64_t)blockIdx.y * g.S * g.C;
  if (part)
    af.load(p, col, D, join_here(p, xs, part, NB, D, prow, lds));
  else
    af.load(p, col, D);
  float r[K][V];
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int j = 0; j < V; ++j) r[k][j] = j < col.dup[k] ? 0.0f : load_param(p.readout, p.pdtype, col.c[k] + j, 0.0f);
  const float off = load_param(p.offset, p.pdtype, 0, 0.0f);
  float* fs = p.field + (int64_t)blockIdx.y * g.S;
  // the lanes of a wave stay together for the shuffles: rows past the end are
  // computed from the first row and not stored
  constexpr int U = kUnroll<K>;
  const int64_t step = col.waves * (U * col.rows);
  for (int64_t w = col.wave_id * (U * col.rows); w < g.S; w += step) {
    Vec<T, V> v[U][K];
    int64_t row[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t at = w + i * col.rows + col.sub;
      row[i] = at < g.S && col.sub < col.rows ? g.S - 1 - at : -1;
      const int64_t from = row[i] < 0 ? 0 : row[i];
#pragma unroll
      for (int k = 0; k < K; ++k) load_vec(xs + from * g.C + col.c[k], v[i][k]);
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      float s = 0.0f;
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j) s = fmaf(act_value<ACT>(af.u(k, j, (float)v[i][k].v[j] - af.mean[k][j])), r[k][j], s);
      s = row_sum(s, col.l, g.L);
      if (col.l == 0 && row[i] >= 0) fs[row[i]] = s + off;
    }
  }
}

// Backward sums: A1, A2 (and, for the grid, A3 = sum df y) per channel, and
// the sum of df behind them.  READ: the gradient is one float32 per voxel.
template <class T, int V, int K, int ACT, bool READ>
__global__ __launch_bounds__(kNT) void norm_sums_kernel(NormGeom g, NormArgs p, int D, double* part, int64_t prow) {
  constexpr int NV = READ ? 3 : 2;
  __shared__ double lds[kSumElems<V> * NV * kNT];
  Cols<V, K> col(g);
  Affine<T, V, K> af;
  af.load(p, col, D);
  const int64_t base = (int64_t)blockIdx.y * g.S * g.C;
  const T* xs = reinterpret_cast<const T*>(p.x) + base;
  const T* gs = READ ? nullptr : reinterpret_cast<const T*>(p.gy) + base;
  const float* fs = READ ? reinterpret_cast<const float*>(p.gy) + (int64_t)blockIdx.y * g.S : nullptr;
  double* out = part + ((int64_t)blockIdx.y * g.NB + blockIdx.x) * prow;
  double total = 0.0;  // of df
  constexpr int U = kSumsUnroll<K, READ>;
  int64_t r = col.template first<U>(g.S);
  for (int run = 0; run < g.runs; ++run) {
    float s[K][V][NV];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int i = 0; i < NV; ++i) s[k][j][i] = 0.0f;
    float sdf = 0.0f;
    for_run<U>(col, g.S, r, [&](const int64_t* rows, auto N) {
      Vec<T, V> v[N.value][K], q[N.value][K];
      float df[N.value];
#pragma unroll
      for (int i = 0; i < N.value; ++i) {
        if constexpr (READ) df[i] = fs[rows[i]];
#pragma unroll
        for (int k = 0; k < K; ++k) {
          load_vec(xs + rows[i] * g.C + col.c[k], v[i][k]);
          if constexpr (!READ) load_vec(gs + rows[i] * g.C + col.c[k], q[i][k]);
        }
      }
      if constexpr (READ) {
        float t = df[0];
#pragma unroll
        for (int i = 1; i < N.value; ++i) t += df[i];
        sdf += t;
      }
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          float t[3] = {};
#pragma unroll
          for (int i = 0; i < N.value; ++i) {
            const float d = (float)v[i][k].v[j] - af.mean[k][j];
            float y;
            const float sl = act_slope<ACT>(af.u(k, j, d), y);
            float dy;
            if constexpr (READ) dy = df[i]; else dy = (float)q[i][k].v[j];
            const float du = dy * sl;
            t[0] = i ? t[0] + du : du;
            t[1] = i ? fmaf(du, d, t[1]) : du * d;
            if constexpr (READ) t[2] = i ? fmaf(dy, y, t[2]) : dy * y;
          }
#pragma unroll
          for (int i = 0; i < NV; ++i) s[k][j][i] += t[i];
        }
    });
    column_sums<V, K, NV>(g, col, lds, out, run > 0, [&](int k, int j, int i) { return (double)s[k][j][i]; });
    total += (double)sdf;
  }
  if constexpr (READ) {
    __syncthreads();
    lds[threadIdx.x] = col.l == 0 ? total : 0.0;
    __syncthreads();
    if (threadIdx.x < 64) {
      double t = 0.0;
      for (int w = 0; w < kNW; ++w) t += lds[w * 64 + threadIdx.x];
      for (int d = 1; d < 64; d *= 2) t += __shfl_xor(t, d);
      if (threadIdx.x == 0) out[g.C * NV] = t;
    }
  }
}

// dx.  Workgroup rows past the samples (blockIdx.y == B) sum the parameter
// gradients over the samples instead; without dx they are the whole launch.
template <class T, int V, int K, int ACT, bool READ>
__global__ __launch_bounds__(kNT) void norm_grad_kernel(NormGeom g, NormArgs p, int D, const double* chan,
                                                        int64_t prow, const float* coef) {
  constexpr int NV = READ ? 3 : 2;
  if (!p.gx || blockIdx.y == p.B) {
    if (blockIdx.z) return;
    for (int64_t c = (int64_t)blockIdx.x * kNT + threadIdx.x; c < g.C + (READ ? 1 : 0); c += (int64_t)g.NB * kNT) {
      double t[3] = {0.0, 0.0, 0.0};
      for (int64_t b = 0; b < p.B; ++b)
        for (int i = 0; i < (c < g.C ? NV : 1); ++i) t[i] += chan[b * prow + c * NV + i];
      if (c == g.C) {
        if (p.go) store_param(p.go, p.pdtype, 0, (float)t[0]);
        continue;
      }
      const double r = READ ? (double)load_param(p.readout, p.pdtype, c, 0.0f) : 1.0;
      if (p.gb) store_param(p.gb, p.pdtype, c, (float)(r * t[0]));
      if (p.gw) store_param(p.gw, p.pdtype, c, (float)(r * t[1]));
      if (READ && p.gr) store_param(p.gr, p.pdtype, c, (float)t[2]);
    }
    return;
  }
  Cols<V, K> col(g);
  Affine<T, V, K> af;
  af.load(p, col, D);
  float c0[K][V], c1[K][V], ar[K][V];
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = col.c[k] + j;
      const int64_t gr = (int64_t)blockIdx.y * p.G + (unsigned)c / (unsigned)D;
      c1[k][j] = coef[2 * gr + 1];
      c0[k][j] = -coef[2 * gr];
      ar[k][j] = READ ? af.a[k][j] * load_param(p.readout, p.pdtype, c, 0.0f) : af.a[k][j];
    }
  const int64_t base = (int64_t)blockIdx.y * g.S * g.C;
  const T* xs = reinterpret_cast<const T*>(p.x) + base;
  const T* gs = READ ? nullptr : reinterpret_cast<const T*>(p.gy) + base;
  const float* fs = READ ? reinterpret_cast<const float*>(p.gy) + (int64_t)blockIdx.y * g.S : nullptr;
  T* os = reinterpret_cast<T*>(p.gx) + base;
  for_rows<kSumsUnroll<K, READ>>(col, g.S, [&](int64_t* rows, auto N) {
    Vec<T, V> v[N.value][K], q[N.value][K];
    float df[N.value];
#pragma unroll
    for (int i = 0; i < N.value; ++i) {
      rows[i] = g.S - 1 - rows[i];  // what the sums read last is read first
      if constexpr (READ) df[i] = fs[rows[i]];
#pragma unroll
      for (int k = 0; k < K; ++k) {
        load_vec(xs + rows[i] * g.C + col.c[k], v[i][k]);
        if constexpr (!READ) load_vec(gs + rows[i] * g.C + col.c[k], q[i][k]);
      }
    }
#pragma unroll
    for (int i = 0; i < N.value; ++i)
#pragma unroll
      for (int k = 0; k < K; ++k) {
        Vec<T, V> o;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float d = (float)v[i][k].v[j] - af.mean[k][j];
          float y;
          const float sl = act_slope<ACT>(af.u(k, j, d), y);
          float dy;
          if constexpr (READ) dy = df[i]; else dy = (float)q[i][k].v[j];
          o.v[j] = (T)fmaf(ar[k][j], dy * sl, fmaf(-d, c1[k][j], c0[k][j]));
        }
        if (col.dup[k] < V) store_vec(os + rows[i] * g.C + col.c[k], o);
      }
  });
}

constexpr int kJT = 1024;  // threads of a join

__device__ __forceinline__ double block_sum(double v, double* lds) {
  for (int d = 1; d < 64; d *= 2) v += __shfl_xor(v, d);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  double t = 0.0;
  for (int w = 0; w < kJT / 64; ++w) t += lds[w];
  return t;
}

// Partial rows to fewer: row blockIdx.y of `out` is the sum of `per` rows of
// `in`, 256 columns per workgroup (norm_fold on the host says when).
__global__ __launch_bounds__(kJT) void norm_fold_kernel(const double* in, double* out, int NB, int per, int64_t cols,
                                                        int64_t prow) {
  __shared__ double lds[kJT];
  const int tx = threadIdx.x & 255, ty = threadIdx.x >> 8;
  const int64_t b = blockIdx.z, c = (int64_t)blockIdx.x * 256 + tx;
  const int r0 = (int)blockIdx.y * per, r1 = r0 + per < NB ? r0 + per : NB;
  double s[1] = {0.0};
  if (c < cols) add_rows<1>(in + b * NB * prow + c, prow, r0 + ty, 4, r1, s);
  lds[threadIdx.x] = s[0];
  __syncthreads();
  if (ty == 0 && c < cols)
    out[(b * gridDim.y + blockIdx.y) * prow + c] = (lds[tx] + lds[tx + 256]) + (lds[tx + 512] + lds[tx + 768]);
}

// Joins the partial rows of one sample and group: statistics (forward).
template <class T>
__global__ __launch_bounds__(kJT) void norm_join_kernel(NormArgs p, const double* part, int NB, int D, int64_t prow) {
  __shared__ double lds[kJT / 64];
  const int64_t b = blockIdx.y, gr = blockIdx.x;
  const int W = D < kJT ? D : kJT, parts = kJT / W;
  const int at = threadIdx.x % W, pt = threadIdx.x / W;
  const T* x = reinterpret_cast<const T*>(p.x) + b * p.S * p.C + gr * D;
  const double pivot = (double)(float)x[0];
  double s[2] = {0.0, 0.0};
  if (pt < parts)
    for (int64_t c = at; c < D; c += W) {
      double t[2] = {0.0, 0.0};
      const double by = (double)(float)x[c] - pivot;
      add_rows<2>(part + b * NB * prow + (gr * D + c) * 2, prow, pt, parts, NB, t);
      shift_sums(t, by, pt == 0 ? (double)p.S : 0.0);
      s[0] += t[0];
      s[1] += t[1];
    }
  const double s1 = block_sum(s[0], lds), s2 = block_sum(s[1], lds);
  if (threadIdx.x == 0) group_stats(s1, s2, (double)p.S * (double)D, pivot, p.eps, p.stats + (b * p.G + gr) * kStat);
}

// s - by, where `by` is a correction: an infinite gradient makes it infinite or
// NaN, and s already what it is.
__device__ __forceinline__ double less(double s, double by) { return isfinite(by) ? s - by : s; }

// Joins the partial rows of one sample and group: channel sums with A2 scaled
// by rstd, and the group's coefficients rstd m1 and rstd^2 m2 (backward).  The
// passes before and after take x less the mean as float32 has it; the rest of
// the mean is taken off A2, and off rstd m1 with the factor that x has there.
template <bool READ>
__global__ __launch_bounds__(kJT) void norm_join_bwd_kernel(NormArgs p, const double* part, int NB, int D,
                                                            int64_t prow, double* chan, float* coef) {
  constexpr int NV = READ ? 3 : 2;
  __shared__ double lds[NV * kJT];
  const int64_t b = blockIdx.y, gr = blockIdx.x;
  const int W = D < kJT ? D : kJT, parts = kJT / W;
  const int at = threadIdx.x % W, pt = threadIdx.x / W;
  const float* st = p.stats + (b * p.G + gr) * kStat;
  const double rstd = (double)st[1], rest = (double)st[2];
  double m1 = 0.0, m2 = 0.0;
  for (int64_t c0 = 0; c0 < D; c0 += W) {
    const int64_t c = gr * D + c0 + at;
    double s[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) s[i] = 0.0;
    if (pt < parts && c0 + at < D) add_rows<NV>(part + b * NB * prow + c * NV, prow, pt, parts, NB, s);
    // halve the rows of W threads until one is left; `parts` need not be a power of two
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) lds[i * kJT + threadIdx.x] = s[i];
    for (int n = parts; n > 1;) {
      const int h = (n + 1) / 2;
      __syncthreads();
      if (pt + h < n)
#pragma unroll
        for (int i = 0; i < NV; ++i) lds[i * kJT + threadIdx.x] += lds[i * kJT + threadIdx.x + h * W];
      n = h;
    }
    __syncthreads();
    if (threadIdx.x < W && c0 + at < D) {
#pragma unroll
      for (int i = 0; i < NV; ++i) s[i] = lds[i * kJT + at];
      s[1] = less(s[1], rest * s[0]) * rstd;
#pragma unroll
      for (int i = 0; i < NV; ++i) chan[b * prow + c * NV + i] = s[i];
      double w = (double)load_param(p.weight, p.pdtype, c, 1.0f);
      if (READ) w *= (double)load_param(p.readout, p.pdtype, c, 0.0f);
      m1 += w * s[0];
      m2 += w * s[1];
    }
  }
  m1 = block_sum(m1, lds);
  m2 = block_sum(m2, lds);
  if (threadIdx.x == 0) {
    const double n = (double)p.S * (double)D, c1 = rstd * rstd * (m2 / n);
    coef[2 * (b * p.G + gr)] = (float)less(rstd * (m1 / n), rest * c1);
    coef[2 * (b * p.G + gr) + 1] = (float)c1;
  }
  if (READ && gr == 0) {
    double t = 0.0;
    for (int blk = threadIdx.x; blk < NB; blk += kJT) t += part[(b * NB + blk) * prow + p.C * NV];
    t = block_sum(t, lds);
    if (threadIdx.x == 0) chan[b * prow + p.C * NV] = t;
  }
}

// Vectors a lane takes at most.  With four of 8 elements each, what a lane keeps
// per channel fills the registers and leaves one or two waves a SIMD: forward
// and training passes of 64 million bfloat16 values took 187 and 476 us with
// 384 channels, 85 and 236 with two vectors, whose lanes are used to 75 % for 94;
// with 1280 channels 208 and 553, in chunks of columns 104 and 282.  Four of 4
// leave three waves, and the read-out needs a row in one wave.
template <class T>
constexpr int kMostK = sizeof(T) == 2 ? 2 : 4;

// Lanes and vectors per row: the fewest vectors per lane that keep within 5 %
// of the best use of the lanes (rows of nv vectors on floor(64 / L) L lanes).
template <class T>
NormGeom norm_geom(const NormArgs& a, int& V, int& K) {
  constexpr int VF = 16 / sizeof(T);
  V = a.C >= VF ? VF : 1;
  NormGeom g{};
  g.S = a.S;
  g.C = a.C;
  g.NB = (int)norm_blocks(a.B, a.S, a.C, kNormSums);
  g.nv = (int)((a.C + V - 1) / V);
  g.chunks = 1;
  K = 1;
  g.L = 64;
  if (g.nv > kMostK<T> * 64) {
    g.chunks = (g.nv + 63) / 64;
    return g;
  }
  double best = 0.0;
  for (int k = 1; k <= (V == 1 ? 1 : kMostK<T>); k *= 2) {
    const int L = (g.nv + k - 1) / k;
    if (L > 64) continue;
    const double use = (double)(g.nv * (64 / L)) / (64.0 * k);
    if (use > 1.05 * best) {
      best = use;
      K = k;
      g.L = L;
    }
  }
  return g;
}

// Runs of the workgroup with most turns, the first, for turns of U rows a lane.
int norm_runs(const NormGeom& g, int U) {
  const int64_t span = (int64_t)g.NB * kNW * U * (64 / g.L), turns = (g.S + span - 1) / span;
  return (int)((turns + kRun - 1) / kRun);
}

template <class F>
hipError_t with_act(int act, F f) {
  switch (act) {
    case kActRelu: return f(std::integral_constant<int, kActRelu>());
    case kActSilu: return f(std::integral_constant<int, kActSilu>());
    case kActGelu: return f(std::integral_constant<int, kActGelu>());
    default: return f(std::integral_constant<int, kActNone>());
  }
}

// f(V, K) with the pair as compile-time constants
template <class T, class F>
hipError_t with_cols(int V, int K, F f) {
  constexpr int VF = 16 / sizeof(T);
  using std::integral_constant;
  if (V == 1) return f(integral_constant<int, 1>(), integral_constant<int, 1>());
  if (K == 1) return f(integral_constant<int, VF>(), integral_constant<int, 1>());
  if constexpr (kMostK<T> == 4)
    if (K == 4) return f(integral_constant<int, VF>(), integral_constant<int, 4>());
  return f(integral_constant<int, VF>(), integral_constant<int, 2>());
}

}  // namespace

// Partial rows of `cols` doubles, folded first where one workgroup per sample
// and group would read more than 128 KB of them; `part` and `NB` become those
// that the join reads.
inline void norm_fold(const NormArgs& a, double*& part, int& NB, int64_t cols, int64_t prow, int64_t NV,
                      hipStream_t stream) {
  if (!norm_folded(NB) || (int64_t)NB * (a.C / a.G) * NV * (int64_t)sizeof(double) <= 128 * 1024) return;
  const int per = (NB + kNormFolded - 1) / kNormFolded, rows = (NB + per - 1) / per;
  double* out = part + a.B * (NB + 1) * prow;
  hipLaunchKernelGGL(norm_fold_kernel, dim3((unsigned)((cols + 255) / 256), (unsigned)rows, (unsigned)a.B), dim3(kJT), 0,
                     stream, part, out, NB, per, cols, prow);
  part = out;
  NB = rows;
}

template <class T>
hipError_t norm_launch_fwd(const NormArgs& a, hipStream_t stream) {
  int V, K;
  NormGeom g = norm_geom<T>(a, V, K);
  const int D = (int)(a.C / a.G);
  const int64_t prow = (int64_t)norm_row(a.C);
  double* part = reinterpret_cast<double*>(a.ws);
  const dim3 grid((unsigned)g.NB, (unsigned)a.B, (unsigned)g.chunks), block(kNT);
  return with_cols<T>(V, K, [&](auto v, auto k) {
    constexpr int VV = v.value, KK = k.value;
    g.runs = norm_runs(g, kUnroll<KK>);
    hipLaunchKernelGGL((norm_stats_kernel<T, VV, KK>), grid, block, 0, stream, g, reinterpret_cast<const T*>(a.x), part,
                       prow);
    // 64 KB of partial rows a workgroup, read from L2, at most
    const bool here = a.C <= kHereChannels && (int64_t)g.NB * a.C * 2 * (int64_t)sizeof(double) <= 64 * 1024;
    if (!here) {
      double* from = part;
      int NB = g.NB;
      norm_fold(a, from, NB, 2 * a.C, prow, 2, stream);
      hipLaunchKernelGGL(norm_join_kernel<T>, dim3((unsigned)a.G, (unsigned)a.B), dim3(kJT), 0, stream, a, from, NB, D, prow);
    }
    const double* joined = here ? part : nullptr;
    NormGeom ga = g;
    ga.NB = (int)norm_blocks(a.B, a.S, a.C, kNormApply);
    const dim3 apply((unsigned)ga.NB, (unsigned)a.B, (unsigned)g.chunks);
    return with_act(a.act, [&](auto act) {
      if (a.field)
        hipLaunchKernelGGL((readout_apply_kernel<T, VV, KK, act.value>), apply, block, 0, stream, ga, a, D, joined, g.NB, prow);
      else
        hipLaunchKernelGGL((norm_apply_kernel<T, VV, KK, act.value>), apply, block, 0, stream, ga, a, D, joined, g.NB, prow);
      return hipGetLastError();
    });
  });
}

template <class T>
hipError_t norm_launch_bwd(const NormArgs& a, hipStream_t stream) {
  int V, K;
  NormGeom g = norm_geom<T>(a, V, K);
  const int D = (int)(a.C / a.G);
  const int64_t prow = (int64_t)norm_row(a.C);
  double* part = reinterpret_cast<double*>(a.ws);
  double* chan = part + (int64_t)a.B * g.NB * prow;
  float* coef = reinterpret_cast<float*>(chan + (1 + norm_folded(g.NB)) * a.B * prow);
  const dim3 grid((unsigned)g.NB, (unsigned)a.B, (unsigned)g.chunks), block(kNT), join((unsigned)a.G, (unsigned)a.B);
  const dim3 last((unsigned)g.NB, a.gx ? (unsigned)a.B + 1 : 1u, a.gx ? (unsigned)g.chunks : 1u);
  return with_cols<T>(V, K, [&](auto v, auto k) {
    constexpr int VV = v.value, KK = k.value;
    g.runs = a.readout ? norm_runs(g, kSumsUnroll<KK, true>) : norm_runs(g, kSumsUnroll<KK, false>);
    return with_act(a.act, [&](auto act) {
      constexpr int A = act.value;
      double* from = part;
      int NB = g.NB;
      if (a.readout) {
        hipLaunchKernelGGL((norm_sums_kernel<T, VV, KK, A, true>), grid, block, 0, stream, g, a, D, part, prow);
        norm_fold(a, from, NB, 3 * a.C + 1, prow, 3, stream);
        hipLaunchKernelGGL((norm_join_bwd_kernel<true>), join, dim3(kJT), 0, stream, a, from, NB, D, prow, chan, coef);
        hipLaunchKernelGGL((norm_grad_kernel<T, VV, KK, A, true>), last, block, 0, stream, g, a, D, chan, prow, coef);
      } else {
        hipLaunchKernelGGL((norm_sums_kernel<T, VV, KK, A, false>), grid, block, 0, stream, g, a, D, part, prow);
        norm_fold(a, from, NB, 2 * a.C, prow, 2, stream);
        hipLaunchKernelGGL((norm_join_bwd_kernel<false>), join, dim3(kJT), 0, stream, a, from, NB, D, prow, chan, coef);
        hipLaunchKernelGGL((norm_grad_kernel<T, VV, KK, A, false>), last, block, 0, stream, g, a, D, chan, prow, coef);
      }
      return hipGetLastError();
    });
  });
}

}  // namespace ecc
