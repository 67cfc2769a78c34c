// The norms before and after a block, fused with its gate and the residual
// scale (contract: include/ecc_train.h).
//
// With r(v) = 1 / sqrt(mean v^2 + eps) over a row of channels,
//   n = branch r(branch) branch_weight   (or the branch itself),
//   y = scale x + gate n,   z = y r(y) weight.
// Backwards, with hat(v) = v r(v),
//   dy += r(y) (dz weight - hat(y) mean(dz weight hat(y))),   dx = scale dy,
//   dn = dy gate,   dgate = sum dy n,   dweight = sum dz hat(y),
//   dbranch = r(branch) (dn branch_weight - hat(branch) mean(dn branch_weight hat(branch))),
//   dbranch_weight = sum dn hat(branch).
//
// A row stays in the registers of the lanes that share it, from its one load to
// its one store: the forward pass moves four streams, the backward pass six,
// which is the least there is.  y is formed again from x in the backward pass:
// x and y would cost the same to read, and y is rounded.  Squares are summed in
// float64, so that no sum over finite values overflows or underflows; it costs a
// few cycles of 64 lanes against some 50 of memory.  (r itself is float32: beyond
// an rms of 2^126 it has fewer bits, below 2^-128 with eps = 0 it is infinite.)
// The remaining sums along a row are float32 over 16 elements a lane and then a
// tree.  Sums over rows: 16 rows of a thread in float32, then those, up to 16 of
// them, then the workgroup's rows by halves, then all workgroups in float64, always
// in the same order.
//
// Both passes are bound by memory (a copy of 1.07 GB: 5.1 TB/s).  16384 rows of
// 1024 bfloat16 beside a float32 stream: forward 46 us, 4.4 TB/s; backward 74 us,
// 4.1 TB/s, and 6 for the join of the sums.  1.8e6 rows of 64 bfloat16: 222 us
// and 305 us, 4.1 and 4.5 TB/s.  One row of 1024: 5.5 us, a launch.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "ecc_act.hpp"
#include "ecc_block_internal.hpp"
#include "ecc_train_internal.hpp"

namespace ecc {
namespace {

constexpr int kRun = 16;  // rows of a thread that are summed before their sum joins the others

struct ResGeom {
  int L, slots;  // lanes of a row, rows of a workgroup at a time
  int64_t samples, rows;  // rows of a sample
  int64_t blocks;         // workgroups of a sample
};

// Where this lane's vectors begin, and how many of the first elements belong to
// the vector before: the last one of a row is moved back to end with the row.
template <int V, int K>
struct Columns {
  int64_t at[K];
  int skip[K];  // V: the lane has no such vector
  __device__ __forceinline__ Columns(int lane, int L, int64_t C) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int64_t c = ((int64_t)k * L + lane) * V;
      at[k] = c + V <= C ? c : (C > V ? C - V : 0);
      skip[k] = c < C ? (int)(c - at[k]) : V;
    }
  }
};

// (Asked anew each time: kept, the answers for every element take more scalar
// registers than there are.)
template <int V, int K>
__device__ __forceinline__ int skip_of(const Columns<V, K>& col, int k) {
  int skip = col.skip[k];
  asm("" : "+v"(skip));
  return skip;
}

// Elements of a row as they lie, and as numbers, or of the parameters; those
// that another vector has are 0.
template <int V, int K, class T>
__device__ __forceinline__ void load_raw(const T* p, const Columns<V, K>& col, bool active, Vec<T, V> (&r)[K]) {
#pragma unroll
  for (int k = 0; k < K; ++k) {
    r[k] = Vec<T, V>{};
    if (active && col.skip[k] < V) load_vec(p + col.at[k], r[k]);
  }
}
template <int V, int K, class T>
__device__ __forceinline__ void unpack(const Vec<T, V> (&v)[K], const Columns<V, K>& col, float (&r)[K][V]) {
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int skip = skip_of(col, k);
#pragma unroll
    for (int j = 0; j < V; ++j) r[k][j] = V > 1 && j < skip ? 0.0f : (float)v[k].v[j];
  }
}
template <int V, int K, class T>
__device__ __forceinline__ void store_row(T* p, const Columns<V, K>& col, const float (&r)[K][V]) {
#pragma unroll
  for (int k = 0; k < K; ++k) {
    Vec<T, V> v;
#pragma unroll
    for (int j = 0; j < V; ++j) v.v[j] = (T)r[k][j];
    const int skip = skip_of(col, k);
    if (skip == 0) {
      store_vec(p + col.at[k], v);
    } else if (skip < V) {
#pragma unroll
      for (int j = 1; j < V; ++j)
        if (j >= skip) p[col.at[k] + j] = v.v[j];
    }
  }
}
template <int V, int K>
__device__ __forceinline__ void load_params(const void* p, int pdtype, int64_t off, const Columns<V, K>& col,
                                            float (&r)[K][V]) {
  const auto take = [&](auto type) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      Vec<decltype(type), V> v = {};
      if (col.skip[k] < V) load_vec(reinterpret_cast<const decltype(type)*>(p) + off + col.at[k], v);
#pragma unroll
      for (int j = 0; j < V; ++j) r[k][j] = V > 1 && j < col.skip[k] ? 0.0f : (float)v.v[j];
    }
  };
  if (!p) {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int j = 0; j < V; ++j) r[k][j] = j < col.skip[k] ? 0.0f : 1.0f;
  } else if (pdtype == kTF32) {
    take(float{});
  } else if (pdtype == kTF16) {
    take(f16{});
  } else {
    take(bf16{});
  }
}

// Sum over the lanes of a row.  Every thread of the workgroup calls it where a
// row has more than a wave.
template <class T>
__device__ __forceinline__ T row_sum(T v, int L, T* lds) {
  const int within = L < 64 ? L : 64;
  for (int d = 1; d < within; d *= 2) v += __shfl_xor(v, d);
  if (L > 64) {
    const int waves = L / 64, wave = threadIdx.x >> 6, first = wave / waves * waves;
    __syncthreads();  // the sums before are read
    if ((threadIdx.x & 63) == 0) lds[wave] = v;
    __syncthreads();
    v = lds[first];
    for (int w = 1; w < waves; ++w) v += lds[first + w];
  }
  return v;
}

// Squares of float32 numbers and their sums fit float64 with room to spare.
template <int V, int K>
__device__ __forceinline__ float inverse_rms(const float (&r)[K][V], int L, int64_t C, float eps, double* lds) {
  double s = 0.0;
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int j = 0; j < V; ++j) s = fma((double)r[k][j], (double)r[k][j], s);
  s = row_sum(s, L, lds);
  return (float)(1.0 / sqrt(s / (double)C + (double)eps));
}

template <class XT, class BT, int V, int K>
__global__ __launch_bounds__(512) void residual_fwd_kernel(ResArgs a, ResGeom g) {
  __shared__ double lds[8];
  const int lane = threadIdx.x & (g.L - 1), slot = threadIdx.x / g.L;
  const int64_t sample = blockIdx.x / g.blocks, block = blockIdx.x - sample * g.blocks, C = a.channels;
  const Columns<V, K> col(lane, g.L, C);
  float gate[K][V], weight[K][V], after[K][V];
  load_params(a.gate, a.pdtype, sample * a.gate_stride, col, gate);
  load_params(a.weight, a.pdtype, 0, col, weight);
  load_params(a.branch_weight, a.pdtype, 0, col, after);
  const int64_t turn = g.blocks * g.slots;
  Vec<XT, V> nx[K];
  Vec<BT, V> nb[K];
  const auto load = [&](int64_t first) {  // the rows of a turn
    const bool active = first + slot < g.rows;
    const int64_t at = (sample * g.rows + first + slot) * C;
    load_raw(reinterpret_cast<const XT*>(a.x) + at, col, active, nx);
    load_raw(reinterpret_cast<const BT*>(a.branch) + at, col, active && a.branch, nb);
  };
  load(block * g.slots);
  for (int64_t first = block * g.slots; first < g.rows; first += turn) {
    const bool active = first + slot < g.rows;
    const int64_t row = sample * g.rows + first + slot;
    float x[K][V], b[K][V];
    unpack(nx, col, x);
    unpack(nb, col, b);
    load(first + turn);  // on their way while these are finished
    float rb = 1.0f;
    if (a.branch) {
      if (a.norm_branch) rb = inverse_rms(b, g.L, C, a.eps, lds);
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j) x[k][j] = fmaf(a.scale, x[k][j], gate[k][j] * (b[k][j] * rb * after[k][j]));
      if (active) store_row(reinterpret_cast<XT*>(a.y) + row * C, col, x);
    }
    const float ry = inverse_rms(x, g.L, C, a.eps, lds);
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int j = 0; j < V; ++j) x[k][j] = x[k][j] * ry * weight[k][j];
    if (active) {
      store_row(reinterpret_cast<BT*>(a.z) + row * C, col, x);
      if (a.stats && lane == 0) {
        a.stats[row * 2] = rb;
        a.stats[row * 2 + 1] = ry;
      }
    }
  }
}

template <class XT, class BT, int V, int K>
__global__ __launch_bounds__(512) void residual_bwd_kernel(ResArgs a, ResGeom g, float* part) {
  extern __shared__ float shared[];  // sums of runs, then of half the slots
  __shared__ float lds[8];
  const int lane = threadIdx.x & (g.L - 1), slot = threadIdx.x / g.L;
  const int64_t sample = blockIdx.x / g.blocks, block = blockIdx.x - sample * g.blocks, C = a.channels;
  const Columns<V, K> col(lane, g.L, C);
  float gate[K][V], weight[K][V], after[K][V];
  load_params(a.gate, a.pdtype, sample * a.gate_stride, col, gate);
  load_params(a.weight, a.pdtype, 0, col, weight);
  load_params(a.branch_weight, a.pdtype, 0, col, after);
  // sums over a run of rows, of the gate, the weight and the branch's weight; the
  // sums of runs are in LDS: in registers they did not fit (16384 x 1024, float32
  // stream: 105 us)
  float run[3][K][V] = {};
  const auto total = [&](int q, int k, int j) -> float& {
    return shared[((q * K + k) * V + j) * blockDim.x + threadIdx.x];
  };
  const float inv = 1.0f / (float)C;
  int turns = 0;
  bool runs = false;
  const int64_t turn = g.blocks * g.slots;
  Vec<XT, V> nx[K], ny[K];
  Vec<BT, V> nb[K], nz[K];
  float nrb, nry;
  // Of 16 elements a lane, as rows beyond 4096 have, the next turn's do not fit the
  // registers beside this one's (64 to 113 of a lane's went to memory and back:
  // 4096 rows of 8192 float32 373 us, 248 so); 16-bit ones do but for grad_z (200
  // us so, 213 with none ahead, 188 with 3 of a lane's in memory).
  constexpr bool kFits = V * K < 16, kAhead = kFits || sizeof(XT) == 2;
  const auto load = [&](int64_t first) {  // the rows of a turn
    const bool active = first + slot < g.rows;
    const int64_t row = sample * g.rows + first + slot, at = row * C;
    load_raw(reinterpret_cast<const XT*>(a.x) + at, col, active, nx);
    load_raw(reinterpret_cast<const BT*>(a.branch) + at, col, active && a.branch, nb);
    load_raw(reinterpret_cast<const XT*>(a.gy) + at, col, active && a.gy, ny);
    if (kFits || !kAhead) load_raw(reinterpret_cast<const BT*>(a.gz) + at, col, active && a.gz, nz);
    nrb = active ? a.stats[row * 2] : 0.0f;
    nry = active ? a.stats[row * 2 + 1] : 0.0f;
  };
  if (kAhead) load(block * g.slots);
  for (int64_t first = block * g.slots; first < g.rows; first += turn) {
    const bool active = first + slot < g.rows;
    const int64_t row = sample * g.rows + first + slot;
    float x[K][V], b[K][V], dy[K][V], dz[K][V];
    if (!kAhead) load(first);
    if (!kFits && kAhead) load_raw(reinterpret_cast<const BT*>(a.gz) + row * C, col, active && a.gz, nz);
    unpack(nx, col, x);
    unpack(nb, col, b);
    unpack(ny, col, dy);
    unpack(nz, col, dz);
    const float rb = nrb, ry = nry;
    if (kAhead) load(first + turn);  // on their way while these are finished
    // b: the branch's hat, or the branch itself; x: y's hat; dz: its gradient
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (a.branch) {
          b[k][j] *= rb;
          x[k][j] = fmaf(a.scale, x[k][j], gate[k][j] * (b[k][j] * after[k][j]));
        }
        x[k][j] *= ry;
        if (active && a.gz) run[1][k][j] = fmaf(dz[k][j], x[k][j], run[1][k][j]);
        dz[k][j] *= weight[k][j];
        s = fmaf(dz[k][j], x[k][j], s);
      }
    if (a.gz) s = row_sum(s, g.L, lds) * inv;  // without it nothing of z, infinite or not, reaches a gradient
    float t = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (a.gz) dy[k][j] = fmaf(ry, fmaf(-x[k][j], s, dz[k][j]), dy[k][j]);
        x[k][j] = a.branch ? a.scale * dy[k][j] : dy[k][j];
        if (active) run[0][k][j] = fmaf(dy[k][j], b[k][j] * after[k][j], run[0][k][j]);
        dy[k][j] *= gate[k][j];
        if (active) run[2][k][j] = fmaf(dy[k][j], b[k][j], run[2][k][j]);
        dy[k][j] *= after[k][j];
        t = fmaf(dy[k][j], b[k][j], t);
      }
    if (a.gx && active) store_row(reinterpret_cast<XT*>(a.gx) + row * C, col, x);
    if (a.norm_branch) {
      t = row_sum(t, g.L, lds) * inv;
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j) dy[k][j] = rb * fmaf(-b[k][j], t, dy[k][j]);
    }
    if (a.gbranch && active) store_row(reinterpret_cast<BT*>(a.gbranch) + row * C, col, dy);
    if (++turns == kRun) {
      turns = 0;
#pragma unroll
      for (int q = 0; q < 3; ++q)
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
          for (int j = 0; j < V; ++j) {
            total(q, k, j) = (runs ? total(q, k, j) : 0.0f) + run[q][k][j];
            run[q][k][j] = 0.0f;
          }
      runs = true;
    }
  }
  if (!part) return;
  part += (int64_t)blockIdx.x * 3 * C;
  if (runs) {
#pragma unroll
    for (int q = 0; q < 3; ++q)
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j) run[q][k][j] += total(q, k, j);
  }
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    // the slots' rows, by halves
    for (int d = g.slots / 2; d > 0; d /= 2) {
      __syncthreads();
      if (slot >= d && slot < 2 * d) {
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
          for (int j = 0; j < V; ++j) shared[(k * V + j) * (d * g.L) + (slot - d) * g.L + lane] = run[q][k][j];
      }
      __syncthreads();
      if (slot < d) {
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
          for (int j = 0; j < V; ++j) run[q][k][j] += shared[(k * V + j) * (d * g.L) + slot * g.L + lane];
      }
    }
    if (slot == 0) store_row(part + q * C, col, run[q]);
  }
}

// Joins the partial rows of a quantity: blockIdx.z 0 the gate (for every sample,
// blockIdx.y), 1 and 2 the weights.  64 rows at a time, 16 columns.
constexpr int kJoin = 1024;
__global__ __launch_bounds__(kJoin) void residual_join_kernel(ResArgs a, ResGeom g, const float* part) {
  __shared__ double lds[kJoin / 16][17];
  const int q = blockIdx.z, c = threadIdx.x & 15, r = threadIdx.x >> 4;
  void* out = q == 0 ? a.ggate : q == 1 ? a.gweight : a.gbranch_weight;
  const bool each = q == 0 && a.gate_stride;
  const int64_t C = a.channels, col = (int64_t)blockIdx.x * 16 + c;
  if (!out) return;
  for (int64_t sample = blockIdx.y; sample < (each ? g.samples : 1); sample += gridDim.y) {
    const int64_t from = each ? sample * g.blocks : 0, rows = each ? g.blocks : g.samples * g.blocks;
    double s = 0.0;
    if (col < C) {
#pragma unroll 4
      for (int64_t i = r; i < rows; i += kJoin / 16) s += (double)part[((from + i) * 3 + q) * C + col];
    }
    lds[r][c] = s;
    __syncthreads();
    for (int d = kJoin / 32; d > 0; d /= 2) {
      if (r < d) lds[r][c] += lds[r + d][c];
      __syncthreads();
    }
    if (r == 0 && col < C) store_param(out, a.pdtype, sample * a.gate_stride * (q == 0) + col, (float)lds[0][c]);
    __syncthreads();
  }
}

template <class F>
hipError_t with_types(int xdtype, int dtype, F f) {
  if (dtype == 0) return f(float{}, float{});
  if (dtype == 1) return xdtype == 0 ? f(float{}, f16{}) : f(f16{}, f16{});
  return xdtype == 0 ? f(float{}, bf16{}) : f(bf16{}, bf16{});
}

// f(V, K) of a row's shape.
template <bool HALF, class F>
hipError_t with_shape(const RowShape& s, F f) {
  using std::integral_constant;
  if (s.V == 1) return f(integral_constant<int, 1>{}, integral_constant<int, 1>{});
  if constexpr (HALF) {
    if (s.K == 1) return f(integral_constant<int, 8>{}, integral_constant<int, 1>{});
    return f(integral_constant<int, 8>{}, integral_constant<int, 2>{});
  } else {
    if (s.K == 1) return f(integral_constant<int, 4>{}, integral_constant<int, 1>{});
    if (s.K == 2) return f(integral_constant<int, 4>{}, integral_constant<int, 2>{});
    if (s.K == 3) return f(integral_constant<int, 4>{}, integral_constant<int, 3>{});
    return f(integral_constant<int, 4>{}, integral_constant<int, 4>{});
  }
}

ResGeom geometry(const ResArgs& a, const RowShape& s, int64_t total) {
  ResGeom g{};
  g.L = s.L;
  g.slots = s.threads / s.L;
  g.samples = a.gate_stride ? a.batch : 1;
  g.rows = a.gate_stride ? a.inner : a.batch * a.inner;
  g.blocks = res_blocks(g.samples, g.rows, g.slots, total);
  return g;
}

}  // namespace

hipError_t launch_residual_fwd(const ResArgs& a, hipStream_t stream) {
  return with_types(a.xdtype, a.dtype, [&](auto xt, auto bt) {
    using XT = decltype(xt);
    using BT = decltype(bt);
    constexpr bool half = sizeof(XT) == 2;
    const RowShape s = res_shape(a.channels, half, false);
    const ResGeom g = geometry(a, s, kResApply);
    return with_shape<half>(s, [&](auto v, auto k) {
      hipLaunchKernelGGL((residual_fwd_kernel<XT, BT, v.value, k.value>), dim3((unsigned)(g.samples * g.blocks)),
                         dim3(s.threads), 0, stream, a, g);
      return hipGetLastError();
    });
  });
}

hipError_t launch_residual_bwd(const ResArgs& a, hipStream_t stream) {
  return with_types(a.xdtype, a.dtype, [&](auto xt, auto bt) {
    using XT = decltype(xt);
    using BT = decltype(bt);
    constexpr bool half = sizeof(XT) == 2;
    const RowShape s = res_shape(a.channels, half, true);
    const ResGeom g = geometry(a, s, kResSums);
    const bool sums = a.ggate || a.gweight || a.gbranch_weight;
    float* part = sums ? reinterpret_cast<float*>(a.ws) : nullptr;
    return with_shape<half>(s, [&](auto v, auto k) {
      // of runs, where there are any, or of half the slots
      const bool runs = g.rows > g.blocks * g.slots * (kRun - 1);
      const size_t lds = (size_t)(runs ? 3 * s.threads : s.threads / 2) * v.value * k.value * sizeof(float);
      hipLaunchKernelGGL((residual_bwd_kernel<XT, BT, v.value, k.value>), dim3((unsigned)(g.samples * g.blocks)),
                         dim3(s.threads), lds, stream, a, g, part);
      if (sums) {
        const int64_t each = a.gate_stride && a.ggate ? a.batch : 1;
        hipLaunchKernelGGL(residual_join_kernel,
                           dim3((unsigned)((a.channels + 15) / 16), (unsigned)(each < 1024 ? each : 1024), 3), dim3(kJoin), 0,
                           stream, a, g, part);
      }
      return hipGetLastError();
    });
  });
}

}  // namespace ecc
