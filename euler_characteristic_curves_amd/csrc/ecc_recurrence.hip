// The gated linear recurrence along the steps of a sequence (contract:
// include/ecc_train.h).
//
// With k = 1 / (1 + exp(-gate)),
//   h_t = k_t h_(t-1) + (1 - k_t) x_t.
// Backwards, with E_t = dL / dh_(t-1) through step t alone,
//   D_t = dh_t + E_(t+1),   E_t = k_t D_t,   dx_t = (1 - k_t) D_t,
//   dgate_t = D_t (h_(t-1) - x_t) k_t (1 - k_t).
// Steps from a sequence's length on keep the state (k = 1) and have no input.
//
// What is kept of a gate is m, the smaller of k and 1 - k with the gate's sign:
// a step is then h + m (x - h), or x + |m| (h - x), exact where a state lasts
// for thousands of steps as well as where it is replaced.  A run of steps maps h
// to A h + B; its A is kept twice, as the product of the k and as c = 1 - A, and
// whichever of the two is small is used, for the same reason.  (Products of
// rounded k are off by half a step of float32 times the number of steps that a
// state lasts: 3e-5 for gates of 7, alike.)
//
// A thread has R steps of V channels in registers, a workgroup G threads along
// the steps: each finds its run's (A, c, B), the runs are joined in LDS, and
// then every thread goes through its steps from its own first state.  The
// backward pass does so in both directions at once: its forward states start
// from those that the forward pass kept before every tile.  A sequence is one
// workgroup's work if there are enough of them, three streams forward and five
// backward; if not, a pass of its own finds the (A, c, B) of its parts, and
// reads two streams once more.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "ecc_act.hpp"
#include "ecc_block_internal.hpp"
#include "ecc_train_internal.hpp"

namespace ecc {
namespace {

constexpr int kThreads = 256;

// The smaller of k and 1 - k, with the gate's sign.  The exponent's rounding
// leaves |gate| 2^-24 relative.
__device__ __forceinline__ float small_gate(float f) {
  const float e = __builtin_amdgcn_exp2f(-1.44269502f * fabsf(f));
  return copysignf(e * __builtin_amdgcn_rcpf(1.0f + e), f);
}
__device__ __forceinline__ bool keeps(float m) { return (__float_as_uint(m) >> 31) == 0; }

// k h + (1 - k) x
__device__ __forceinline__ float step(float h, float x, float m) {
  const bool up = keeps(m);
  const float base = up ? h : x, other = up ? x : h;
  return fmaf(fabsf(m), other - base, base);
}
// k d
__device__ __forceinline__ float kept(float d, float m) { return keeps(m) ? fmaf(-m, d, d) : -m * d; }

// What a run of steps does to a state: h -> A h + B, c = 1 - A.
struct Run {
  float A, c, B;
};
__device__ __forceinline__ float keep(const Run& r, float h) { return r.c < 0.5f ? fmaf(-r.c, h, h) : r.A * h; }
__device__ __forceinline__ float apply(const Run& r, float h) { return r.B + keep(r, h); }
__device__ __forceinline__ Run then(const Run& first, const Run& r) {
  return Run{first.A * r.A, r.c + keep(r, first.c), apply(r, first.B)};
}

struct Place {
  int64_t b, seg, c;  // sample, part, first channel of this thread
  int g;
  bool active;
};
template <int V>
__device__ __forceinline__ Place place(const RecArgs& a, const RecShape& s) {
  Place p;
  const int lane = threadIdx.x & (s.L - 1);
  const int64_t block = blockIdx.x % s.blocks, rest = blockIdx.x / s.blocks;
  p.seg = rest % s.segments;
  p.b = rest / s.segments;
  p.g = threadIdx.x / s.L;
  const int64_t c = (block * s.L + lane) * V;
  p.active = c < a.channels;
  // the last lane's channels end with the row; what two lanes have, both write alike
  p.c = c + V <= a.channels ? c : a.channels - V;
  return p;
}
__device__ __forceinline__ int64_t length_of(const RecArgs& a, int64_t b) {
  if (!a.lengths) return a.steps;
  const int64_t n = a.lengths[b];
  return n < 0 ? 0 : (n < a.steps ? n : a.steps);
}

// R steps from t on; what lies at or behind `end` is not read.
template <class T, int V, int R>
__device__ __forceinline__ void load_steps(const T* p, const Place& at, int64_t t, int64_t end, int64_t C,
                                           Vec<T, V> (&r)[R]) {
#pragma unroll
  for (int i = 0; i < R; ++i) {
    r[i] = Vec<T, V>{};
    if (at.active && t + i < end) load_vec(p + (t + i) * C, r[i]);
  }
}
template <class T, int V, int R>
__device__ __forceinline__ void gates_of(const Vec<T, V> (&f)[R], int64_t t, int64_t end, float (&m)[R][V]) {
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int v = 0; v < V; ++v) m[i][v] = t + i < end ? small_gate((float)f[i].v[v]) : 0.0f;
}

// Runs of the groups in LDS, [number][group][lane].
template <int V>
struct Shared {
  float* at;
  int L, G, lane;
  __device__ __forceinline__ float& ref(int number, int g, int v) { return at[((number * G + g) * V + v) * L + lane]; }
  __device__ __forceinline__ void put(int g, int v, const Run& r) {
    ref(0, g, v) = r.A;
    ref(1, g, v) = r.c;
    ref(2, g, v) = r.B;
  }
  __device__ __forceinline__ Run get(int g, int v) { return Run{ref(0, g, v), ref(1, g, v), ref(2, g, v)}; }
};

// State before this workgroup's part from `start`: the parts before it, in the
// order in which they apply (BACK: from the last one on), shared out over the groups.
template <int V, bool BACK>
__device__ __forceinline__ void join_parts(const RecArgs& a, const RecShape& s, const Place& at, Shared<V> sh,
                                           float (&state)[V]) {
  const int64_t n = BACK ? s.segments - 1 - at.seg : at.seg;
  if (n == 0) return;
  const int64_t each = (n + s.G - 1) / s.G, from = at.g * each, to = from + each < n ? from + each : n;
  const float* parts = reinterpret_cast<const float*>(a.ws) + at.b * s.segments * 3 * a.channels + at.c;
  Run mine[V];
#pragma unroll
  for (int v = 0; v < V; ++v) mine[v] = Run{1.0f, 0.0f, 0.0f};
  if (at.active) {
#pragma unroll 4
    for (int64_t i = from; i < to; ++i) {
      const float* p = parts + (BACK ? s.segments - 1 - i : i) * 3 * a.channels;
#pragma unroll
      for (int v = 0; v < V; ++v) mine[v] = then(mine[v], Run{p[v], p[a.channels + v], p[2 * a.channels + v]});
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) sh.put(at.g, v, mine[v]);
  __syncthreads();
  for (int g = 0; g < s.G; ++g)
#pragma unroll
    for (int v = 0; v < V; ++v) state[v] = apply(sh.get(g, v), state[v]);
  __syncthreads();
}

// (A, c, B) of every part: of the states, or (BACK) of the gradients.
template <class T, int V, int R, bool BACK>
__global__ __launch_bounds__(kThreads) void recurrence_parts_kernel(RecArgs a, RecShape s) {
  __shared__ float lds[3 * kThreads * V];
  const Place at = place<V>(a, s);
  Shared<V> sh{lds, s.L, s.G, (int)(threadIdx.x & (s.L - 1))};
  const int64_t len = length_of(a, at.b), C = a.channels, off = at.b * a.steps * C + at.c;
  const T* second = reinterpret_cast<const T*>(BACK ? a.gh : a.x);
  Run all[V];
#pragma unroll
  for (int v = 0; v < V; ++v) all[v] = Run{1.0f, 0.0f, 0.0f};
  const int64_t first = at.seg * s.per, last = first + s.per < s.tiles ? first + s.per : s.tiles;
  for (int64_t i = 0; i < last - first; ++i) {
    const int64_t tile = BACK ? last - 1 - i : first + i, t = (tile * s.G + at.g) * R;
    Vec<T, V> f[R], x[R];
    float m[R][V];
    load_steps<T, V, R>(reinterpret_cast<const T*>(a.gate) + off, at, t, len, C, f);
    load_steps<T, V, R>(second + off, at, t, second ? len : 0, C, x);
    gates_of<T, V, R>(f, t, len, m);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      Run r{1.0f, 0.0f, 0.0f};
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const int q = BACK ? R - 1 - j : j;
        r.A = step(r.A, 0.0f, m[q][v]);
        r.c = step(r.c, 1.0f, m[q][v]);
        r.B = BACK ? kept(r.B + (float)x[q].v[v], m[q][v]) : step(r.B, (float)x[q].v[v], m[q][v]);
      }
      sh.put(at.g, v, r);
    }
    __syncthreads();
    for (int j = 0; j < s.G; ++j)
#pragma unroll
      for (int v = 0; v < V; ++v) all[v] = then(all[v], sh.get(BACK ? s.G - 1 - j : j, v));
    __syncthreads();
  }
  if (at.g == 0 && at.active) {
    float* p = reinterpret_cast<float*>(a.ws) + (at.b * s.segments + at.seg) * 3 * C + at.c;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      p[v] = all[v].A;
      p[C + v] = all[v].c;
      p[2 * C + v] = all[v].B;
    }
  }
}

template <class T, int V, int R>
__global__ __launch_bounds__(kThreads) void recurrence_fwd_kernel(RecArgs a, RecShape s) {
  __shared__ float lds[3 * kThreads * V];
  const Place at = place<V>(a, s);
  Shared<V> sh{lds, s.L, s.G, (int)(threadIdx.x & (s.L - 1))};
  const int64_t len = length_of(a, at.b), C = a.channels, off = at.b * a.steps * C + at.c;
  float state[V];
#pragma unroll
  for (int v = 0; v < V; ++v) state[v] = a.state && at.active ? a.state[at.b * C + at.c + v] : 0.0f;
  join_parts<V, false>(a, s, at, sh, state);
  const int64_t first = at.seg * s.per, last = first + s.per < s.tiles ? first + s.per : s.tiles;
  for (int64_t tile = first; tile < last; ++tile) {
    const int64_t t = (tile * s.G + at.g) * R;
    Vec<T, V> f[R], x[R];
    float m[R][V], h[V];
    load_steps<T, V, R>(reinterpret_cast<const T*>(a.gate) + off, at, t, len, C, f);
    load_steps<T, V, R>(reinterpret_cast<const T*>(a.x) + off, at, t, len, C, x);
    if (a.saved && at.g == 0 && at.active) {
#pragma unroll
      for (int v = 0; v < V; ++v) a.saved[(at.b * s.tiles + tile) * C + at.c + v] = state[v];
    }
    gates_of<T, V, R>(f, t, len, m);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      Run r{1.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < R; ++i) {
        r.A = step(r.A, 0.0f, m[i][v]);
        r.c = step(r.c, 1.0f, m[i][v]);
        r.B = step(r.B, (float)x[i].v[v], m[i][v]);
      }
      sh.put(at.g, v, r);
    }
    __syncthreads();
    for (int g = 0; g < s.G; ++g)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (g == at.g) h[v] = state[v];
        state[v] = apply(sh.get(g, v), state[v]);
      }
    __syncthreads();
    T* out = reinterpret_cast<T*>(a.h) + off;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      Vec<T, V> y;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        h[v] = step(h[v], (float)x[i].v[v], m[i][v]);
        y.v[v] = (T)(t + i < len ? h[v] : 0.0f);
      }
      if (at.active && t + i < a.steps) store_vec(out + (t + i) * C, y);
    }
  }
  if (at.seg == s.segments - 1 && at.g == 0 && at.active) {
#pragma unroll
    for (int v = 0; v < V; ++v) a.last[at.b * C + at.c + v] = state[v];
  }
}

template <class T, int V, int R>
__global__ __launch_bounds__(kThreads) void recurrence_bwd_kernel(RecArgs a, RecShape s) {
  __shared__ float lds[4 * kThreads * V];  // (A, c, B) of the states, B of the gradients
  const Place at = place<V>(a, s);
  Shared<V> sh{lds, s.L, s.G, (int)(threadIdx.x & (s.L - 1))};
  const int64_t len = length_of(a, at.b), C = a.channels, off = at.b * a.steps * C + at.c;
  float grad[V];  // of the state after the tile, through later steps
#pragma unroll
  for (int v = 0; v < V; ++v) grad[v] = a.glast && at.active ? a.glast[at.b * C + at.c + v] : 0.0f;
  join_parts<V, true>(a, s, at, sh, grad);
  const int64_t first = at.seg * s.per, last = first + s.per < s.tiles ? first + s.per : s.tiles;
  for (int64_t tile = last - 1; tile >= first; --tile) {
    const int64_t t = (tile * s.G + at.g) * R;
    Vec<T, V> f[R], x[R], d[R];
    float m[R][V], diff[R][V], h[V], e[V];
    load_steps<T, V, R>(reinterpret_cast<const T*>(a.gate) + off, at, t, len, C, f);
    load_steps<T, V, R>(reinterpret_cast<const T*>(a.x) + off, at, t, len, C, x);
    load_steps<T, V, R>(reinterpret_cast<const T*>(a.gh) + off, at, t, a.gh ? len : 0, C, d);
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = at.active ? a.saved[(at.b * s.tiles + tile) * C + at.c + v] : 0.0f;
    gates_of<T, V, R>(f, t, len, m);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      Run r{1.0f, 0.0f, 0.0f};
      float back = 0.0f;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        r.A = step(r.A, 0.0f, m[i][v]);
        r.c = step(r.c, 1.0f, m[i][v]);
        r.B = step(r.B, (float)x[i].v[v], m[i][v]);
        back = kept(back + (float)d[R - 1 - i].v[v], m[R - 1 - i][v]);
      }
      sh.put(at.g, v, r);
      sh.ref(3, at.g, v) = back;
    }
    __syncthreads();
    for (int g = 0; g < at.g; ++g)
#pragma unroll
      for (int v = 0; v < V; ++v) h[v] = apply(sh.get(g, v), h[v]);
    for (int g = s.G - 1; g >= 0; --g)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (g == at.g) e[v] = grad[v];
        Run r = sh.get(g, v);
        r.B = sh.ref(3, g, v);
        grad[v] = apply(r, grad[v]);
      }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float xv = (float)x[i].v[v];
        diff[i][v] = h[v] - xv;
        h[v] = step(h[v], xv, m[i][v]);
      }
    T* gx = reinterpret_cast<T*>(a.gx) + off;
    T* gf = reinterpret_cast<T*>(a.ggate) + off;
#pragma unroll
    for (int i = R - 1; i >= 0; --i) {
      Vec<T, V> ox, of;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float D = (float)d[i].v[v] + e[v], small = fabsf(m[i][v]);
        const float minor = small * D, major = fmaf(-small, D, D);
        const bool up = keeps(m[i][v]), in = t + i < len;
        e[v] = up ? major : minor;
        ox.v[v] = (T)(in ? (up ? minor : major) : 0.0f);
        of.v[v] = (T)(in ? diff[i][v] * (minor - small * minor) : 0.0f);
      }
      if (at.active && t + i < a.steps) {
        if (a.gx) store_vec(gx + (t + i) * C, ox);
        if (a.ggate) store_vec(gf + (t + i) * C, of);
      }
    }
  }
  if (a.gstate && at.seg == 0 && at.g == 0 && at.active) {
#pragma unroll
    for (int v = 0; v < V; ++v) a.gstate[at.b * C + at.c + v] = grad[v];
  }
}

template <class T, class F>
hipError_t with_shape(const RecShape& s, F f) {
  using std::integral_constant;
  constexpr int R = sizeof(T) == 2 ? 16 : 8;
  const auto steps = [&](auto v) {
    if (s.R == 1) return f(v, integral_constant<int, 1>{});
    return f(v, integral_constant<int, R>{});
  };
  if (s.V == 1) return steps(integral_constant<int, 1>{});
  return steps(integral_constant<int, 2>{});
}

}  // namespace

template <class T>
hipError_t launch_recurrence_fwd(const RecArgs& a, hipStream_t stream) {
  const RecShape s = rec_shape(a.batch, a.steps, a.channels, sizeof(T) == 2);
  return with_shape<T>(s, [&](auto v, auto r) {
    const dim3 grid((unsigned)(a.batch * s.segments * s.blocks)), block(kThreads);
    if (s.segments > 1) hipLaunchKernelGGL((recurrence_parts_kernel<T, v.value, r.value, false>), grid, block, 0, stream, a, s);
    hipLaunchKernelGGL((recurrence_fwd_kernel<T, v.value, r.value>), grid, block, 0, stream, a, s);
    return hipGetLastError();
  });
}

template <class T>
hipError_t launch_recurrence_bwd(const RecArgs& a, hipStream_t stream) {
  const RecShape s = rec_shape(a.batch, a.steps, a.channels, sizeof(T) == 2);
  return with_shape<T>(s, [&](auto v, auto r) {
    const dim3 grid((unsigned)(a.batch * s.segments * s.blocks)), block(kThreads);
    if (s.segments > 1) hipLaunchKernelGGL((recurrence_parts_kernel<T, v.value, r.value, true>), grid, block, 0, stream, a, s);
    hipLaunchKernelGGL((recurrence_bwd_kernel<T, v.value, r.value>), grid, block, 0, stream, a, s);
    return hipGetLastError();
  });
}

template hipError_t launch_recurrence_fwd<float>(const RecArgs&, hipStream_t);
template hipError_t launch_recurrence_fwd<f16>(const RecArgs&, hipStream_t);
template hipError_t launch_recurrence_fwd<bf16>(const RecArgs&, hipStream_t);
template hipError_t launch_recurrence_bwd<float>(const RecArgs&, hipStream_t);
template hipError_t launch_recurrence_bwd<f16>(const RecArgs&, hipStream_t);
template hipError_t launch_recurrence_bwd<bf16>(const RecArgs&, hipStream_t);

}  // namespace ecc
