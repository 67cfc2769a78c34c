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
// a step is then h + m (x - h), or x - |m| (x - h), exact where a state lasts
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
// backward; if not, a pass of its own finds the (A, c, B) of its parts, which
// reads two streams once more, and a small one the states between them.
//
// Bound by memory and, in a tile, by the wait for the joined runs.  64 x 256 x
// 1024 bfloat16: forward 27 us, 3.7 TB/s, backward 44 us, 3.8 TB/s.  12 x 8192 x
// 201 float16: parts 26 us each way, forward 30, backward 62 (rows of 402 bytes
// begin inside a line).  1 x 65536 x 96 float32: parts 14 us, states between
// them 6, forward 18.  One step of 64 x 1024: 4.4 us, a launch.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "ecc_act.hpp"
#include "ecc_block_internal.hpp"
#include "ecc_train_internal.hpp"

namespace ecc {
namespace {

constexpr int kThreads = 256;

// The smaller of k and 1 - k, with the gate's sign, and k.  The exponent's
// rounding leaves |gate| 2^-24 relative.
__device__ __forceinline__ float small_gate(float f, float& k) {
  const float e = __builtin_amdgcn_exp2f(-1.44269502f * fabsf(f));
  const float r = __builtin_amdgcn_rcpf(1.0f + e), m = e * r;
  k = __float_as_int(f) < 0 ? m : r;
  return copysignf(m, f);
}
__device__ __forceinline__ bool keeps(float m) { return (__float_as_uint(m) >> 31) == 0; }

// k h + (1 - k) x: h + m (x - h), or x - |m| (x - h)
__device__ __forceinline__ float step(float h, float x, float m) { return fmaf(m, x - h, keeps(m) ? h : x); }
// k d, and (1 - k) d
__device__ __forceinline__ float kept(float d, float m) { return fmaf(-m, d, keeps(m) ? d : 0.0f); }
__device__ __forceinline__ float taken(float d, float m) { return fmaf(m, d, keeps(m) ? 0.0f : d); }

// What follows finds anew what it needs of v.  (Kept from one pass over the steps
// to the next, whether each keeps more than half, whether it is there and where it
// lies take more registers than there are, 196 scalar ones in the backward pass.)
template <class N>
__device__ __forceinline__ void anew(N& v) {
  asm("" : "+v"(v));
}
template <int R, int V>
__device__ __forceinline__ void anew(float (&m)[R][V]) {
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int v = 0; v < V; ++v) anew(m[i][v]);
}

// What a run of steps does to a state: h -> A h + B, c = 1 - A.
struct Run {
  float A, c, B;
};
// One step more, whose x is taken separately.  c is the sum of what the steps
// take away where all of them keep more than half; where one does not, A is
// below a half and exact enough for both.
__device__ __forceinline__ void lengthen(Run& r, float m, float k) {
  r.A *= k;
  r.c = fmaf(fabsf(m), 1.0f - r.c, r.c);
}
__device__ __forceinline__ void settle(Run& r) { r.c = r.A < 0.5f ? 1.0f - r.A : r.c; }
// (Where nothing is taken, an infinity too stays what it is.)
__device__ __forceinline__ float keep(const Run& r, float h) {
  return r.c < 0.5f ? fmaf(-r.c, r.c == 0.0f ? 0.0f : h, h) : r.A * h;
}
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
  const uint32_t blocks = (uint32_t)s.blocks, segments = (uint32_t)s.segments;
  const uint32_t rest = blockIdx.x / blocks, b = rest / segments;
  // (divisions leave the scalar registers, where loads want their bases)
  p.seg = __builtin_amdgcn_readfirstlane(rest - b * segments);
  p.b = __builtin_amdgcn_readfirstlane(b);
  p.g = threadIdx.x / s.L;
  const int64_t c = ((int64_t)(blockIdx.x - rest * blocks) * s.L + lane) * V;
  p.active = c < a.channels;
  // the last lane's channels end with the row; what two lanes have, both write alike
  p.c = c + V <= a.channels ? c : a.channels - V;
  return p;
}
__device__ __forceinline__ int64_t length_of(const RecArgs& a, int64_t b) {
  if (!a.lengths) return a.steps;
  int64_t n = a.lengths[b];
  n = n < 0 ? 0 : (n < a.steps ? n : a.steps);
  return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)n) |
                   (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)((uint64_t)n >> 32)) << 32);
}

// R steps of a tile.  `whole`: all of the workgroup's lie before the end; what
// lies at or behind it is not read otherwise.  p: the tile's first step, the same
// for all lanes, so that a stream has one scalar base; offset and pitch are in
// bytes and fit 32 bits.
template <class T, int V, int R>
__device__ __forceinline__ void load_steps(const T* p, uint32_t offset, int left, bool whole, uint32_t pitch,
                                           Vec<T, V> (&r)[R]) {
  const char* base = reinterpret_cast<const char*>(p);
  anew(offset);
  if (whole) {
#pragma unroll
    for (int i = 0; i < R; ++i) load_vec(reinterpret_cast<const T*>(base + (offset + i * pitch)), r[i]);
  } else {
    anew(left);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      r[i] = Vec<T, V>{};
      if (i < left) load_vec(reinterpret_cast<const T*>(base + (offset + i * pitch)), r[i]);
    }
  }
}
template <class T, int V, int R>
__device__ __forceinline__ void store_steps(T* p, uint32_t offset, int left, bool whole, uint32_t pitch,
                                            const Vec<T, V> (&r)[R]) {
  char* base = reinterpret_cast<char*>(p);
  anew(offset);
#pragma unroll
  for (int i = 0; i < R; ++i)
    if (whole || i < left) store_vec(reinterpret_cast<T*>(base + (offset + i * pitch)), r[i]);
}

// Tiles that begin before a sequence's end.
template <int R>
__device__ __forceinline__ int64_t live_tiles(const RecShape& s, int64_t len, int64_t first, int64_t last) {
  const int64_t live = (len + s.G * R - 1) / (s.G * R);
  return live < first ? first : (live < last ? live : last);
}

// A tile's place: how many of this thread's steps lie before the sequence's end
// and before the row's, and whether all of the workgroup's do.
template <int R>
struct Tile {
  int left, rows;
  bool whole, full;
  __device__ __forceinline__ Tile(const RecArgs& a, const RecShape& s, int64_t tile, int g, int64_t len) {
    const int64_t t = (tile * s.G + g) * R, end = (tile + 1) * s.G * R;
    const auto of_mine = [&](int64_t n) { return (int)(n < 0 ? 0 : n < R ? n : R); };
    left = of_mine(len - t);
    rows = of_mine(a.steps - t);
    whole = end <= len;
    full = end <= a.steps;
  }
};

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

// The state before every part, from the parts' (A, c, B) and the first state
// (BACK: the gradient after every part, from the last one on).  64 groups of
// threads share the parts of a sequence, 16 channels a workgroup.
constexpr int kJoin = 1024, kJoinGroups = kJoin / 16;
template <bool BACK>
__global__ __launch_bounds__(kJoin) void recurrence_starts_kernel(RecArgs a, RecShape s) {
  __shared__ float lds[3][kJoinGroups][16];
  const int lane = threadIdx.x & 15, group = threadIdx.x >> 4;
  const int64_t across = (a.channels + 15) / 16, b = blockIdx.x / across, c = (blockIdx.x - b * across) * 16 + lane;
  const int64_t n = s.segments, C = a.channels;
  const bool active = c < C;
  const int64_t each = (n + kJoinGroups - 1) / kJoinGroups, from = group * each, to = from + each < n ? from + each : n;
  const float* parts = reinterpret_cast<const float*>(a.ws) + b * n * 3 * C + c;
  float* starts = reinterpret_cast<float*>(a.ws) + a.batch * n * 3 * C + b * n * C + c;
  const auto part = [&](int64_t i) {
    const float* p = parts + (BACK ? n - 1 - i : i) * 3 * C;
    return Run{p[0], p[C], p[2 * C]};
  };
  Run mine{1.0f, 0.0f, 0.0f};
  if (active) {
#pragma unroll 4
    for (int64_t i = from; i < to; ++i) mine = then(mine, part(i));
  }
  lds[0][group][lane] = mine.A;
  lds[1][group][lane] = mine.c;
  lds[2][group][lane] = mine.B;
  const float* first = BACK ? a.glast : a.state;
  float state = active && first ? first[b * C + c] : 0.0f;
  __syncthreads();
  if (!active) return;
  for (int g = 0; g < group; ++g) state = apply(Run{lds[0][g][lane], lds[1][g][lane], lds[2][g][lane]}, state);
#pragma unroll 4
  for (int64_t i = from; i < to; ++i) {
    starts[(BACK ? n - 1 - i : i) * C] = state;
    state = apply(part(i), state);
  }
}

// The first state of this workgroup's part.
template <int V>
__device__ __forceinline__ void first_state(const RecArgs& a, const RecShape& s, const Place& at, const float* first,
                                            float (&state)[V]) {
  const float* p = first ? first + at.b * a.channels : nullptr;
  if (s.segments > 1)
    p = reinterpret_cast<const float*>(a.ws) + (a.batch * 3 + at.b) * s.segments * a.channels + at.seg * a.channels;
#pragma unroll
  for (int v = 0; v < V; ++v) state[v] = p ? p[at.c + v] : 0.0f;
}

// What a tile takes from memory.
template <class T, int V, int R, bool GRAD>
struct Raw {
  Vec<T, V> f[R], x[R], d[GRAD ? R : 1];
};

// (A, c, B) of every part: of the states, or (BACK) of the gradients.
template <class T, int V, int R, bool BACK>
__global__ __launch_bounds__(kThreads) void recurrence_parts_kernel(RecArgs a, RecShape s) {
  __shared__ float lds[3 * kThreads * V];
  const Place at = place<V>(a, s);
  Shared<V> sh{lds, s.L, s.G, (int)(threadIdx.x & (s.L - 1))};
  const int64_t len = length_of(a, at.b), C = a.channels, stride = (int64_t)s.G * R * C, row = at.b * a.steps * C;
  const uint32_t pitch = (uint32_t)(C * (int64_t)sizeof(T)), offset = at.g * R * pitch + (uint32_t)(at.c * (int64_t)sizeof(T));
  const T *gate = reinterpret_cast<const T*>(a.gate) + row, *second = reinterpret_cast<const T*>(BACK ? a.gh : a.x) + row;
  const bool there = BACK ? a.gh != nullptr : true;
  Run all[V];
#pragma unroll
  for (int v = 0; v < V; ++v) all[v] = Run{1.0f, 0.0f, 0.0f};
  const int64_t first = at.seg * s.per;
  const int64_t last = live_tiles<R>(s, len, first, first + s.per < s.tiles ? first + s.per : s.tiles);
  for (int64_t i = 0; i < last - first; ++i) {
    const int64_t tile = BACK ? last - 1 - i : first + i;
    const Tile<R> in(a, s, tile, at.g, len);
    Vec<T, V> f[R], x[R];
    load_steps<T, V, R>(gate + tile * stride, offset, in.left, in.whole, pitch, f);
    load_steps<T, V, R>(second + tile * stride, offset, there ? in.left : 0, in.whole && there, pitch, x);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      Run r{1.0f, 0.0f, 0.0f};
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const int q = BACK ? R - 1 - j : j;
        float k, m = small_gate((float)f[q].v[v], k);
        const bool none = !in.whole && q >= in.left;
        if (none) m = 0.0f, k = 1.0f;
        lengthen(r, m, k);
        const float B = BACK ? kept(r.B + (float)x[q].v[v], m) : step(r.B, (float)x[q].v[v], m);
        r.B = none ? r.B : B;
      }
      settle(r);
      sh.put(at.g, v, r);
    }
    __syncthreads();
    for (int four = 0; four < s.G; four += 4)
#pragma unroll
      for (int j = four; j < four + 4; ++j)
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
  const int64_t len = length_of(a, at.b), C = a.channels, stride = (int64_t)s.G * R * C, row = at.b * a.steps * C;
  const uint32_t pitch = (uint32_t)(C * (int64_t)sizeof(T)), offset = at.g * R * pitch + (uint32_t)(at.c * (int64_t)sizeof(T));
  const T *gate = reinterpret_cast<const T*>(a.gate) + row, *xs = reinterpret_cast<const T*>(a.x) + row;
  T* hs = reinterpret_cast<T*>(a.h) + row;
  float state[V];
  const int64_t first = at.seg * s.per, end = first + s.per < s.tiles ? first + s.per : s.tiles;
  const int64_t last = live_tiles<R>(s, len, first, end);
  Raw<T, V, R, false> now;
  const auto load = [&](int64_t tile, Raw<T, V, R, false>& r) {
    const Tile<R> in(a, s, tile, at.g, len);
    load_steps<T, V, R>(gate + tile * stride, offset, in.left, in.whole, pitch, r.f);
    load_steps<T, V, R>(xs + tile * stride, offset, in.left, in.whole, pitch, r.x);
  };
  if (first < last) load(first, now);
  first_state(a, s, at, a.state, state);
  for (int64_t tile = first; tile < last; ++tile) {
    Tile<R> in(a, s, tile, at.g, len);
    float m[R][V], h[V];
    if (a.saved && at.g == 0 && at.active) {
#pragma unroll
      for (int v = 0; v < V; ++v) a.saved[(at.b * s.tiles + tile) * C + at.c + v] = state[v];
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      Run r{1.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < R; ++i) {
        float k;
        m[i][v] = small_gate((float)now.f[i].v[v], k);
        const bool none = !in.whole && i >= in.left;
        if (none) m[i][v] = 0.0f, k = 1.0f;
        lengthen(r, m[i][v], k);
        const float B = step(r.B, (float)now.x[i].v[v], m[i][v]);
        r.B = none ? r.B : B;
      }
      settle(r);
      sh.put(at.g, v, r);
    }
    Raw<T, V, R, false> next;  // on its way while this tile is finished
    if (tile + 1 < last) load(tile + 1, next);
    __syncthreads();
    for (int four = 0; four < s.G; four += 4)
#pragma unroll
      for (int g = four; g < four + 4; ++g)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          if (g == at.g) h[v] = state[v];
          state[v] = apply(sh.get(g, v), state[v]);
        }
    __syncthreads();
    anew(m);
    anew(in.left);
    Vec<T, V> y[R];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        h[v] = step(h[v], (float)now.x[i].v[v], m[i][v]);
        y[i].v[v] = (T)(in.whole || i < in.left ? h[v] : 0.0f);
      }
    if (at.active) store_steps<T, V, R>(hs + tile * stride, offset, in.rows, in.full, pitch, y);
    now = next;
  }
  const Vec<T, V> zeros[R] = {};
  for (int64_t tile = last; tile < end && at.active; ++tile) {
    const Tile<R> in(a, s, tile, at.g, len);
    store_steps<T, V, R>(hs + tile * stride, offset, in.rows, in.full, pitch, zeros);
  }
  if (at.seg == s.segments - 1 && at.g == 0 && at.active) {
#pragma unroll
    for (int v = 0; v < V; ++v) a.last[at.b * C + at.c + v] = state[v];
  }
}

template <class T, int V, int R>
__global__ __launch_bounds__(kThreads, 2) void recurrence_bwd_kernel(RecArgs a, RecShape s) {
  __shared__ float lds[4 * kThreads * V];  // (A, c, B) of the states, B of the gradients
  const Place at = place<V>(a, s);
  Shared<V> sh{lds, s.L, s.G, (int)(threadIdx.x & (s.L - 1))};
  const int64_t len = length_of(a, at.b), C = a.channels, stride = (int64_t)s.G * R * C, row = at.b * a.steps * C;
  const uint32_t pitch = (uint32_t)(C * (int64_t)sizeof(T)), offset = at.g * R * pitch + (uint32_t)(at.c * (int64_t)sizeof(T));
  const T *gate = reinterpret_cast<const T*>(a.gate) + row, *xs = reinterpret_cast<const T*>(a.x) + row;
  const T* gh = reinterpret_cast<const T*>(a.gh) + row;
  float grad[V];  // of the state after the tile, through later steps
  const int64_t first = at.seg * s.per, end = first + s.per < s.tiles ? first + s.per : s.tiles;
  const int64_t last = live_tiles<R>(s, len, first, end);
  Raw<T, V, R, true> now;
  float start[V];
  const auto load = [&](int64_t tile, Raw<T, V, R, true>& r, float(&h)[V]) {
    const Tile<R> in(a, s, tile, at.g, len);
    load_steps<T, V, R>(gate + tile * stride, offset, in.left, in.whole, pitch, r.f);
    load_steps<T, V, R>(xs + tile * stride, offset, in.left, in.whole, pitch, r.x);
    load_steps<T, V, R>(gh + tile * stride, offset, a.gh ? in.left : 0, in.whole && a.gh, pitch, r.d);
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = a.saved[(at.b * s.tiles + tile) * C + at.c + v];
  };
  if (first < last) load(last - 1, now, start);
  first_state(a, s, at, a.glast, grad);
  for (int64_t tile = last - 1; tile >= first; --tile) {
    Tile<R> in(a, s, tile, at.g, len);
    float m[R][V], h[V], e[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      Run r{1.0f, 0.0f, 0.0f};
      float back = 0.0f;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        float k;
        m[i][v] = small_gate((float)now.f[i].v[v], k);
        if (!in.whole && i >= in.left) m[i][v] = 0.0f, k = 1.0f;
        lengthen(r, m[i][v], k);
        r.B = step(r.B, (float)now.x[i].v[v], m[i][v]);
      }
#pragma unroll
      for (int i = R - 1; i >= 0; --i) {
        anew(m[i][v]);
        back = kept(back + (float)now.d[i].v[v], m[i][v]);
      }
      settle(r);
      sh.put(at.g, v, r);
      sh.ref(3, at.g, v) = back;
      h[v] = start[v];
    }
    Raw<T, V, R, true> next;  // on its way while this tile is finished
    if (tile > first) load(tile - 1, next, start);
    __syncthreads();
#pragma unroll 1  // (several at a time take more scalar registers than there are)
    for (int g = 0; g < at.g; ++g)
#pragma unroll
      for (int v = 0; v < V; ++v) h[v] = apply(sh.get(g, v), h[v]);
#pragma unroll 1
    for (int two = s.G - 2; two >= 0; two -= 2)
#pragma unroll
      for (int j = 1; j >= 0; --j)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const int g = two + j;
          if (g == at.g) e[v] = grad[v];
          Run r = sh.get(g, v);
          r.B = sh.ref(3, g, v);
          grad[v] = apply(r, grad[v]);
        }
    __syncthreads();
    anew(m);
    float diff[R][V];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float xv = (float)now.x[i].v[v];
        diff[i][v] = h[v] - xv;
        h[v] = step(h[v], xv, m[i][v]);
      }
    anew(m);
    anew(in.left);
    Vec<T, V> ox[R], of[R];
#pragma unroll
    for (int i = R - 1; i >= 0; --i)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float D = (float)now.d[i].v[v] + e[v], small = fabsf(m[i][v]);
        const bool is = in.whole || i < in.left;
        e[v] = is ? kept(D, m[i][v]) : D;
        ox[i].v[v] = (T)(is ? taken(D, m[i][v]) : 0.0f);
        of[i].v[v] = (T)(is ? diff[i][v] * D * fmaf(-small, small, small) : 0.0f);
      }
    if (at.active) {
      if (a.gx) store_steps<T, V, R>(reinterpret_cast<T*>(a.gx) + row + tile * stride, offset, in.rows, in.full, pitch, ox);
      anew(in.rows);
      if (a.ggate) store_steps<T, V, R>(reinterpret_cast<T*>(a.ggate) + row + tile * stride, offset, in.rows, in.full, pitch, of);
    }
    now = next;
  }
  const Vec<T, V> zeros[R] = {};
  for (int64_t tile = last; tile < end && at.active; ++tile) {
    const Tile<R> in(a, s, tile, at.g, len);
    if (a.gx) store_steps<T, V, R>(reinterpret_cast<T*>(a.gx) + row + tile * stride, offset, in.rows, in.full, pitch, zeros);
    if (a.ggate) store_steps<T, V, R>(reinterpret_cast<T*>(a.ggate) + row + tile * stride, offset, in.rows, in.full, pitch, zeros);
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

// launch(args) for as many sequences at a time as a launch may have threads for,
// which are counted in 32 bits.  A batch of that size has no parts.
template <class T, class F>
hipError_t in_runs(const RecArgs& a, const RecShape& s, F launch) {
  const int64_t most = rec_run(s);
  const auto move = [](auto& p, int64_t n) { p = p ? p + n : p; };
  const auto move_features = [](auto& p, int64_t n) {
    using V = std::remove_reference_t<decltype(p)>;
    p = p ? (V)((uintptr_t)p + (uintptr_t)n * sizeof(T)) : p;
  };
  for (int64_t b = 0; b < a.batch; b += most) {
    RecArgs r = a;
    r.batch = a.batch - b < most ? a.batch - b : most;
    const int64_t features = b * a.steps * a.channels;
    move_features(r.x, features);
    move_features(r.gate, features);
    move_features(r.h, features);
    move_features(r.gh, features);
    move_features(r.gx, features);
    move_features(r.ggate, features);
    move(r.state, b * a.channels);
    move(r.lengths, b);
    move(r.last, b * a.channels);
    move(r.saved, b * s.tiles * a.channels);
    move(r.glast, b * a.channels);
    move(r.gstate, b * a.channels);
    const hipError_t st = launch(r);
    if (st != hipSuccess) return st;
  }
  return hipSuccess;
}

}  // namespace

template <class T>
hipError_t launch_recurrence_fwd(const RecArgs& all, hipStream_t stream) {
  const RecShape s = rec_shape(all.batch, all.steps, all.channels, sizeof(T) == 2);
  return with_shape<T>(s, [&](auto v, auto r) {
    return in_runs<T>(all, s, [&](const RecArgs& a) {
      const dim3 grid((unsigned)(a.batch * s.segments * s.blocks)), block(kThreads);
      if (s.segments > 1) {
        hipLaunchKernelGGL((recurrence_parts_kernel<T, v.value, r.value, false>), grid, block, 0, stream, a, s);
        hipLaunchKernelGGL(recurrence_starts_kernel<false>, dim3((unsigned)(a.batch * ((a.channels + 15) / 16))), dim3(kJoin), 0,
                           stream, a, s);
      }
      hipLaunchKernelGGL((recurrence_fwd_kernel<T, v.value, r.value>), grid, block, 0, stream, a, s);
      return hipGetLastError();
    });
  });
}

template <class T>
hipError_t launch_recurrence_bwd(const RecArgs& all, hipStream_t stream) {
  const RecShape s = rec_shape(all.batch, all.steps, all.channels, sizeof(T) == 2);
  return with_shape<T>(s, [&](auto v, auto r) {
    return in_runs<T>(all, s, [&](const RecArgs& a) {
      const dim3 grid((unsigned)(a.batch * s.segments * s.blocks)), block(kThreads);
      if (s.segments > 1) {
        hipLaunchKernelGGL((recurrence_parts_kernel<T, v.value, r.value, true>), grid, block, 0, stream, a, s);
        hipLaunchKernelGGL(recurrence_starts_kernel<true>, dim3((unsigned)(a.batch * ((a.channels + 15) / 16))), dim3(kJoin), 0,
                           stream, a, s);
      }
      hipLaunchKernelGGL((recurrence_bwd_kernel<T, v.value, r.value>), grid, block, 0, stream, a, s);
      return hipGetLastError();
    });
  });
}

template hipError_t launch_recurrence_fwd<float>(const RecArgs&, hipStream_t);
template hipError_t launch_recurrence_fwd<f16>(const RecArgs&, hipStream_t);
template hipError_t launch_recurrence_fwd<bf16>(const RecArgs&, hipStream_t);
template hipError_t launch_recurrence_bwd<float>(const RecArgs&, hipStream_t);
template hipError_t launch_recurrence_bwd<f16>(const RecArgs&, hipStream_t);
template hipError_t launch_recurrence_bwd<bf16>(const RecArgs&, hipStream_t);

}  // namespace ecc
