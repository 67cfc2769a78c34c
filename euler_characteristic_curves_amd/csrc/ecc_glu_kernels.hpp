// The gated pair of projections of a feed-forward block (contract:
// include/ecc_train.h), included by one source per element type.
//
//   a = x Wg^T + bg,  b = x Wu^T + bu,  h = act(a) b.
// Backwards, from a and b formed anew,
//   da = dh b act'(a),  db = dh act(a),
//   dx = da Wg + db Wu,  dWg = da^T x,  dWu = db^T x,  dbg = sum da,  dbu = sum db.
//
// All of it is products of matrices on the matrix unit: tiles of 64 FM x 64 FN
// results a workgroup of four waves, steps of 64 bytes along the summed axis
// through LDS, float32 sums.  A tile of the forward product holds the same 64
// hidden units of both projections, so activation and product are its epilogue;
// the backward one's is da and db, written to the workspace as the next products'
// operands.  Of 16 bits they are kept in two parts, the number rounded and what
// that leaves, and both are multiplied: with the first alone dx and dW were 1.41
// times as far off as their own rounding (1.6 times in single elements), however
// many terms a sum has, as relative errors of the terms pass on to it.  It makes
// dx and dW twice the products.
//
// Operands of two kinds: those that lie along the summed axis, and those that
// lie across it (the weights in dx, both operands in dW).  The second are kept
// in LDS as they lie and turned on the way to the registers, by the transposing
// read where elements have 16 bits.
//
// Large products are bound by the matrix unit at the clock that the power
// leaves: 16384 x 1024 to 2816, bfloat16, forward 198 us (9.5e14 operations a
// second), gradients of the projections 256 us, the two parts of dx 392 us, of dW
// 429 us and 14 for its join.  1999 x 333 to 877, float32: 29 to 35 us each
// (6.7e13 to 8.1e13 of 1.5e14: 448 to 504 workgroups, two to some compute units
// and one to others).  2^19 x 64 to 160, float16: 80, 211, 219 and 203 us, bound by
// the bytes of the results and of da and db's two parts, 2.9 to 4 TB/s.

#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "ecc_act.hpp"
#include "ecc_block_internal.hpp"

namespace ecc {
namespace {

constexpr int kNT = 256;
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef f16 f16x8 __attribute__((ext_vector_type(8)));
typedef bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

enum Kind { kForward, kGates, kInput, kWeight };
constexpr bool is_dual(int kind) { return kind == kForward || kind == kGates; }
// Whether the operands lie along the summed axis.
constexpr bool a_along(int kind) { return kind != kWeight; }
constexpr bool b_along(int kind) { return is_dual(kind); }

template <class T>
constexpr int kPer = 16 / (int)sizeof(T);  // elements of a 16-byte chunk
template <class T>
constexpr int kStep = 64 / (int)sizeof(T);  // elements of a step along the summed axis
template <class T>
constexpr bool kPairs = sizeof(T) == 2;  // da and db in two parts: what rounding leaves, 2 pitch further on what it rounds to
// float16 has the mantissa but not the range: da is 2^4 (second + 2^-11 first) of
// its parts, so that numbers up to 2^20 are there, and steps of 2^-31 (of parts
// that are simply added 65504, and 2^-24: a loss that is scaled for training in
// float16 went beyond the one, 5000 rows of gradients of 2^-22 had dW off by 57
// times its rounding for the other).
template <class T>
constexpr bool kScaled = std::is_same<T, f16>::value;
constexpr float kPartScale = 0x1p-4f, kRestScale = 0x1p11f;

// One product.
template <class T>
struct Product {
  const T* A;
  int64_t pitchA, stepA;  // stepA: from one matrix, or part of the sum, to the next
  const T* B[2];
  int64_t pitchB;
  int64_t M, N, K;  // N: hidden units of one projection in a dual product; K of one part of the sum
  int parts;        // parts of the sum, rests first: in dx A + i stepA with B[i % 2], in dW A + (z + 2 i) stepA
  int splits;
  int64_t tiles_m, tiles_n;
  float* part;
  GluArgs a;
  int64_t pitch;   // of the workspace's gradients
  T* dab;
  float* bias;     // partial sums of da and db, null: not wanted
  T* out[2];
  int64_t pitch_out;
};

// ---------------------------------------------------------------- loading
// Rows (of the operand, across the sum) of a tile in LDS.  Along: rows of 64
// bytes, four chunks, permuted so that 16 neighbouring rows at one chunk meet
// every bank once.  Across: a row of ROWS elements for every step of the sum,
// chunks permuted so that the rows that one read serves lie in different banks.
template <class T, bool ALONG, int ROWS>
struct Tile {
  static constexpr int kChunks = ROWS / 64;                       // a thread
  static constexpr int kLine = ROWS * (int)sizeof(T) / 16;        // chunks of a line, across
  __device__ static __forceinline__ int permuted(int line, int chunk) {
    if (ALONG) return chunk ^ (line >> 2 & 3);
    if (sizeof(T) == 4) return chunk ^ (line >> 2 & 1) * 8;
    return kLine == 8 ? chunk ^ (line >> 1 & 1) * 4 : chunk ^ (line & 3) * 4;
  }
  // Line (row along, summed index across) and chunk of this thread's chunk i.
  __device__ static __forceinline__ void mine(int i, int& line, int& chunk) {
    const int q = i * kNT + threadIdx.x, per = ALONG ? 4 : kLine;
    line = q / per;
    chunk = permuted(line, q % per);
  }
  // A chunk from anywhere, with zeros behind `n` rows and `end` along the sum.
  __device__ static __forceinline__ u32x4 fetch(const T* p, int64_t pitch, int64_t row0, int64_t n, int64_t k0, int64_t end,
                                                int i) {
    int line, chunk;
    mine(i, line, chunk);
    const int64_t row = ALONG ? row0 + line : row0 + chunk * kPer<T>, k = ALONG ? k0 + chunk * kPer<T> : k0 + line;
    const int64_t left = ALONG ? (row < n ? end - k : 0) : (k < end ? n - row : 0);
    Vec<T, kPer<T>> v = {};
    if (left > 0) {
      const T* at = ALONG ? p + row * pitch + k : p + k * pitch + row;
      if (left >= kPer<T>) {
        load_vec(at, v);
      } else {
#pragma unroll
        for (int j = 0; j < kPer<T> - 1; ++j)
          if (j < left) v.v[j] = at[j];
      }
    }
    u32x4 r;
    __builtin_memcpy(&r, &v, 16);
    return r;
  }
  // Bytes from the tile's first element of a step to this thread's chunk i, of
  // lines and chunks that are there (what those behind them would be is not used).
  __device__ static __forceinline__ uint32_t offset(int64_t pitch, int64_t row0, int64_t n, int i) {
    int line, chunk;
    mine(i, line, chunk);
    if (ALONG)
      line = line < n - row0 ? line : (int)(n - row0 - 1);
    else
      chunk = chunk < (n - row0) / kPer<T> ? chunk : (int)((n - row0) / kPer<T>) - 1;
    return (uint32_t)((int64_t)line * pitch * (int64_t)sizeof(T)) + chunk * 16;
  }
};

// One of this thread's chunks of step s, straight to LDS, if s is before `last`:
// the base is the same for all lanes, and so is where a wave's 64 chunks go.  In
// assembly, because the compiler would wait for all such loads before it reads
// what one of them may have written, as it cannot tell which are complete; the
// waits are wait_loads.  (m0 is not the compiler's to keep anything in.)
__device__ __forceinline__ void load_chunk(const void* step, uint32_t offset, uint32_t lds, int s, int last) {
  // (uniform values do not always stay in scalar registers)
  const uint64_t at = (uint64_t)step;
  const uint64_t base = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)at) |
                        (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(at >> 32)) << 32;
  s = __builtin_amdgcn_readfirstlane(s);
  last = __builtin_amdgcn_readfirstlane(last);
  asm volatile(
      "s_cmp_ge_i32 %3, %4\n\ts_cbranch_scc1 .Lnot_wanted%=\n\ts_mov_b32 m0, %0\n\ts_nop 0\n\t"
      "global_load_lds_dwordx4 %1, %2\n.Lnot_wanted%=:"
      :
      : "s"(lds), "v"(offset), "s"(base), "s"(s), "s"(last)
      : "memory", "scc");
}
// Where this wave's part of a tile begins in LDS.
__device__ __forceinline__ uint32_t wave_lds(char* lds) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds +
         __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * 1024;
}

// Waits for all but the newest VM loads of this wave and for what it has read
// of LDS, then for the other waves.
template <int VM>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(VM) : "memory");
}

// ---------------------------------------------------------------- fragments
template <class T>
struct Fragment {
  u32x4 v;
};

// 32 rows from row0 on, chunks 2 s and 2 s + 1 of the step (lanes 32 and up have the second).
template <class T, bool ALONG, int ROWS>
__device__ __forceinline__ Fragment<T> read_fragment(const char* lds, int row0, int s) {
  const int lane = threadIdx.x & 63, high = lane >> 5;
  Fragment<T> f;
  if constexpr (ALONG) {
    const int row = row0 + (lane & 31);
    f.v = *reinterpret_cast<const u32x4*>(lds + row * 64 + (Tile<T, ALONG, ROWS>::permuted(row, s * 2 + high) << 4));
  } else if constexpr (sizeof(T) == 4) {
    const int col = row0 + (lane & 31);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int k = s * 8 + high * 4 + j;
      f.v[j] = *reinterpret_cast<const uint32_t*>(lds + k * (ROWS * 4) + (Tile<T, ALONG, ROWS>::permuted(k, col >> 2) << 4) +
                                                  (col & 3) * 4);
    }
  } else {
    // 16 lanes read 4 lines of 16 elements, and each gets a column of them
    const int i = lane & 15, col = row0 + (lane & 16) + (i & 3) * 4;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int k = s * 16 + high * 8 + j * 4 + (i >> 2);
      const char* at = lds + k * (ROWS * 2) + (Tile<T, ALONG, ROWS>::permuted(k, col >> 3) << 4) + (col & 7) * 2;
      const s16x4 r = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (__attribute__((address_space(3))) s16x4*)reinterpret_cast<const s16x4*>(at));
      __builtin_memcpy(reinterpret_cast<char*>(&f.v) + j * 8, &r, 8);
    }
  }
  return f;
}

__device__ __forceinline__ f32x16 multiply(const Fragment<f16>& a, const Fragment<f16>& b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a.v), __builtin_bit_cast(f16x8, b.v), c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 multiply(const Fragment<bf16>& a, const Fragment<bf16>& b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a.v), __builtin_bit_cast(bf16x8, b.v), c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 multiply(const Fragment<float>& a, const Fragment<float>& b, f32x16 c) {
  const f32x4 u = __builtin_bit_cast(f32x4, a.v), v = __builtin_bit_cast(f32x4, b.v);
#pragma unroll
  for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_32x32x2f32(u[j], v[j], c, 0, 0, 0);
  return c;
}

// A fragment's result r of a lane: row lane % 32 of the operand with M rows,
// and this one of the other.
__device__ __forceinline__ int result_col(int r) { return (r >> 2) * 8 + (threadIdx.x >> 5 & 1) * 4 + (r & 3); }

// ---------------------------------------------------------------- epilogues
// A fragment's 32 x 32 results pass through LDS, so that memory sees whole
// chunks of rows: 4 KB of its own for every wave, whose accesses keep their
// order.  Chunks of a row are permuted as they are in the tiles.
constexpr int kStage = 4096;
template <class T>
struct Stage {
  static constexpr int kLine = 32 * (int)sizeof(T), kChunks = kLine / 16, kTurns = 32 * kChunks / 64;
  char* lds;
  __device__ __forceinline__ char* at(int row, int chunk) const {
    return lds + row * kLine + ((sizeof(T) == 2 ? chunk ^ (row >> 2 & 3) : chunk ^ (row >> 1 & 7)) << 4);
  }
  __device__ __forceinline__ char* mine(int q) const {  // results 4 q to 4 q + 3
    const int lane = threadIdx.x & 63, byte = (q * 8 + (lane >> 5) * 4) * (int)sizeof(T);
    return at(lane & 31, byte >> 4) + (byte & 15);
  }
  __device__ __forceinline__ void put(const float (&v)[16]) const {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      Vec<T, 4> u;
#pragma unroll
      for (int r = 0; r < 4; ++r) u.v[r] = (T)v[q * 4 + r];
      __builtin_memcpy(__builtin_assume_aligned(mine(q), sizeof(u)), &u, sizeof(u));
    }
    __builtin_amdgcn_wave_barrier();
  }
  __device__ __forceinline__ void get(float (&v)[16]) const {
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      Vec<T, 4> u;
      __builtin_memcpy(&u, __builtin_assume_aligned(mine(q), sizeof(u)), sizeof(u));
#pragma unroll
      for (int r = 0; r < 4; ++r) v[q * 4 + r] = (float)u.v[r];
    }
    __builtin_amdgcn_wave_barrier();
  }
  // To and from memory: rows and columns that are left from p on.  p is the same
  // for all lanes, and 32 rows of any pitch fit 32 bits.
  __device__ __forceinline__ static uint32_t offset(int row, int col, int64_t pitch) {
    return (uint32_t)row * (uint32_t)(pitch * (int64_t)sizeof(T)) + (uint32_t)(col * (int)sizeof(T));
  }
  __device__ __forceinline__ void store(T* p, int64_t pitch, int64_t rows, int64_t cols) const {
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
      const int id = i * 64 + (threadIdx.x & 63), row = id / kChunks, chunk = id % kChunks, col = chunk * kPer<T>;
      const u32x4 u = *reinterpret_cast<const u32x4*>(at(row, chunk));
      if (row >= rows || col >= cols) continue;
      char* out = reinterpret_cast<char*>(p) + offset(row, col, pitch);
      if (col + kPer<T> <= cols) {
        // (one store of any alignment: of elements, the compiler makes three)
        typedef u32x4 u32x4_any __attribute__((aligned(2)));
        *reinterpret_cast<u32x4_any*>(out) = u;
      } else {
#pragma unroll
        for (int j = 0; j < kPer<T> - 1; ++j)
          if (col + j < cols) {
            if constexpr (sizeof(T) == 4)
              reinterpret_cast<uint32_t*>(out)[j] = u[j];
            else
              reinterpret_cast<uint16_t*>(out)[j] = (uint16_t)(u[j / 2] >> (j % 2 * 16));
          }
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
  __device__ __forceinline__ static void load(const T* p, int64_t pitch, int64_t rows, int64_t cols, u32x4 (&u)[kTurns]) {
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
      const int id = i * 64 + (threadIdx.x & 63), row = id / kChunks, col = id % kChunks * kPer<T>;
      u[i] = u32x4{};
      if (row >= rows || col >= cols) continue;
      const char* in = reinterpret_cast<const char*>(p) + offset(row, col, pitch);
      if (col + kPer<T> <= cols) {
        __builtin_memcpy(&u[i], in, 16);
      } else {
#pragma unroll
        for (int j = 0; j < kPer<T> - 1; ++j)
          if (col + j < cols) {
            if constexpr (sizeof(T) == 4)
              u[i][j] = reinterpret_cast<const uint32_t*>(in)[j];
            else
              u[i][j / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(in)[j] << (j % 2 * 16);
          }
      }
    }
  }
  __device__ __forceinline__ void place(const u32x4 (&u)[kTurns]) const {
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
      const int id = i * 64 + (threadIdx.x & 63);
      *reinterpret_cast<u32x4*>(at(id / kChunks, id % kChunks)) = u[i];
    }
  }
};

// Sums of 16 values a lane over the 32 rows of all waves' fragments: lanes 0 to
// 31 get one each.  lds: the wave's.
__device__ __forceinline__ float sum_rows(const float (&v)[16], float* lds) {
  const int lane = threadIdx.x & 63;
  // [row][column], columns turned by the row
#pragma unroll
  for (int r = 0; r < 16; ++r) lds[(lane & 31) * 32 + ((result_col(r) + lane) & 31)] = v[r];
  __builtin_amdgcn_wave_barrier();
  float s = 0.0f;
#pragma unroll 8
  for (int i = 0; i < 32; ++i) s += lds[i * 32 + ((lane + i) & 31)];
  __builtin_amdgcn_wave_barrier();
  return s;
}

// A tile's biases, of both projections, to `shared`.
template <class T>
__device__ __forceinline__ void load_biases(const Product<T>& p, int64_t tn, float* shared) {
  if (threadIdx.x < 128) {
    const T* bias = reinterpret_cast<const T*>(threadIdx.x < 64 ? p.a.bg : p.a.bu);
    const int64_t unit = tn * 64 + (threadIdx.x & 63);
    shared[threadIdx.x] = bias && unit < p.N ? (float)bias[unit] : 0.0f;
  }
}

// The results of a fragment of both projections, from row and unit0 on.
template <class T, int ACT>
__device__ __forceinline__ void forward_fragment(const Product<T>& p, const Stage<T>& stage, const f32x4* bias, const f32x16& a,
                                                 const f32x16& b, int64_t row, int64_t unit0) {
  float v[16];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const f32x4 ug = bias[q * 2], uu = bias[16 + q * 2];
#pragma unroll
    for (int r = q * 4; r < q * 4 + 4; ++r) v[r] = act_value<ACT>(a[r] + ug[r & 3]) * (b[r] + uu[r & 3]);
  }
  stage.put(v);
  stage.store(reinterpret_cast<T*>(p.a.h) + row * p.N + unit0, p.N, p.M - row, p.N - unit0);
}

// What rounding leaves: nothing of an infinity or a NaN, which the number itself passes on.
template <class T>
__device__ __forceinline__ float rest_of(float v) {
  const float first = (float)(T)v;
  return fabsf(first) < __builtin_inff() ? (v - first) * (kScaled<T> ? kRestScale : 1.0f) : 0.0f;
}

// Its gradients: `gh` has the result's.  sums(q, in, da, db) adds numbers 4 q to
// 4 q + 3 to the sums over rows; rows that are not there (`in`) have no gradient,
// but may have infinite projections.
template <class T, int ACT, class Sums, class Between>
__device__ __forceinline__ void gates_fragment(const Product<T>& p, const Stage<T>& stage, const f32x4* bias, const f32x16& a,
                                               const f32x16& b, int64_t row, int64_t unit0,
                                               u32x4 (&gh)[Stage<T>::kTurns], Sums sums, Between between) {
  const bool in = row + (threadIdx.x & 31) < p.M;
  float g[16], da[16];
  stage.place(gh);
  stage.get(g);
  between();  // gh is free
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const f32x4 ug = bias[q * 2], uu = bias[16 + q * 2];
#pragma unroll
    for (int r = q * 4; r < q * 4 + 4; ++r) {
      float y;
      const float u = b[r] + uu[r & 3], slope = act_slope<ACT>(a[r] + ug[r & 3], y);
      da[r] = g[r] * u * slope;
      g[r] *= y;
      // both parts come from this number: a product rounded straight to 16 bits
      // for one of them alone is a step off where it lies between two
      if constexpr (kPairs<T>) asm("" : "+v"(da[r]), "+v"(g[r]));
    }
    sums(q, in, da, g);
    if constexpr (kScaled<T>) {
#pragma unroll
      for (int r = q * 4; r < q * 4 + 4; ++r) {
        da[r] *= kPartScale;
        g[r] *= kPartScale;
      }
    }
    __builtin_amdgcn_sched_barrier(0);  // all at once would not fit the registers
  }
  const int64_t line = (kPairs<T> ? 4 : 2) * p.pitch;
  T* rest = p.dab + row * line + unit0;
  T* out = rest + (kPairs<T> ? 2 : 0) * p.pitch;
  stage.put(da);
  stage.store(out, line, p.M - row, p.N - unit0);
  stage.put(g);
  stage.store(out + p.pitch, line, p.M - row, p.N - unit0);
  if constexpr (kPairs<T>) {
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      asm("" : "+v"(da[r]), "+v"(g[r]));  // (rounded again: kept, the first parts do not fit the registers)
      da[r] = rest_of<T>(da[r]);
    }
    stage.put(da);
    stage.store(rest, line, p.M - row, p.N - unit0);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int r = 0; r < 16; ++r) g[r] = rest_of<T>(g[r]);
    stage.put(g);
    stage.store(rest + p.pitch, line, p.M - row, p.N - unit0);
  }
}

// A workgroup's sums over rows, to partial row `part`.  lds: 4 KB for this wave.
template <class T>
__device__ __forceinline__ void store_bias_sums(const Product<T>& p, int64_t part, int64_t tn, const float (&sum_a)[16],
                                                const float (&sum_b)[16], char* lds, float* shared) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wm = wave >> 1, wn = wave & 1;
  const int64_t unit0 = tn * 64 + wn * 32;
  const float a = sum_rows(sum_a, reinterpret_cast<float*>(lds)), b = sum_rows(sum_b, reinterpret_cast<float*>(lds));
  __syncthreads();  // the biases are read
  if (wm == 1 && lane < 32) {
    shared[wn * 32 + lane] = a;
    shared[64 + wn * 32 + lane] = b;
  }
  __syncthreads();
  if (wm == 0 && lane < p.N - unit0 && lane < 32) {
    float* out = p.bias + part * 2 * p.pitch + unit0 + lane;
    out[0] = a + shared[wn * 32 + lane];
    out[p.pitch] = b + shared[64 + wn * 32 + lane];
  }
}

// A workgroup's results: acc[i][j] is the fragment of rows wm FM 32 + 32 i.
// lds: kStage bytes for this wave; shared: 128 floats for all of them; sums_a,
// sums_b: 16 floats a thread, where FM > 1.
template <class T, int KIND, int FM, int FN, int ACT>
__device__ __forceinline__ void epilogue(const Product<T>& p, int z, int64_t tm, int64_t tn, f32x16 (&acc)[FM][FN], char* lds,
                                         float* shared, f32x4* sums_a, f32x4* sums_b) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wm = wave >> 1, wn = wave & 1;
  const int64_t row0 = tm * 64 * FM + wm * FM * 32;
  const Stage<T> stage{lds};
  if constexpr (is_dual(KIND)) {
    const int64_t unit0 = tn * 64 + wn * 32;
    load_biases(p, tn, shared);
    __syncthreads();
    const f32x4* bias = reinterpret_cast<const f32x4*>(shared + wn * 32 + (lane >> 5) * 4);
    if constexpr (KIND == kForward) {
#pragma unroll
      for (int i = 0; i < FM; ++i) forward_fragment<T, ACT>(p, stage, bias, acc[i][0], acc[i][1], row0 + i * 32, unit0);
    } else {
      const T* gh = reinterpret_cast<const T*>(p.a.gh);
      u32x4 next[Stage<T>::kTurns];
      Stage<T>::load(gh + row0 * p.N + unit0, p.N, p.M - row0, p.N - unit0, next);
      // sums of several fragments are in LDS: in registers they did not fit (46 of
      // a lane's went to memory and back, 78 with float16)
      float sum_a[16], sum_b[16];
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const int64_t row = row0 + i * 32;
        const auto sums = [&](int q, bool in, const float(&da)[16], const float(&db)[16]) {
          if (!p.bias) return;
          f32x4 va = {}, vb = {};
          const int at = q * kNT + threadIdx.x;
          if (i > 0) va = sums_a[at], vb = sums_b[at];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            va[r] += in ? da[q * 4 + r] : 0.0f;
            vb[r] += in ? db[q * 4 + r] : 0.0f;
          }
          if constexpr (FM > 1) {
            sums_a[at] = va, sums_b[at] = vb;
          } else {
#pragma unroll
            for (int r = 0; r < 4; ++r) sum_a[q * 4 + r] = va[r], sum_b[q * 4 + r] = vb[r];
          }
        };
        gates_fragment<T, ACT>(p, stage, bias, acc[i][0], acc[i][1], row, unit0, next, sums, [&] {
          if (i + 1 < FM) Stage<T>::load(gh + (row + 32) * p.N + unit0, p.N, p.M - row - 32, p.N - unit0, next);
        });
      }
      if (!p.bias) return;
      if constexpr (FM > 1) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const f32x4 va = sums_a[q * kNT + threadIdx.x], vb = sums_b[q * kNT + threadIdx.x];
#pragma unroll
          for (int r = 0; r < 4; ++r) sum_a[q * 4 + r] = va[r], sum_b[q * 4 + r] = vb[r];
        }
      }
      store_bias_sums(p, tm, tn, sum_a, sum_b, lds, shared);
    }
  } else {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int64_t row = row0 + i * 32, col = tn * 64 * FN + wn * FN * 32 + j * 32;
        float v[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) v[r] = kScaled<T> ? acc[i][j][r] * (1.0f / kPartScale) : acc[i][j][r];
        stage.put(v);
        stage.store(p.out[z] + row * p.pitch_out + col, p.pitch_out, p.M - row, p.N - col);
      }
  }
}

// Which tile a workgroup takes.  Workgroups are dealt out to the eight dies in
// turn, so that each gets a run of neighbours: eight tiles along M for every one
// along N, whose operands its cache then holds.  `shares` of all tiles come one
// after the other.
struct TileId {
  int tm, tn, share;  // tm counts the rows of all matrices
};
__device__ __forceinline__ TileId tile_of(uint32_t rows, uint32_t cols, uint32_t shares) {
  const uint32_t all = rows * cols * shares, die = blockIdx.x & 7, each = all >> 3, more = all & 7;
  uint32_t id = die * each + (die < more ? die : more) + (blockIdx.x >> 3);
  const uint32_t share = id / (rows * cols);
  id -= share * (rows * cols);
  const uint32_t group = id / (8 * cols), in = id - group * 8 * cols, high = rows - group * 8 < 8 ? rows - group * 8 : 8;
  const uint32_t tn = in / high;
  // (divisions leave the scalar registers, where loads want their bases)
  return TileId{__builtin_amdgcn_readfirstlane(group * 8 + (in - tn * high)), __builtin_amdgcn_readfirstlane(tn),
                __builtin_amdgcn_readfirstlane(share)};
}

// ---------------------------------------------------------------- products
// A step from LDS.  The second half's reads stand between the first half's
// products, and so do loads of a later step, `load(i)` with i below FM + FN, one
// with every second product: issued together, before the first read, they kept
// the wave from it for as long as the memory unit took to accept them.
template <class T, int KIND, int FM, int FN, class Load>
__device__ __forceinline__ void multiply_step(const char* la, const char* lb, f32x16 (&acc)[FM][FN], Load load) {
  constexpr int TM = 64 * FM, TN = 64 * FN;
  const int wave = threadIdx.x >> 6, wm = wave >> 1, wn = wave & 1;
  Fragment<T> a[2][FM], b[2][FN];
  const auto read = [&](int c, int n) {  // fragment n of half c
    if (n < FN)
      b[c][n] = read_fragment<T, b_along(KIND), TN>(lb, is_dual(KIND) ? n * 64 + wn * 32 : wn * FN * 32 + n * 32, c);
    else
      a[c][n - FN] = read_fragment<T, a_along(KIND), TM>(la, wm * FM * 32 + (n - FN) * 32, c);
  };
#pragma unroll
  for (int n = 0; n < FM + FN; ++n) read(0, n);
  constexpr int kProducts = FM * FN, kAll = FM + FN;
  int reads = 0, loads = 0;
#pragma unroll
  for (int n = 0; n < 2 * kProducts; ++n) {
    const int c = n / kProducts, i = n % kProducts / FN, j = n % FN;
    acc[i][j] = multiply(b[c][j], a[c][i], acc[i][j]);
    // (n + 1) kAll / kProducts reads by now, and half as many loads
#pragma unroll
    for (int k = 0; k < kAll; ++k) {
      if (reads < kAll && reads * kProducts < (n + 1) * kAll) read(1, reads++);
      if (loads < kAll && loads * 2 * kProducts < (n + 1) * kAll) load(loads++);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
}

// ALIGNED: operands and their rows begin at multiples of 16 bytes.  Whole steps
// then go straight to LDS, two of them on their way while a third is used; what
// is left of each part of the sum comes last, through registers.  Otherwise
// every step goes through registers, one ahead.
template <class T, int KIND, int FM, int FN, bool ALIGNED, int ACT>
__global__ __launch_bounds__(kNT, 2) void glu_kernel(Product<T> p) {
  constexpr int TM = 64 * FM, TN = 64 * FN, kA = TM * 64, kB = TN * 64;
  using TileA = Tile<T, a_along(KIND), TM>;
  using TileB = Tile<T, b_along(KIND), TN>;
  // arrays of their own, so that a read of one is known not to wait for another's loads
  __shared__ __align__(16) char a0[kA], b0[kB], a1[kA], b1[kB], a2[ALIGNED ? kA : 512], b2[ALIGNED ? kB : 16];
  const TileId id = tile_of((uint32_t)p.tiles_m * (KIND == kWeight ? 2 : 1), (uint32_t)p.tiles_n, (uint32_t)p.splits);
  const int z = KIND == kWeight && id.tm >= p.tiles_m ? 1 : 0, split = id.share;
  const int64_t tm = id.tm - z * p.tiles_m, tn = id.tn;
  if (KIND == kWeight && !p.out[z]) return;  // not wanted
  // steps of the sum: the whole ones of every part, then what is left of each; in
  // two groups where the rests have a scale of their own
  constexpr int kGroups = kScaled<T> && !is_dual(KIND) ? 2 : 1;
  const int left = (int)(p.K % kStep<T>), whole = (int)(p.K / kStep<T>) + (!ALIGNED && left ? 1 : 0);
  const int parts = p.parts / kGroups, direct = whole * parts, all = ALIGNED && left ? direct + parts : direct;
  const int share = __builtin_amdgcn_readfirstlane((all * kGroups + p.splits - 1) / p.splits);
  int group = 0;
  const auto place = [&](int s, int& part, int64_t& k0) {  // step s of the group
    part = 0;
    if (ALIGNED && s >= direct) {
      part = s - direct;
      k0 = (int64_t)whole * kStep<T>;
    } else {
      if (!is_dual(KIND)) part = (s >= whole) + (s >= 2 * whole) + (s >= 3 * whole);
      k0 = (int64_t)(s - part * whole) * kStep<T>;
    }
    part += group * parts;
  };
  const auto base_a = [&](int part) { return p.A + (KIND == kWeight ? z + 2 * part : part) * p.stepA; };
  f32x16 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
  u32x4 ra[TileA::kChunks], rb[TileB::kChunks];
  const auto fetch = [&](int s) {
    int part;
    int64_t k0;
    place(s, part, k0);
#pragma unroll
    for (int i = 0; i < TileA::kChunks; ++i) ra[i] = TileA::fetch(base_a(part), p.pitchA, tm * TM, p.M, k0, p.K, i);
#pragma unroll
    for (int i = 0; i < TileB::kChunks; ++i) {
      if constexpr (is_dual(KIND))  // 64 rows of either projection: chunk i is one of rows 64 i to 64 i + 63
        rb[i] = TileB::fetch(p.B[i] - i * 64 * p.pitchB, p.pitchB, tn * 64, p.N + i * 64, k0, p.K, i);
      else
        rb[i] = TileB::fetch(p.B[KIND == kInput ? part & 1 : 0], p.pitchB, tn * TN, p.N, k0, p.K, i);
    }
  };
  const auto put = [&](char* la, char* lb) {
#pragma unroll
    for (int i = 0; i < TileA::kChunks; ++i) *reinterpret_cast<u32x4*>(la + (i * kNT + threadIdx.x) * 16) = ra[i];
#pragma unroll
    for (int i = 0; i < TileB::kChunks; ++i) *reinterpret_cast<u32x4*>(lb + (i * kNT + threadIdx.x) * 16) = rb[i];
  };
  uint32_t offA[TileA::kChunks], offB[TileB::kChunks];
  if constexpr (ALIGNED) {
#pragma unroll
    for (int i = 0; i < TileA::kChunks; ++i) offA[i] = TileA::offset(p.pitchA, tm * TM, KIND == kWeight ? p.pitch : p.M, i);
#pragma unroll
    for (int i = 0; i < TileB::kChunks; ++i) {
      if constexpr (is_dual(KIND))
        offB[i] = Tile<T, true, 64>::offset(p.pitchB, tn * 64, p.N, 0);
      else
        offB[i] = TileB::offset(p.pitchB, tn * TN, b_along(KIND) ? p.N : p.pitchB, i);
    }
  }
#pragma unroll 1
  for (; group < kGroups; ++group) {
    // this workgroup's steps are [from, to)
    const auto within = [&](int s) { return s < 0 ? 0 : (s < all ? s : all); };
    const int from = within(split * share - group * all), to = within((split + 1) * share - group * all);
    if constexpr (ALIGNED) {
      const int last = to < direct ? to : direct;  // of those that go straight to LDS
      const T *const first0 = p.B[0], *const first1 = p.B[1];
      // a step's first elements of A, and of B (of both projections)
      struct Bases {
        const T *a, *b0, *b1;
      };
      const auto bases = [&](int s) {
        int part;
        int64_t k0;
        place(s, part, k0);
        const T* A = base_a(part);
        Bases r;
        r.a = a_along(KIND) ? A + tm * TM * p.pitchA + k0 : A + k0 * p.pitchA + tm * TM;
        if constexpr (is_dual(KIND)) {
          r.b0 = first0 + tn * 64 * p.pitchB + k0;
          r.b1 = first1 + tn * 64 * p.pitchB + k0;
        } else {
          const T* B = first0;
          if (KIND == kInput && part & 1) B = first1;
          r.b0 = r.b1 = B + k0 * p.pitchB + tn * TN;
        }
        return r;
      };
      const auto load = [&](const Bases& r, int s, char* la, char* lb, int i) {  // chunk i, A's first
        if (i < FM)
          load_chunk(r.a, offA[i], wave_lds(la) + i * (kNT * 16), s, last);
        else
          load_chunk(is_dual(KIND) && i > FM ? r.b1 : r.b0, offB[i - FM], wave_lds(lb) + (i - FM) * (kNT * 16), s, last);
      };
      const auto load_all = [&](int s, char* la, char* lb) {
        const Bases r = bases(s);
#pragma unroll
        for (int i = 0; i < FM + FN; ++i) load(r, s, la, lb, i);
      };
      const auto step = [&](int s, char* la, char* lb, char* na, char* nb) {
        if (s >= last) return;
        const Bases r = bases(s + 2);
        if (s + 1 < last)
          wait_loads<FM + FN>();
        else
          wait_loads<0>();
        multiply_step<T, KIND, FM, FN>(la, lb, acc, [&](int i) { load(r, s + 2, na, nb, i); });
      };
      load_all(from, a0, b0);
      load_all(from + 1, a1, b1);
      for (int s = from; s < last; s += 3) {
        step(s, a0, b0, a2, b2);
        step(s + 1, a1, b1, a0, b0);
        step(s + 2, a2, b2, a1, b1);
      }
      for (int s = from > direct ? from : direct; s < to; ++s) {
        __syncthreads();
        fetch(s);
        put(a0, b0);
        __syncthreads();
        multiply_step<T, KIND, FM, FN>(a0, b0, acc, [](int) {});
      }
    } else {
      if (from < to) {
        fetch(from);
        put(a0, b0);
      }
      __syncthreads();
      const auto step = [&](int s, char* la, char* lb, char* na, char* nb) {
        if (s >= to) return;
        if (s + 1 < to) fetch(s + 1);
        multiply_step<T, KIND, FM, FN>(la, lb, acc, [](int) {});
        if (s + 1 < to) put(na, nb);
        __syncthreads();
      };
      for (int s = from; s < to; s += 2) {
        step(s, a0, b0, a1, b1);
        step(s + 1, a1, b1, a0, b0);
      }
    }
    if (group + 1 < kGroups) {
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int r = 0; r < 16; ++r) acc[i][j][r] *= 1.0f / kRestScale;
      __syncthreads();  // the stages are free
    }
  }
  if (p.splits > 1) {
    const int64_t tile = id.tm * p.tiles_n + tn;
    float* out = p.part + (tile * p.splits + split) * (kNT * FM * FN * 16) + threadIdx.x * 4;
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          f32x4 v;
#pragma unroll
          for (int r = 0; r < 4; ++r) v[r] = acc[i][j][q * 4 + r];
          *reinterpret_cast<f32x4*>(out + ((i * FN + j) * 4 + q) * (kNT * 4)) = v;
        }
    return;
  }
  if (ALIGNED) wait_loads<0>();  // the stages are free
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  epilogue<T, KIND, FM, FN, ACT>(p, z, tm, tn, acc, (wave & 2 ? b1 : b0) + (wave & 1) * kStage, reinterpret_cast<float*>(a2),
                                     reinterpret_cast<f32x4*>(a0), reinterpret_cast<f32x4*>(a1));
}

// Narrow sums, of up to four steps: a workgroup keeps the weights of its 64 units
// in LDS and walks over the rows, 64 at a time, two turns' rows and a turn's
// gradients on their way (2 x 64^3 x 64 to 160, float16, in tiles: 107 us forward,
// 306 us for the gates' gradients).
template <class T>
struct Narrow {
  static constexpr int kW = 128 * 64, kX = 64 * 64, kOut = 4 * 32 * 32 * (int)sizeof(T);  // bytes of a step, of the stages
  static size_t bytes(int steps) { return (size_t)steps * (kW + 3 * kX) + kOut + 128 * sizeof(float); }
};
template <class T, int KIND, int ACT>
__global__ __launch_bounds__(kNT, 2) void glu_narrow_kernel(Product<T> p, int walkers, int steps) {
  extern __shared__ __align__(16) char lds[];
  using N = Narrow<T>;
  char* const w = lds;
  char* const x = lds + steps * N::kW;
  char* const out = x + 3 * steps * N::kX;
  float* const shared = reinterpret_cast<float*>(out + N::kOut);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wm = wave >> 1, wn = wave & 1;
  const uint32_t tiles_n = (uint32_t)p.tiles_n, k = blockIdx.x >> 3, far = k / tiles_n;
  const int64_t tn = __builtin_amdgcn_readfirstlane(k - far * tiles_n);
  const int walker = __builtin_amdgcn_readfirstlane((blockIdx.x & 7) + 8 * far);
  const int64_t tiles_m = (p.M + 63) / 64, unit0 = tn * 64 + wn * 32;
  // zeros where a row ends within a step: no load writes them
  for (int i = threadIdx.x; i < steps * (N::kW + 3 * N::kX) / 16; i += kNT) reinterpret_cast<u32x4*>(lds)[i] = u32x4{};
  load_biases(p, tn, shared);
  __syncthreads();
  int line, chunk;
  Tile<T, true, 64>::mine(0, line, chunk);
  const auto fetch = [&](const T* base, int row, char* to, int s) {  // this thread's chunk of step s
    if (s * kStep<T> + chunk * kPer<T> < p.K)
      load_chunk(base + s * kStep<T>, (uint32_t)((int64_t)row * p.pitchA * (int64_t)sizeof(T)) + chunk * 16, wave_lds(to), 0, 1);
  };
  for (int s = 0; s < steps; ++s) {
    const int64_t left = p.N - tn * 64;
    const int row = line < left ? line : (int)left - 1;
    fetch(p.B[0] + tn * 64 * p.pitchB, row, w + s * N::kW, s);
    fetch(p.B[1] + tn * 64 * p.pitchB, row, w + s * N::kW + N::kW / 2, s);
  }
  const auto fetch_rows = [&](int64_t tm, char* to) {
    const int64_t left = p.M - tm * 64;
    const int row = line < left ? line : (int)left - 1;
    for (int s = 0; s < steps; ++s) fetch(p.A + tm * 64 * p.pitchA, row, to + s * N::kX, s);
  };
  constexpr int kTurns = Stage<T>::kTurns;
  u32x4 next[kTurns] = {};
  const auto fetch_gradients = [&](int64_t tm) {
    const int64_t row = tm * 64 + wm * 32;
    Stage<T>::load(reinterpret_cast<const T*>(p.a.gh) + row * p.N + unit0, p.N, p.M - row, p.N - unit0, next);
  };
  if (walker < tiles_m) {
    fetch_rows(walker, x);
    if (walker + walkers < tiles_m) fetch_rows(walker + walkers, x + steps * N::kX);
    if constexpr (KIND == kGates) fetch_gradients(walker);
  }
  const Stage<T> stage{out + wave * (N::kOut / 4)};
  const f32x4* bias = reinterpret_cast<const f32x4*>(shared + wn * 32 + (lane >> 5) * 4);
  float sum_a[16] = {}, sum_b[16] = {};
  // What a wave whose units are all there issues in a turn after its rows' loads,
  // which two turns later are complete when so much is left: stores, the
  // gradients' loads, and one of the rows' in between.
  constexpr int kAfter = 2 * (KIND == kGates ? (kPairs<T> ? 5 : 3) * kTurns : kTurns) + 1;
  const bool counted = unit0 + 32 <= p.N;
  int turn = 0;
  for (int64_t tm = walker; tm < tiles_m; tm += walkers) {
    if (counted && tm != walker && tm + walkers < tiles_m)
      wait_loads<kAfter>();
    else
      wait_loads<0>();
    const int ahead = turn == 0 ? 2 : turn - 1;
    if (tm + 2 * walkers < tiles_m) fetch_rows(tm + 2 * walkers, x + ahead * steps * N::kX);
    f32x16 acc[1][2] = {};
    for (int s = 0; s < steps; ++s)
      multiply_step<T, KIND, 1, 2>(x + (turn * steps + s) * N::kX, w + s * N::kW, acc, [](int) {});
    turn = turn == 2 ? 0 : turn + 1;
    const int64_t row = tm * 64 + wm * 32;
    if constexpr (KIND == kForward)
      forward_fragment<T, ACT>(p, stage, bias, acc[0][0], acc[0][1], row, unit0);
    else
      gates_fragment<T, ACT>(
          p, stage, bias, acc[0][0], acc[0][1], row, unit0, next,
          [&](int q, bool in, const float(&da)[16], const float(&db)[16]) {
#pragma unroll
            for (int r = q * 4; r < q * 4 + 4; ++r) {
              sum_a[r] += in ? da[r] : 0.0f;
              sum_b[r] += in ? db[r] : 0.0f;
            }
          },
          [&] {
            if (tm + walkers < tiles_m) fetch_gradients(tm + walkers);
          });
  }
  if constexpr (KIND == kGates) {
    if (!p.bias) return;
    wait_loads<0>();
    store_bias_sums(p, walker, tn, sum_a, sum_b, lds + wave * kStage, shared);
  }
}

constexpr int kJoin = 1024;

// Joins the shares of a tile, each of four groups of threads every fourth one,
// in order.  A workgroup has one fragment of each of the four waves.
template <class T, int KIND, int FM, int FN>
__global__ __launch_bounds__(kJoin) void glu_join_kernel(Product<T> p) {
  __shared__ f32x4 lds[3][4][kNT];
  __shared__ __align__(16) char staged[4 * kStage];
  const int64_t tile = blockIdx.x;
  const int z = (int)(tile / (p.tiles_n * p.tiles_m));
  if (!p.out[z]) return;
  const int j = blockIdx.y % FN, i = blockIdx.y / FN;
  const int thread = threadIdx.x & (kNT - 1), group = threadIdx.x / kNT;
  constexpr int64_t next = (int64_t)kNT * (FM * FN * 16);  // from one share to the next
  const float* in = p.part + tile * p.splits * next + (i * FN + j) * (kNT * 16) + thread * 4;
  f32x4 v[4] = {};
#pragma unroll 4
  for (int s = group; s < p.splits; s += 4)
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] += *reinterpret_cast<const f32x4*>(in + s * next + q * (kNT * 4));
  if (group)
#pragma unroll
    for (int q = 0; q < 4; ++q) lds[group - 1][q][thread] = v[q];
  __syncthreads();
  if (group) return;
  float u[16];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    for (int g = 0; g < 3; ++g) v[q] += lds[g][q][thread];
#pragma unroll
    for (int r = 0; r < 4; ++r) u[q * 4 + r] = kScaled<T> ? v[q][r] * (1.0f / kPartScale) : v[q][r];
  }
  const int64_t tn = tile % p.tiles_n, tm = tile / p.tiles_n - z * p.tiles_m;
  const int wave = __builtin_amdgcn_readfirstlane(thread >> 6), wm = wave >> 1, wn = wave & 1;
  const int64_t row = tm * 64 * FM + wm * FM * 32 + i * 32, col = tn * 64 * FN + wn * FN * 32 + j * 32;
  const Stage<T> stage{staged + wave * kStage};
  stage.put(u);
  stage.store(p.out[z] + row * p.pitch_out + col, p.pitch_out, p.M - row, p.N - col);
}

// Bias gradients from the tiles' sums, in float64.  16 units a workgroup.
template <class T>
__global__ __launch_bounds__(kJoin) void glu_bias_kernel(Product<T> p) {
  __shared__ double lds[kJoin / 16][17];
  const int c = threadIdx.x & 15, r = threadIdx.x >> 4;
  const int64_t unit = (int64_t)blockIdx.x * 16 + c;
  T* out = reinterpret_cast<T*>(blockIdx.y == 0 ? p.a.gbg : p.a.gbu);
  if (!out) return;
  double s = 0.0;
  if (unit < p.N) {
#pragma unroll 4
    for (int64_t t = r; t < p.tiles_m; t += kJoin / 16) s += (double)p.bias[(t * 2 + blockIdx.y) * p.pitch + unit];
  }
  lds[r][c] = s;
  __syncthreads();
  for (int d = kJoin / 32; d > 0; d /= 2) {
    if (r < d) lds[r][c] += lds[r + d][c];
    __syncthreads();
  }
  if (r == 0 && unit < p.N) out[unit] = (T)(float)lds[0][c];
}

// ---------------------------------------------------------------- few rows
__device__ __forceinline__ f32x4 multiply16(const Fragment<f16>& a, const Fragment<f16>& b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a.v), __builtin_bit_cast(f16x8, b.v), c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 multiply16(const Fragment<bf16>& a, const Fragment<bf16>& b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a.v), __builtin_bit_cast(bf16x8, b.v), c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 multiply16(const Fragment<float>& a, const Fragment<float>& b, f32x4 c) {
  const f32x4 u = __builtin_bit_cast(f32x4, a.v), v = __builtin_bit_cast(f32x4, b.v);
#pragma unroll
  for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(u[j], v[j], c, 0, 0, 0);
  return c;
}

// Up to 16 RB rows: bound by the weights' one way from memory.  A workgroup has
// 16 hidden units of both projections, its eight waves every eighth step of the
// sum each, whose operands go straight to the registers; everything is on its
// way at once.  (1 x 1024 to 2816, bfloat16, 11.5 MB: 9.8 us in tiles.)
constexpr int kFewThreads = 512;
template <class T, int RB>
__global__ __launch_bounds__(kFewThreads) void glu_few_kernel(Product<T> p) {
  constexpr int kWaves = kFewThreads / 64, kAhead = RB == 1 ? 4 : 2;
  __shared__ f32x4 lds[kWaves][2][RB][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, line = lane & 15, chunk = lane >> 4;
  const int64_t unit0 = (int64_t)blockIdx.x * 16, unit = unit0 + line < p.N ? unit0 + line : p.N - 1;
  const T* w[2] = {p.B[0] + unit * p.pitchB, p.B[1] + unit * p.pitchB};
  const auto fetch = [&](const T* at, int64_t k) {
    Fragment<T> f;
    if (k + kPer<T> <= p.K) {
      __builtin_memcpy(&f.v, at + k, 16);
    } else {  // zeros behind the end
      Vec<T, kPer<T>> v = {};
#pragma unroll
      for (int j = 0; j < kPer<T> - 1; ++j)
        if (k + j < p.K) v.v[j] = at[k + j];
      __builtin_memcpy(&f.v, &v, 16);
    }
    return f;
  };
  f32x4 acc[2][RB];
#pragma unroll
  for (int z = 0; z < 2; ++z)
#pragma unroll
    for (int i = 0; i < RB; ++i) acc[z][i] = f32x4{};
  const int64_t steps = (p.K + kStep<T> - 1) / kStep<T>;
  for (int64_t s0 = wave; s0 < steps; s0 += kWaves * kAhead) {
    Fragment<T> a[kAhead][2], b[kAhead][RB];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int64_t k = (s0 + u * kWaves) * kStep<T> + chunk * kPer<T>;
#pragma unroll
      for (int z = 0; z < 2; ++z) a[u][z] = fetch(w[z], k);
#pragma unroll
      for (int i = 0; i < RB; ++i) {
        const int64_t row = i * 16 + line;
        b[u][i] = fetch(p.A + (row < p.M ? row : p.M - 1) * p.pitchA, k);
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
#pragma unroll
      for (int z = 0; z < 2; ++z)
#pragma unroll
        for (int i = 0; i < RB; ++i) acc[z][i] = multiply16(a[u][z], b[u][i], acc[z][i]);
  }
#pragma unroll
  for (int z = 0; z < 2; ++z)
#pragma unroll
    for (int i = 0; i < RB; ++i) lds[wave][z][i][lane] = acc[z][i];
  __syncthreads();
  // a thread for every result: unit and row within the 16 x 16 block
  const float* all = reinterpret_cast<const float*>(lds);
  for (int id = threadIdx.x; id < RB * 256; id += kFewThreads) {
    const int i = id >> 8, u = id & 15, r = id >> 4 & 15;
    const int64_t row = i * 16 + r, at = unit0 + u;
    if (row >= p.M || at >= p.N) continue;
    float v[2];
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      const void* bias = z ? p.a.bu : p.a.bg;
      float s = 0.0f;
#pragma unroll
      for (int g = 0; g < kWaves; ++g) s += all[(((g * 2 + z) * RB + i) * 64 + (u >> 2) * 16 + r) * 4 + (u & 3)];
      v[z] = s + (bias ? (float)reinterpret_cast<const T*>(bias)[at] : 0.0f);
    }
    float y = v[0];
    if (p.a.act == kActRelu) y = act_value<kActRelu>(y);
    if (p.a.act == kActSilu) y = act_value<kActSilu>(y);
    if (p.a.act == kActGelu) y = act_value<kActGelu>(y);
    reinterpret_cast<T*>(p.a.h)[row * p.N + at] = (T)(y * v[1]);
  }
}

// --------------------------------------------------------------- packing
// x and the weights with rows of `wide` elements, zeros at the end of each.
template <class T>
__global__ __launch_bounds__(kNT) void glu_pack_kernel(GluArgs a, T* x, T* wg, T* wu, int64_t wide) {
  const int64_t chunks = wide / kPer<T>, all = (a.rows + 2 * a.hidden) * chunks;
  for (int64_t id = (int64_t)blockIdx.x * kNT + threadIdx.x; id < all; id += (int64_t)gridDim.x * kNT) {
    int64_t row = id / chunks;
    const int64_t k = (id - row * chunks) * kPer<T>;
    const T* in = reinterpret_cast<const T*>(a.x);
    T* out = x;
    if (row >= a.rows) {
      row -= a.rows;
      const bool up = row >= a.hidden;
      if (up) row -= a.hidden;
      in = reinterpret_cast<const T*>(up ? a.wu : a.wg);
      out = up ? wu : wg;
    }
    in += row * a.channels + k;
    Vec<T, kPer<T>> v = {};
    if (k + kPer<T> <= a.channels) {
      load_vec(in, v);
    } else {
#pragma unroll
      for (int j = 0; j < kPer<T> - 1; ++j)
        if (k + j < a.channels) v.v[j] = in[j];
    }
    store_vec(out + row * wide + k, v);
  }
}

// ---------------------------------------------------------------- launches
template <class T>
bool is_aligned(const Product<T>& p) {
  const auto ok = [](const void* q, int64_t pitch) {
    return reinterpret_cast<uintptr_t>(q) % 16 == 0 && pitch % kPer<T> == 0;
  };
  return ok(p.A, p.pitchA) && ok(p.B[0], p.pitchB) && ok(p.B[1], p.pitchB);
}

template <class T, int KIND, int FM>
hipError_t launch_tiles(Product<T> p, hipStream_t stream) {
  const int both = KIND == kWeight ? 2 : 1;
  const int64_t tiles = p.tiles_m * p.tiles_n * both;
  const dim3 grid((unsigned)(tiles * p.splits)), block(kNT);
  const auto launch = [&](auto act) {
    if (is_aligned(p))
      hipLaunchKernelGGL((glu_kernel<T, KIND, FM, 2, true, act.value>), grid, block, 0, stream, p);
    else
      hipLaunchKernelGGL((glu_kernel<T, KIND, FM, 2, false, act.value>), grid, block, 0, stream, p);
  };
  using std::integral_constant;
  if (!is_dual(KIND) || p.a.act == kActNone)
    launch(integral_constant<int, kActNone>{});
  else if constexpr (is_dual(KIND)) {
    // (chosen in the kernel, the activation costs it more registers than there are)
    if (p.a.act == kActRelu)
      launch(integral_constant<int, kActRelu>{});
    else if (p.a.act == kActSilu)
      launch(integral_constant<int, kActSilu>{});
    else
      launch(integral_constant<int, kActGelu>{});
  }
  if constexpr (!is_dual(KIND)) {
    if (p.splits > 1)
      hipLaunchKernelGGL((glu_join_kernel<T, KIND, FM, 2>), dim3((unsigned)tiles, FM * 2), dim3(kJoin), 0, stream, p);
  }
  return hipGetLastError();
}
template <class T, int KIND>
hipError_t launch_product(Product<T> p, const GluShare& s, hipStream_t stream) {
  p.splits = s.splits;
  p.tiles_m = s.tiles_m;
  p.tiles_n = s.tiles_n;
  return s.FM == 4 ? launch_tiles<T, KIND, 4>(p, stream) : launch_tiles<T, KIND, 1>(p, stream);
}

// Both projections; `sums`: partial rows of the bias gradients.
template <class T, int KIND>
hipError_t launch_projections(Product<T> p, const GluPlan& plan, hipStream_t stream, int64_t* sums = nullptr) {
  if (sums) *sums = plan.gates.tiles_m;
  if (!plan.walkers || !is_aligned(p)) return launch_product<T, KIND>(p, plan.gates, stream);
  if (sums) *sums = plan.walkers;
  p.tiles_n = plan.gates.tiles_n;
  const int steps = (int)((p.K + kStep<T> - 1) / kStep<T>);
  const dim3 grid((unsigned)(plan.walkers * p.tiles_n)), block(kNT);
  const auto launch = [&](auto act) {
    hipLaunchKernelGGL((glu_narrow_kernel<T, KIND, act.value>), grid, block, Narrow<T>::bytes(steps), stream, p,
                       (int)plan.walkers, steps);
    return hipGetLastError();
  };
  using std::integral_constant;
  if (p.a.act == kActRelu) return launch(integral_constant<int, kActRelu>{});
  if (p.a.act == kActSilu) return launch(integral_constant<int, kActSilu>{});
  if (p.a.act == kActGelu) return launch(integral_constant<int, kActGelu>{});
  return launch(integral_constant<int, kActNone>{});
}

// The projections' product, of packed operands if there are any.
template <class T>
Product<T> projections(const GluArgs& a, const GluPlan& plan, hipStream_t stream) {
  Product<T> p{};
  p.A = reinterpret_cast<const T*>(a.x);
  p.pitchA = p.pitchB = p.K = a.channels;
  p.B[0] = reinterpret_cast<const T*>(a.wg);
  p.B[1] = reinterpret_cast<const T*>(a.wu);
  p.M = a.rows;
  p.N = a.hidden;
  p.parts = 1;
  p.a = a;
  if (plan.packed) {
    char* ws = reinterpret_cast<char*>(a.ws);
    T *x = reinterpret_cast<T*>(ws + plan.at_x), *wg = reinterpret_cast<T*>(ws + plan.at_wg),
      *wu = reinterpret_cast<T*>(ws + plan.at_wu);
    const int64_t blocks = ((a.rows + 2 * a.hidden) * (plan.wide / kPer<T>) + kNT - 1) / kNT;
    hipLaunchKernelGGL(glu_pack_kernel<T>, dim3((unsigned)(blocks < 16384 ? blocks : 16384)), dim3(kNT), 0, stream, a, x, wg,
                       wu, plan.wide);
    p.A = x;
    p.B[0] = wg;
    p.B[1] = wu;
    p.pitchA = p.pitchB = p.K = plan.wide;
  }
  return p;
}

}  // namespace

template <class T>
hipError_t launch_glu_fwd(const GluArgs& a, hipStream_t stream) {
  const GluPlan plan = glu_plan(a.rows, a.channels, a.hidden, sizeof(T), false);
  const Product<T> p = projections<T>(a, plan, stream);
  if (a.rows > kGluFew) return launch_projections<T, kForward>(p, plan, stream);
  const dim3 grid((unsigned)((a.hidden + 15) / 16)), block(kFewThreads);
  if (a.rows <= 16)
    hipLaunchKernelGGL((glu_few_kernel<T, 1>), grid, block, 0, stream, p);
  else if (a.rows <= 32)
    hipLaunchKernelGGL((glu_few_kernel<T, 2>), grid, block, 0, stream, p);
  else
    hipLaunchKernelGGL((glu_few_kernel<T, 4>), grid, block, 0, stream, p);
  return hipGetLastError();
}

template <class T>
hipError_t launch_glu_bwd(const GluArgs& a, hipStream_t stream) {
  const GluPlan plan = glu_plan(a.rows, a.channels, a.hidden, sizeof(T), true);
  char* ws = reinterpret_cast<char*>(a.ws);
  Product<T> p = projections<T>(a, plan, stream);
  const T* x = p.A;
  p.pitch = plan.pitch;
  p.dab = reinterpret_cast<T*>(ws + plan.at_dab);
  p.bias = a.gbg || a.gbu ? reinterpret_cast<float*>(ws + plan.at_bias) : nullptr;
  p.part = reinterpret_cast<float*>(ws + plan.at_part);
  hipError_t st = launch_projections<T, kGates>(p, plan, stream, &p.tiles_m);
  if (st != hipSuccess) return st;
  if (p.bias) {
    hipLaunchKernelGGL(glu_bias_kernel<T>, dim3((unsigned)((a.hidden + 15) / 16), 2), dim3(kJoin), 0, stream, p);
  }
  p.A = p.dab;
  p.pitchA = (plan.pairs ? 4 : 2) * plan.pitch;
  p.stepA = plan.pitch;
  if (a.gx) {
    p.N = a.channels;
    p.K = a.hidden;
    p.parts = plan.pairs ? 4 : 2;
    p.out[0] = reinterpret_cast<T*>(a.gx);
    p.pitch_out = a.channels;
    st = launch_product<T, kInput>(p, plan.input, stream);
    if (st != hipSuccess) return st;
  }
  if (a.gwg || a.gwu) {
    p.M = a.hidden;
    p.N = a.channels;
    p.K = a.rows;
    p.parts = plan.pairs ? 2 : 1;
    p.B[0] = p.B[1] = x;
    p.out[0] = reinterpret_cast<T*>(a.gwg);
    p.out[1] = reinterpret_cast<T*>(a.gwu);
    p.pitch_out = a.channels;
    st = launch_product<T, kWeight>(p, plan.weight, stream);
  }
  return st != hipSuccess ? st : hipGetLastError();
}

}  // namespace ecc
