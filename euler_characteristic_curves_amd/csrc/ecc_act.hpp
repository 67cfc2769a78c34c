// Element types, activations and their slopes for the training operators.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ecc {

typedef _Float16 f16;
typedef __bf16 bf16;

// V elements from memory aligned to one element only: the target's global
// loads and stores take any alignment, so one 16-byte access serves rows that
// are not a multiple of 16 bytes too.
template <class T, int V>
struct Vec {
  T v[V];
};
template <class T, int V>
__device__ __forceinline__ void load_vec(const T* p, Vec<T, V>& r) {
  __builtin_memcpy(&r, p, sizeof(T) * V);
}
template <class T, int V>
__device__ __forceinline__ void store_vec(T* p, const Vec<T, V>& r) {
  __builtin_memcpy(p, &r, sizeof(T) * V);
}

// One parameter as float32; null stands for `dflt`.
__device__ __forceinline__ float load_param(const void* p, int pdtype, int64_t i, float dflt) {
  if (!p) return dflt;
  if (pdtype == 0) return reinterpret_cast<const float*>(p)[i];
  if (pdtype == 1) return (float)reinterpret_cast<const f16*>(p)[i];
  return (float)reinterpret_cast<const bf16*>(p)[i];
}
__device__ __forceinline__ void store_param(void* p, int pdtype, int64_t i, float v) {
  if (pdtype == 0)
    reinterpret_cast<float*>(p)[i] = v;
  else if (pdtype == 1)
    reinterpret_cast<f16*>(p)[i] = (f16)v;
  else
    reinterpret_cast<bf16*>(p)[i] = (bf16)v;
}

constexpr int kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3;

// Upper tail of the normal distribution at z = |u|, and e = exp(-z^2/2).  The
// tail is e * t * p(t) with t = 1 / (1 + 0.3 z): t p(t) is erfcx(z / sqrt 2) /
// 2, a polynomial in t fitted to it over z in [0, 14] (relative error 1.5e-7),
// so it keeps its relative accuracy, where 1 + erf(u / sqrt 2) cancels.  The
// exponent's rounding adds z^2 2^-25 relative, which is below 2^-25 of 1 after
// e multiplies it.
__device__ __forceinline__ float normal_tail(float u, float& e) {
  e = __builtin_amdgcn_exp2f(u * (-0.721347520f * u));
  const float t = __builtin_amdgcn_rcpf(fmaf(0.3f, fabsf(u), 1.0f));
  float p = 0.0356748769f;
  p = fmaf(p, t, -0.1572034993f);
  p = fmaf(p, t, 0.2063541957f);
  p = fmaf(p, t, -0.0536842455f);
  p = fmaf(p, t, 0.1285619242f);
  p = fmaf(p, t, 0.0999134088f);
  p = fmaf(p, t, 0.1207539682f);
  p = fmaf(p, t, 0.1196292981f);
  return e * (t * p);
}

// 1 / (1 + exp(-u)).  The product that scales the exponent is off by half a
// step of it, so the logistic function by u (1 - s) s 2^-24 at most, below 2^-25
// wherever it is multiplied by u; exp2 and the reciprocal add a step each.
// Beyond the exponent's range they give infinity and 0, or 0 and 1.
__device__ __forceinline__ float logistic(float u) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269502f * u));
}

// Infinite arguments, which finite features and parameters can reach, have the
// values and slopes that the activations tend to: a factor of the tail or of
// the logistic function, which are 0 there, is kept finite.
constexpr float kHuge = 3.40282347e38f;

template <int ACT>
__device__ __forceinline__ float act_value(float u) {
  if constexpr (ACT == kActRelu) return u <= 0.0f ? 0.0f : u;
  if constexpr (ACT == kActSilu) return fmaxf(u, -kHuge) * logistic(u);
  if constexpr (ACT == kActGelu) {
    float e;
    return fmaf(-fminf(fabsf(u), kHuge), normal_tail(u, e), fmaxf(u, 0.0f));
  }
  return u;
}

// Slope; y receives the value.
template <int ACT>
__device__ __forceinline__ float act_slope(float u, float& y) {
  if constexpr (ACT == kActRelu) {
    y = u <= 0.0f ? 0.0f : u;
    return u > 0.0f ? 1.0f : (u <= 0.0f ? 0.0f : u);
  }
  if constexpr (ACT == kActSilu) {
    const float s = logistic(u);
    y = __builtin_amdgcn_fmed3f(u, -kHuge, kHuge) * s;
    return fmaf(y, 1.0f - s, s);
  }
  if constexpr (ACT == kActGelu) {
    // both from the tail q: y = max(u, 0) - |u| q, y' = q - |u| e / sqrt(2 pi), from 1 where u > 0
    float e;
    const float q = normal_tail(u, e), z = fminf(fabsf(u), kHuge);
    y = fmaf(-z, q, fmaxf(u, 0.0f));
    const float w = fmaf(-0.398942280f * z, e, q);
    return u > 0.0f ? 1.0f - w : w;
  }
  y = u;
  return 1.0f;
}

}  // namespace ecc
