// Argument checks and errors that the C-ABI layers of the training operators share.
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdio.h>

#include "../../include/ecc.h"
#include "../../include/ecc_train.h"
#include "ecc_train_internal.hpp"

namespace ecc {

inline int fail(int status, const char* fmt, long long a = 0, long long b = 0) {
  char msg[256];
  snprintf(msg, sizeof(msg), fmt, a, b);
  set_error(msg);
  return status;
}

inline int hip_status(hipError_t e) {
  if (e == hipSuccess) return ECC_OK;
  char msg[256];
  snprintf(msg, sizeof(msg), "HIP error: %s", hipGetErrorString(e));
  set_error(msg);
  return ECC_E_HIP;
}

inline bool is_dtype(int d) { return d == ECC_T_F32 || d == ECC_T_F16 || d == ECC_T_BF16; }

inline int check_workspace(const void* ws, size_t ws_bytes, size_t need) {
  if (!ws) return fail(ECC_E_WORKSPACE, "workspace is NULL");
  if (reinterpret_cast<uintptr_t>(ws) % 256) return fail(ECC_E_WORKSPACE, "workspace is not 256-byte aligned");
  if (ws_bytes < need)
    return fail(ECC_E_WORKSPACE, "workspace has %lld bytes, needs %lld", (long long)ws_bytes, (long long)need);
  return ECC_OK;
}

inline int check_eps(float eps) {
  if (!(eps >= 0.0f) || !isfinite(eps)) return fail(ECC_E_VALUE, "eps must be finite and >= 0");
  return ECC_OK;
}

}  // namespace ecc
