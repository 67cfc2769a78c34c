// C ABI of the training operators (include/ecc_train.h): argument validation,
// error reporting, dispatch.

#include "../../include/ecc_train.h"

#include <hip/hip_runtime.h>
#include <math.h>

#include "../../include/ecc.h"
#include "ecc_act.hpp"
#include "ecc_check.hpp"
#include "ecc_internal.hpp"
#include "ecc_train_internal.hpp"

namespace {

using ecc::check_eps;
using ecc::check_workspace;
using ecc::fail;
using ecc::hip_status;
using ecc::is_dtype;

int check_norm_shape(int64_t B, int64_t S, int64_t C, int64_t G) {
  if (B < 1 || S < 1 || C < 1)
    return fail(ECC_E_SHAPE, "batch, voxels and channels must be >= 1 (got voxels=%lld channels=%lld)", S, C);
  if (B > ECC_MAX_NORM_BATCH) return fail(ECC_E_SHAPE, "batch=%lld exceeds %lld", B, ECC_MAX_NORM_BATCH);
  if (C > ECC_MAX_CHANNELS) return fail(ECC_E_SHAPE, "channels=%lld exceeds %lld", C, ECC_MAX_CHANNELS);
  if (S > ECC_MAX_VOXELS / C || B > ECC_MAX_VOXELS / (S * C)) return fail(ECC_E_SHAPE, "more than 2^40 elements");
  if (G < 1 || C % G) return fail(ECC_E_GROUPS, "groups=%lld does not divide channels=%lld", G, C);
  return ECC_OK;
}

// Checks shared by the four norm calls, and the part of the arguments they share.
int check_norm(ecc::NormArgs& a, const void* x, int dtype, int64_t B, int64_t S, int64_t C, int64_t G,
               const void* weight, const void* bias, int pdtype, int act, const float* stats, void* ws,
               size_t ws_bytes) {
  ecc::set_error("");
  if (!x) return fail(ECC_E_NULL, "x is NULL");
  if (!stats) return fail(ECC_E_NULL, "stats is NULL");
  if (!is_dtype(dtype)) return fail(ECC_E_DTYPE, "dtype %lld is not one of ECC_T_*", dtype);
  if (pdtype != ECC_T_F32 && pdtype != dtype)
    return fail(ECC_E_DTYPE, "pdtype %lld is neither ECC_T_F32 nor the dtype of x (%lld)", pdtype, dtype);
  if (act < ECC_ACT_NONE || act > ECC_ACT_GELU) return fail(ECC_E_ACT, "act %lld is not one of ECC_ACT_*", act);
  int st = check_norm_shape(B, S, C, G);
  if (st != ECC_OK) return st;
  st = check_workspace(ws, ws_bytes, ecc::norm_workspace_bytes(B, S, C, G));
  if (st != ECC_OK) return st;
  a = ecc::NormArgs{};
  a.x = x;
  a.B = B;
  a.S = S;
  a.C = C;
  a.G = G;
  a.weight = weight;
  a.bias = bias;
  a.pdtype = pdtype;
  a.act = act;
  a.stats = const_cast<float*>(stats);
  a.ws = ws;
  return ECC_OK;
}

int run_fwd(const ecc::NormArgs& a, int dtype, void* stream) {
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (dtype == ECC_T_F32) return hip_status(ecc::norm_launch_fwd<float>(a, s));
  if (dtype == ECC_T_F16) return hip_status(ecc::norm_launch_fwd<ecc::f16>(a, s));
  return hip_status(ecc::norm_launch_fwd<ecc::bf16>(a, s));
}

int run_bwd(const ecc::NormArgs& a, int dtype, void* stream) {
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (dtype == ECC_T_F32) return hip_status(ecc::norm_launch_bwd<float>(a, s));
  if (dtype == ECC_T_F16) return hip_status(ecc::norm_launch_bwd<ecc::f16>(a, s));
  return hip_status(ecc::norm_launch_bwd<ecc::bf16>(a, s));
}

int check_matrix(int64_t B, int64_t rows, int64_t cols) {
  if (B < 1 || rows < 1 || cols < 1)
    return fail(ECC_E_SHAPE, "batch, rows and cols must be >= 1 (got rows=%lld cols=%lld)", rows, cols);
  if (B > ECC_MAX_NORM_BATCH) return fail(ECC_E_SHAPE, "batch=%lld exceeds %lld", B, ECC_MAX_NORM_BATCH);
  if (rows > ECC_MAX_MATRIX || cols > ECC_MAX_MATRIX)
    return fail(ECC_E_SHAPE, "a matrix of %lld x %lld exceeds the limit per side", rows, cols);
  if (B > ECC_MAX_VOXELS / (rows * cols)) return fail(ECC_E_SHAPE, "more than 2^40 elements");
  return ECC_OK;
}

// Checks shared by the two matrix calls, once sizes, types and coefficients are in o.
int check_orth(ecc::OrthArgs& o, size_t ws_bytes) {
  if (!is_dtype(o.gdtype) || !is_dtype(o.odtype))
    return fail(ECC_E_DTYPE, "dtypes %lld, %lld are not both of ECC_T_*", o.gdtype, o.odtype);
  int st = check_matrix(o.batch, o.rows, o.cols);
  if (st != ECC_OK) return st;
  if (o.steps < 1 || o.steps > ECC_MAX_NS_STEPS)
    return fail(ECC_E_VALUE, "steps=%lld outside [1, %lld]", o.steps, ECC_MAX_NS_STEPS);
  st = check_eps(o.eps);
  if (st != ECC_OK) return st;
  if (!isfinite(o.a) || !isfinite(o.b) || !isfinite(o.c)) return fail(ECC_E_VALUE, "coefficients must be finite");
  if (!ecc::orth_bounds(o))
    return fail(ECC_E_VALUE, "under these coefficients singular values in [0, 1] leave [-16, 16]");
  return check_workspace(o.ws, ws_bytes, ecc::orth_workspace_bytes(o.batch, o.rows, o.cols));
}

}  // namespace

namespace ecc {

bool orth_bounds(OrthArgs& o) {
  // 256 samples of the attained range; 2 % covers what lies between them
  constexpr int kSamples = 256;
  double r = 1.0, pmax = 0.0, gram = 0.0, cap = 1.0, all = 1.0;
  o.amplify = 1.0;
  for (int k = 0; k < o.steps; ++k) {
    double f = 0.0, q = 0.0;
    for (int i = 0; i <= kSamples; ++i) {
      const double x = r * i / kSamples, p = o.a + x * x * (o.b + x * x * o.c);
      f = fmax(f, fabs(p * x));
      q = fmax(q, fabs(p));
    }
    gram = fmax(gram, r * r);
    pmax = fmax(pmax, 1.02 * q);
    all *= 1.02 * q;
    if (k + 1 < o.steps) o.amplify *= fmax(1.0, q * q);
    r = 1.02 * f;
    cap = fmax(cap, r);
    if (!(cap <= 16.0) || !(pmax <= 4096.0)) return false;
  }
  int e;
  frexp(gram, &e);
  o.sa = ldexpf(1.0f, 14 - e);
  frexp(fmax(pmax, 1e-30), &e);
  o.sp = ldexpf(1.0f, 14 - e);
  // (beyond 2^40 the entries are too unlike for a pair; kMaxAmplify is passed long before)
  frexp(fmin(fmax(all, 1e-30), 1e12), &e);
  o.sq = ldexpf(1.0f, 14 - e);
  o.growth = (float)pmax;
  o.cap = (float)cap;
  return true;
}

}  // namespace ecc

extern "C" {

size_t ecc_norm_workspace_bytes(int64_t batch, int64_t voxels, int64_t channels, int64_t groups) {
  if (check_norm_shape(batch, voxels, channels, groups) != ECC_OK) return 0;
  return ecc::norm_workspace_bytes(batch, voxels, channels, groups);
}

int ecc_norm_fwd(const void* x, int dtype, int64_t batch, int64_t voxels, int64_t channels, int64_t groups,
                 const void* weight, const void* bias, int pdtype, int act, float eps, void* y, float* stats,
                 void* ws, size_t ws_bytes, void* stream) {
  ecc::NormArgs a;
  int st = check_norm(a, x, dtype, batch, voxels, channels, groups, weight, bias, pdtype, act, stats, ws, ws_bytes);
  if (st != ECC_OK) return st;
  if (!y) return fail(ECC_E_NULL, "y is NULL");
  st = check_eps(eps);
  if (st != ECC_OK) return st;
  a.eps = eps;
  a.y = y;
  return run_fwd(a, dtype, stream);
}

int ecc_norm_bwd(const void* x, int dtype, int64_t batch, int64_t voxels, int64_t channels, int64_t groups,
                 const void* weight, const void* bias, int pdtype, int act, const float* stats, const void* grad_y,
                 void* grad_x, void* grad_weight, void* grad_bias, void* ws, size_t ws_bytes, void* stream) {
  ecc::NormArgs a;
  const int st =
      check_norm(a, x, dtype, batch, voxels, channels, groups, weight, bias, pdtype, act, stats, ws, ws_bytes);
  if (st != ECC_OK) return st;
  if (!grad_y) return fail(ECC_E_NULL, "grad_y is NULL");
  if (!grad_x && !grad_weight && !grad_bias) return fail(ECC_E_NULL, "every gradient is NULL");
  a.gy = grad_y;
  a.gx = grad_x;
  a.gw = grad_weight;
  a.gb = grad_bias;
  return run_bwd(a, dtype, stream);
}

int ecc_norm_readout_fwd(const void* x, int dtype, int64_t batch, int64_t voxels, int64_t channels, int64_t groups,
                         const void* weight, const void* bias, const void* readout, const void* offset, int pdtype,
                         int act, float eps, float* field, float* stats, void* ws, size_t ws_bytes, void* stream) {
  ecc::NormArgs a;
  int st = check_norm(a, x, dtype, batch, voxels, channels, groups, weight, bias, pdtype, act, stats, ws, ws_bytes);
  if (st != ECC_OK) return st;
  if (channels > ECC_MAX_READOUT_CHANNELS)
    return fail(ECC_E_SHAPE, "channels=%lld exceeds %lld", channels, ECC_MAX_READOUT_CHANNELS);
  if (!readout) return fail(ECC_E_NULL, "readout is NULL");
  if (!field) return fail(ECC_E_NULL, "field is NULL");
  st = check_eps(eps);
  if (st != ECC_OK) return st;
  a.eps = eps;
  a.readout = readout;
  a.offset = offset;
  a.field = field;
  return run_fwd(a, dtype, stream);
}

int ecc_norm_readout_bwd(const void* x, int dtype, int64_t batch, int64_t voxels, int64_t channels, int64_t groups,
                         const void* weight, const void* bias, const void* readout, int pdtype, int act,
                         const float* stats, const float* grad_field, void* grad_x, void* grad_weight,
                         void* grad_bias, void* grad_readout, void* grad_offset, void* ws, size_t ws_bytes,
                         void* stream) {
  ecc::NormArgs a;
  const int st =
      check_norm(a, x, dtype, batch, voxels, channels, groups, weight, bias, pdtype, act, stats, ws, ws_bytes);
  if (st != ECC_OK) return st;
  if (channels > ECC_MAX_READOUT_CHANNELS)
    return fail(ECC_E_SHAPE, "channels=%lld exceeds %lld", channels, ECC_MAX_READOUT_CHANNELS);
  if (!readout) return fail(ECC_E_NULL, "readout is NULL");
  if (!grad_field) return fail(ECC_E_NULL, "grad_field is NULL");
  if (!grad_x && !grad_weight && !grad_bias && !grad_readout && !grad_offset)
    return fail(ECC_E_NULL, "every gradient is NULL");
  a.readout = readout;
  a.gy = grad_field;
  a.gx = grad_x;
  a.gw = grad_weight;
  a.gb = grad_bias;
  a.gr = grad_readout;
  a.go = grad_offset;
  return run_bwd(a, dtype, stream);
}

size_t ecc_orth_workspace_bytes(int64_t batch, int64_t rows, int64_t cols) {
  if (check_matrix(batch, rows, cols) != ECC_OK) return 0;
  return ecc::orth_workspace_bytes(batch, rows, cols);
}

int ecc_orthogonalize(const void* g, int dtype, int64_t batch, int64_t rows, int64_t cols, int32_t steps, float eps,
                      float a, float b, float c, void* out, void* ws, size_t ws_bytes, void* stream) {
  ecc::set_error("");
  if (!g) return fail(ECC_E_NULL, "g is NULL");
  if (!out) return fail(ECC_E_NULL, "out is NULL");
  ecc::OrthArgs o{};
  o.g = g;
  o.gdtype = o.odtype = dtype;
  o.batch = batch;
  o.rows = rows;
  o.cols = cols;
  o.out = out;
  o.steps = steps;
  o.eps = eps;
  o.a = a;
  o.b = b;
  o.c = c;
  o.ws = ws;
  const int st = check_orth(o, ws_bytes);
  if (st != ECC_OK) return st;
  return hip_status(ecc::launch_orth(o, reinterpret_cast<hipStream_t>(stream)));
}

int ecc_muon_step(void* param, int pdtype, const void* grad, int gdtype, float* buffer, int64_t batch, int64_t rows,
                  int64_t cols, double lr, double momentum, int nesterov, double weight_decay, double scale,
                  int32_t steps, float eps, float a, float b, float c, void* ws, size_t ws_bytes, void* stream) {
  ecc::set_error("");
  if (!param) return fail(ECC_E_NULL, "param is NULL");
  if (!grad) return fail(ECC_E_NULL, "grad is NULL");
  if (!buffer) return fail(ECC_E_NULL, "buffer is NULL");
  if (!isfinite(lr) || !isfinite(momentum) || !isfinite(weight_decay) || !isfinite(scale))
    return fail(ECC_E_VALUE, "lr, momentum, weight_decay and scale must be finite");
  ecc::OrthArgs o{};
  o.g = grad;
  o.gdtype = gdtype;
  o.odtype = pdtype;
  o.batch = batch;
  o.rows = rows;
  o.cols = cols;
  o.out = param;
  o.buffer = buffer;
  o.momentum = (float)momentum;
  o.blend = (float)(1.0 - momentum);
  o.nesterov = nesterov != 0;
  o.keep = (float)(1.0 - lr * weight_decay);
  o.rate = (float)(lr * scale);
  if (!isfinite(o.momentum) || !isfinite(o.blend) || !isfinite(o.keep) || !isfinite(o.rate))
    return fail(ECC_E_VALUE, "momentum, 1 - lr weight_decay and lr scale must be finite in float32");
  o.steps = steps;
  o.eps = eps;
  o.a = a;
  o.b = b;
  o.c = c;
  o.ws = ws;
  const int st = check_orth(o, ws_bytes);
  if (st != ECC_OK) return st;
  return hip_status(ecc::launch_orth(o, reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"
