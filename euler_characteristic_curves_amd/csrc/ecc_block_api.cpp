// C ABI of a residual block's operators (include/ecc_train.h): argument
// validation, error reporting, dispatch.

#include "../../include/ecc_train.h"

#include <hip/hip_runtime.h>
#include <math.h>

#include "../../include/ecc.h"
#include "ecc_act.hpp"
#include "ecc_block_internal.hpp"
#include "ecc_check.hpp"

namespace {

using ecc::check_eps;
using ecc::check_workspace;
using ecc::fail;
using ecc::hip_status;
using ecc::is_dtype;

int check_residual_shape(int64_t batch, int64_t inner, int64_t channels, bool sample_gates) {
  if (batch < 1 || inner < 1 || channels < 1)
    return fail(ECC_E_SHAPE, "batch, inner and channels must be >= 1 (got inner=%lld channels=%lld)", inner, channels);
  if (channels > ECC_MAX_CHANNELS) return fail(ECC_E_SHAPE, "channels=%lld exceeds %lld", channels, ECC_MAX_CHANNELS);
  if (inner > ECC_MAX_VOXELS / channels || batch > ECC_MAX_VOXELS / (inner * channels))
    return fail(ECC_E_SHAPE, "more than 2^40 elements");
  if (sample_gates && batch > ECC_MAX_NORM_BATCH)
    return fail(ECC_E_SHAPE, "batch=%lld with gates of their own exceeds %lld", batch, ECC_MAX_NORM_BATCH);
  return ECC_OK;
}

// Checks shared by both directions, and the part of the arguments they share.
int check_residual(ecc::ResArgs& a, const void* x, int xdtype, const void* branch, int dtype, int64_t batch, int64_t inner,
                   int64_t channels, const void* gate, int per_sample, const void* weight, const void* branch_weight,
                   int pdtype, int norm_branch, float scale) {
  ecc::set_error("");
  if (!x) return fail(ECC_E_NULL, "x is NULL");
  if (!is_dtype(dtype)) return fail(ECC_E_DTYPE, "dtype %lld is not one of ECC_T_*", dtype);
  if (xdtype != ECC_T_F32 && xdtype != dtype)
    return fail(ECC_E_DTYPE, "xdtype %lld is neither ECC_T_F32 nor dtype (%lld)", xdtype, dtype);
  if (pdtype != ECC_T_F32 && pdtype != dtype)
    return fail(ECC_E_DTYPE, "pdtype %lld is neither ECC_T_F32 nor dtype (%lld)", pdtype, dtype);
  const int st = check_residual_shape(batch, inner, channels, gate && per_sample);
  if (st != ECC_OK) return st;
  if (!branch && (gate || branch_weight || norm_branch))
    return fail(ECC_E_NULL, "branch is NULL, but its gate or its norm is given");
  if (!norm_branch && branch_weight) return fail(ECC_E_VALUE, "branch_weight is given without norm_branch");
  if (!isfinite(scale)) return fail(ECC_E_VALUE, "scale must be finite");
  a = ecc::ResArgs{};
  a.x = x;
  a.branch = branch;
  a.xdtype = xdtype;
  a.dtype = dtype;
  a.batch = batch;
  a.inner = inner;
  a.channels = channels;
  a.gate = gate;
  a.gate_stride = gate && per_sample ? channels : 0;
  a.weight = weight;
  a.branch_weight = branch_weight;
  a.pdtype = pdtype;
  a.norm_branch = norm_branch != 0;
  a.scale = scale;
  return ECC_OK;
}

int check_recurrence_shape(int64_t batch, int64_t steps, int64_t channels, int dtype) {
  if (!is_dtype(dtype)) return fail(ECC_E_DTYPE, "dtype %lld is not one of ECC_T_*", dtype);
  if (batch < 1 || steps < 1 || channels < 1)
    return fail(ECC_E_SHAPE, "batch, steps and channels must be >= 1 (got steps=%lld channels=%lld)", steps, channels);
  if (batch > ECC_MAX_VOXELS || steps > ECC_MAX_VOXELS / channels || batch > ECC_MAX_VOXELS / (steps * channels))
    return fail(ECC_E_SHAPE, "more than 2^40 elements");
  if (channels > ECC_MAX_RECURRENCE_CHANNELS)
    return fail(ECC_E_SHAPE, "channels=%lld exceeds %lld", channels, ECC_MAX_RECURRENCE_CHANNELS);
  if (batch > INT32_MAX) return fail(ECC_E_SHAPE, "batch=%lld exceeds 2^31 - 1", batch);
  return ECC_OK;
}

int check_recurrence(ecc::RecArgs& a, const void* x, const void* gate, int dtype, int64_t batch, int64_t steps,
                     int64_t channels, const int64_t* lengths, void* ws, size_t ws_bytes) {
  ecc::set_error("");
  if (!x) return fail(ECC_E_NULL, "x is NULL");
  if (!gate) return fail(ECC_E_NULL, "gate is NULL");
  const int st = check_recurrence_shape(batch, steps, channels, dtype);
  if (st != ECC_OK) return st;
  a = ecc::RecArgs{};
  a.x = x;
  a.gate = gate;
  a.batch = batch;
  a.steps = steps;
  a.channels = channels;
  a.lengths = lengths;
  a.ws = ws;
  return check_workspace(ws, ws_bytes, ecc::rec_workspace_bytes(batch, steps, channels, dtype != ECC_T_F32));
}

int check_glu_shape(int64_t rows, int64_t channels, int64_t hidden, int dtype, bool backward, bool aligned) {
  if (!is_dtype(dtype)) return fail(ECC_E_DTYPE, "dtype %lld is not one of ECC_T_*", dtype);
  if (rows < 1 || channels < 1 || hidden < 1)
    return fail(ECC_E_SHAPE, "rows, channels and hidden must be >= 1 (got channels=%lld hidden=%lld)", channels, hidden);
  if (channels > ECC_MAX_MATRIX || hidden > ECC_MAX_MATRIX)
    return fail(ECC_E_SHAPE, "weights of %lld x %lld exceed the limit per side", hidden, channels);
  const int64_t wide = channels > hidden ? channels : hidden;
  if (rows > ECC_MAX_VOXELS / wide) return fail(ECC_E_SHAPE, "more than 2^40 elements");
  const ecc::GluPlan plan = ecc::glu_plan(rows, channels, hidden, dtype == ECC_T_F32 ? 4 : 2, backward);
  if (!ecc::glu_launches(plan, backward, aligned)) return fail(ECC_E_SHAPE, "rows=%lld are too many for one launch", rows);
  return ECC_OK;
}

int check_glu(ecc::GluArgs& a, const void* x, int dtype, int64_t rows, int64_t channels, int64_t hidden, const void* w_gate,
              const void* w_up, const void* b_gate, const void* b_up, int act, bool backward) {
  ecc::set_error("");
  if (!x) return fail(ECC_E_NULL, "x is NULL");
  if (!w_gate) return fail(ECC_E_NULL, "w_gate is NULL");
  if (!w_up) return fail(ECC_E_NULL, "w_up is NULL");
  if (act < ECC_ACT_NONE || act > ECC_ACT_GELU) return fail(ECC_E_ACT, "act %lld is not one of ECC_ACT_*", act);
  const auto at16 = [](const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
  const int st = check_glu_shape(rows, channels, hidden, dtype, backward, at16(x) && at16(w_gate) && at16(w_up));
  if (st != ECC_OK) return st;
  a = ecc::GluArgs{};
  a.x = x;
  a.wg = w_gate;
  a.wu = w_up;
  a.bg = b_gate;
  a.bu = b_up;
  a.act = act;
  a.rows = rows;
  a.channels = channels;
  a.hidden = hidden;
  return ECC_OK;
}

}  // namespace

extern "C" {

size_t ecc_residual_norm_workspace_bytes(int64_t batch, int64_t inner, int64_t channels, int gate_per_sample) {
  if (check_residual_shape(batch, inner, channels, gate_per_sample != 0) != ECC_OK) return 0;
  return ecc::res_workspace_bytes(batch, inner, channels, gate_per_sample != 0);
}

int ecc_residual_norm_fwd(const void* x, int xdtype, const void* branch, int dtype, int64_t batch, int64_t inner,
                          int64_t channels, const void* gate, int gate_per_sample, const void* weight,
                          const void* branch_weight, int pdtype, int norm_branch, float scale, float eps, void* y, void* z,
                          float* stats, void* stream) {
  ecc::ResArgs a;
  int st = check_residual(a, x, xdtype, branch, dtype, batch, inner, channels, gate, gate_per_sample, weight, branch_weight,
                          pdtype, norm_branch, scale);
  if (st != ECC_OK) return st;
  if (!z) return fail(ECC_E_NULL, "z is NULL");
  if (branch && !y) return fail(ECC_E_NULL, "y is NULL");
  st = check_eps(eps);
  if (st != ECC_OK) return st;
  a.eps = eps;
  a.y = y;
  a.z = z;
  a.stats = stats;
  return hip_status(ecc::launch_residual_fwd(a, reinterpret_cast<hipStream_t>(stream)));
}

int ecc_residual_norm_bwd(const void* x, int xdtype, const void* branch, int dtype, int64_t batch, int64_t inner,
                          int64_t channels, const void* gate, int gate_per_sample, const void* weight,
                          const void* branch_weight, int pdtype, int norm_branch, float scale, const float* stats,
                          const void* grad_y, const void* grad_z, void* grad_x, void* grad_branch, void* grad_gate,
                          void* grad_weight, void* grad_branch_weight, void* ws, size_t ws_bytes, void* stream) {
  ecc::ResArgs a;
  int st = check_residual(a, x, xdtype, branch, dtype, batch, inner, channels, gate, gate_per_sample, weight, branch_weight,
                          pdtype, norm_branch, scale);
  if (st != ECC_OK) return st;
  if (!stats) return fail(ECC_E_NULL, "stats is NULL");
  if (!grad_y && !grad_z) return fail(ECC_E_NULL, "grad_y and grad_z are both NULL");
  if (!grad_x && !grad_branch && !grad_gate && !grad_weight && !grad_branch_weight)
    return fail(ECC_E_NULL, "every gradient is NULL");
  if ((grad_branch && !branch) || (grad_gate && !gate) || (grad_weight && !weight) || (grad_branch_weight && !branch_weight))
    return fail(ECC_E_NULL, "a gradient of an argument that is NULL is wanted");
  st = check_workspace(ws, ws_bytes, ecc::res_workspace_bytes(batch, inner, channels, a.gate_stride != 0));
  if (st != ECC_OK) return st;
  a.stats = const_cast<float*>(stats);
  a.gy = grad_y;
  a.gz = grad_z;
  a.gx = grad_x;
  a.gbranch = grad_branch;
  a.ggate = grad_gate;
  a.gweight = grad_weight;
  a.gbranch_weight = grad_branch_weight;
  a.ws = ws;
  return hip_status(ecc::launch_residual_bwd(a, reinterpret_cast<hipStream_t>(stream)));
}

size_t ecc_gated_recurrence_workspace_bytes(int64_t batch, int64_t steps, int64_t channels, int dtype) {
  if (check_recurrence_shape(batch, steps, channels, dtype) != ECC_OK) return 0;
  return ecc::rec_workspace_bytes(batch, steps, channels, dtype != ECC_T_F32);
}

size_t ecc_gated_recurrence_saved_bytes(int64_t batch, int64_t steps, int64_t channels, int dtype) {
  if (check_recurrence_shape(batch, steps, channels, dtype) != ECC_OK) return 0;
  return (size_t)(batch * ecc::rec_shape(batch, steps, channels, dtype != ECC_T_F32).tiles * channels) * sizeof(float);
}

int ecc_gated_recurrence_fwd(const void* x, const void* gate, int dtype, int64_t batch, int64_t steps, int64_t channels,
                             const float* state, const int64_t* lengths, void* h, float* last, float* saved, void* ws,
                             size_t ws_bytes, void* stream) {
  ecc::RecArgs a;
  const int st = check_recurrence(a, x, gate, dtype, batch, steps, channels, lengths, ws, ws_bytes);
  if (st != ECC_OK) return st;
  if (!h) return fail(ECC_E_NULL, "h is NULL");
  if (!last) return fail(ECC_E_NULL, "last is NULL");
  a.state = state;
  a.h = h;
  a.last = last;
  a.saved = saved;
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (dtype == ECC_T_F32) return hip_status(ecc::launch_recurrence_fwd<float>(a, s));
  if (dtype == ECC_T_F16) return hip_status(ecc::launch_recurrence_fwd<ecc::f16>(a, s));
  return hip_status(ecc::launch_recurrence_fwd<ecc::bf16>(a, s));
}

int ecc_gated_recurrence_bwd(const void* x, const void* gate, int dtype, int64_t batch, int64_t steps, int64_t channels,
                             const int64_t* lengths, const float* saved, const void* grad_h, const float* grad_last,
                             void* grad_x, void* grad_gate, float* grad_state, void* ws, size_t ws_bytes, void* stream) {
  ecc::RecArgs a;
  const int st = check_recurrence(a, x, gate, dtype, batch, steps, channels, lengths, ws, ws_bytes);
  if (st != ECC_OK) return st;
  if (!saved) return fail(ECC_E_NULL, "saved is NULL");
  if (!grad_h && !grad_last) return fail(ECC_E_NULL, "grad_h and grad_last are both NULL");
  if (!grad_x && !grad_gate && !grad_state) return fail(ECC_E_NULL, "every gradient is NULL");
  a.saved = const_cast<float*>(saved);
  a.gh = grad_h;
  a.glast = grad_last;
  a.gx = grad_x;
  a.ggate = grad_gate;
  a.gstate = grad_state;
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (dtype == ECC_T_F32) return hip_status(ecc::launch_recurrence_bwd<float>(a, s));
  if (dtype == ECC_T_F16) return hip_status(ecc::launch_recurrence_bwd<ecc::f16>(a, s));
  return hip_status(ecc::launch_recurrence_bwd<ecc::bf16>(a, s));
}

size_t ecc_gated_linear_workspace_bytes(int64_t rows, int64_t channels, int64_t hidden, int dtype, int backward) {
  if (check_glu_shape(rows, channels, hidden, dtype, backward != 0, true) != ECC_OK) return 0;
  return ecc::glu_plan(rows, channels, hidden, dtype == ECC_T_F32 ? 4 : 2, backward != 0).bytes;
}

int ecc_gated_linear_fwd(const void* x, int dtype, int64_t rows, int64_t channels, int64_t hidden, const void* w_gate,
                         const void* w_up, const void* b_gate, const void* b_up, int act, void* h, void* ws, size_t ws_bytes,
                         void* stream) {
  ecc::GluArgs a;
  int st = check_glu(a, x, dtype, rows, channels, hidden, w_gate, w_up, b_gate, b_up, act, false);
  if (st != ECC_OK) return st;
  if (!h) return fail(ECC_E_NULL, "h is NULL");
  const ecc::GluPlan plan = ecc::glu_plan(rows, channels, hidden, dtype == ECC_T_F32 ? 4 : 2, false);
  if (plan.packed) st = check_workspace(ws, ws_bytes, plan.bytes);
  if (st != ECC_OK) return st;
  a.h = h;
  a.ws = ws;
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (dtype == ECC_T_F32) return hip_status(ecc::launch_glu_fwd<float>(a, s));
  if (dtype == ECC_T_F16) return hip_status(ecc::launch_glu_fwd<ecc::f16>(a, s));
  return hip_status(ecc::launch_glu_fwd<ecc::bf16>(a, s));
}

int ecc_gated_linear_bwd(const void* x, int dtype, int64_t rows, int64_t channels, int64_t hidden, const void* w_gate,
                         const void* w_up, const void* b_gate, const void* b_up, int act, const void* grad_h, void* grad_x,
                         void* grad_w_gate, void* grad_w_up, void* grad_b_gate, void* grad_b_up, void* ws, size_t ws_bytes,
                         void* stream) {
  ecc::GluArgs a;
  int st = check_glu(a, x, dtype, rows, channels, hidden, w_gate, w_up, b_gate, b_up, act, true);
  if (st != ECC_OK) return st;
  if (!grad_h) return fail(ECC_E_NULL, "grad_h is NULL");
  if (!grad_x && !grad_w_gate && !grad_w_up && !grad_b_gate && !grad_b_up)
    return fail(ECC_E_NULL, "every gradient is NULL");
  if ((grad_b_gate && !b_gate) || (grad_b_up && !b_up))
    return fail(ECC_E_NULL, "a gradient of an argument that is NULL is wanted");
  st = check_workspace(ws, ws_bytes, ecc::glu_plan(rows, channels, hidden, dtype == ECC_T_F32 ? 4 : 2, true).bytes);
  if (st != ECC_OK) return st;
  a.gh = grad_h;
  a.gx = grad_x;
  a.gwg = grad_w_gate;
  a.gwu = grad_w_up;
  a.gbg = grad_b_gate;
  a.gbu = grad_b_up;
  a.ws = ws;
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (dtype == ECC_T_F32) return hip_status(ecc::launch_glu_bwd<float>(a, s));
  if (dtype == ECC_T_F16) return hip_status(ecc::launch_glu_bwd<ecc::f16>(a, s));
  return hip_status(ecc::launch_glu_bwd<ecc::bf16>(a, s));
}

}  // extern "C"
