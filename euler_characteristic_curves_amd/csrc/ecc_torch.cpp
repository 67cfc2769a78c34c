// Autograd nodes of the norm calls (include/ecc_train.h), for train.py.
//
// A node written in Python runs on the engine's thread, which has to wait for
// the interpreter: a training pass over a few voxels, three launches each way,
// took 127 us of host time so.  Arguments are checked in train.py; here
// tensors become pointers, and scratch comes from torch's allocator per call,
// on the current stream.

#include <ATen/hip/impl/HIPStreamMasqueradingAsCUDA.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/core/DeviceGuard.h>
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/csrc/utils/pybind.h>

#include <optional>
#include <string>
#include <vector>

#include "../../include/ecc.h"
#include "../../include/ecc_train.h"

namespace {

using torch::autograd::AutogradContext;
using torch::autograd::variable_list;
using Optional = std::optional<at::Tensor>;

// What a call needs besides its tensors.
struct Plan {
  int64_t batch, voxels, channels, groups, dtype, pdtype, act, bytes;
  double eps;
  bool read;
};

const void* ptr(const at::Tensor& t) { return t.defined() ? t.const_data_ptr() : nullptr; }
void* out_ptr(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
at::Tensor dense(const at::Tensor& t) { return t.defined() ? t.contiguous() : t; }
at::Tensor dense(const Optional& t) { return t ? t->contiguous() : at::Tensor(); }
void* stream_of(const at::Tensor& t) { return c10::hip::getCurrentHIPStreamMasqueradingAsCUDA(t.get_device()).stream(); }

void check(int status, const char* what) {
  if (status == ECC_OK) return;
  const std::string detail = ecc_last_error();
  pybind11::gil_scoped_acquire gil;  // backward runs on the engine's thread
  const auto error = pybind11::module_::import("euler_characteristic_curves_amd._lib").attr("EccError");
  const auto value = error(status, std::string(what) + ": " + ecc_status_string(status) + " (" + detail + ")");
  PyErr_SetObject(error.ptr(), value.ptr());
  throw pybind11::error_already_set();
}

// x and the parameters are contiguous, absent ones undefined.
at::Tensor run_forward(const Plan& p, const at::Tensor& x, const at::Tensor& w, const at::Tensor& b, const at::Tensor& r,
                       const at::Tensor& o, at::Tensor* keep) {
  const c10::DeviceGuard guard(x.device());
  const auto f32 = x.options().dtype(at::kFloat).requires_grad(false);
  at::Tensor out = p.read ? at::empty(x.sizes().slice(0, x.dim() - 1), f32) : at::empty_like(x);
  if (keep) *keep = at::empty({p.batch, p.groups, 3}, f32);
  if (!p.bytes) return out;
  // statistics that nobody keeps lie behind the workspace, whose size is a multiple of 8
  const int64_t more = keep ? 0 : p.batch * p.groups * 12;
  at::Tensor ws = at::empty({p.bytes + more}, x.options().dtype(at::kByte).requires_grad(false));
  char* at_ws = static_cast<char*>(ws.data_ptr());
  float* stats = keep ? keep->data_ptr<float>() : reinterpret_cast<float*>(at_ws + p.bytes);
  const int dt = (int)p.dtype, pd = (int)p.pdtype, act = (int)p.act;
  if (p.read)
    check(ecc_norm_readout_fwd(ptr(x), dt, p.batch, p.voxels, p.channels, p.groups, ptr(w), ptr(b), ptr(r), ptr(o), pd, act,
                               (float)p.eps, out.data_ptr<float>(), stats, at_ws, p.bytes, stream_of(x)),
          "ecc_norm_readout_fwd");
  else
    check(ecc_norm_fwd(ptr(x), dt, p.batch, p.voxels, p.channels, p.groups, ptr(w), ptr(b), pd, act, (float)p.eps,
                       out.data_ptr(), stats, at_ws, p.bytes, stream_of(x)),
          "ecc_norm_fwd");
  return out;
}

struct Norm : torch::autograd::Function<Norm> {
  static at::Tensor forward(AutogradContext* ctx, const at::Tensor& x, const Optional& w, const Optional& b,
                            const Optional& r, const Optional& o, const Plan& p) {
    at::Tensor stats;
    at::Tensor out = run_forward(p, dense(x), dense(w), dense(b), dense(r), dense(o), &stats);
    ctx->save_for_backward({x, w.value_or(at::Tensor()), b.value_or(at::Tensor()), r.value_or(at::Tensor()),
                            o.value_or(at::Tensor()), stats});
    auto& d = ctx->saved_data;
    d["sizes"] = std::vector<int64_t>{p.batch, p.voxels, p.channels, p.groups, p.dtype, p.pdtype, p.act, p.bytes, p.read};
    return out;
  }

  static variable_list backward(AutogradContext* ctx, const variable_list& grads) {
    const std::vector<int64_t> s = ctx->saved_data["sizes"].toIntVector();
    const int64_t B = s[0], S = s[1], C = s[2], G = s[3], bytes = s[7];
    const int dt = (int)s[4], pd = (int)s[5], act = (int)s[6];
    const bool read = s[8];
    const bool again = at::GradMode::is_enabled();
    at::AutoGradMode off(false);
    const variable_list saved = ctx->get_saved_variables();
    variable_list in(5), out(6);
    bool any = false;
    // strided inputs are copied again here: the copy of the forward pass would hold their memory twice until now
    for (int i = 0, edge = 0; i < 5; ++i) {
      in[i] = dense(saved[i]);
      if (!in[i].defined() || !ctx->needs_input_grad(edge++)) continue;  // absent inputs have no edge
      out[i] = at::empty_like(in[i]);
      any = true;
      if (!bytes) out[i].zero_();
    }
    if (any && bytes) {
      const at::Tensor &x = in[0], g = dense(grads[0]);
      const c10::DeviceGuard guard(x.device());
      at::Tensor ws = at::empty({bytes}, x.options().dtype(at::kByte).requires_grad(false));
      const float* stats = saved[5].const_data_ptr<float>();
      if (read)
        check(ecc_norm_readout_bwd(ptr(x), dt, B, S, C, G, ptr(in[1]), ptr(in[2]), ptr(in[3]), pd, act, stats,
                                   g.const_data_ptr<float>(), out_ptr(out[0]), out_ptr(out[1]), out_ptr(out[2]),
                                   out_ptr(out[3]), out_ptr(out[4]), ws.data_ptr(), bytes, stream_of(x)),
              "ecc_norm_readout_bwd");
      else
        check(ecc_norm_bwd(ptr(x), dt, B, S, C, G, ptr(in[1]), ptr(in[2]), pd, act, stats, ptr(g), out_ptr(out[0]),
                           out_ptr(out[1]), out_ptr(out[2]), ws.data_ptr(), bytes, stream_of(x)),
              "ecc_norm_bwd");
    }
    if (again && any) {  // a gradient of these gradients is an error, not zero
      const auto error = std::make_shared<torch::autograd::DelayedError>(
          "group norm's backward pass is differentiable once only", (int64_t)out.size());
      variable_list leaves(out.size());
      for (size_t i = 0; i < out.size(); ++i)
        if (out[i].defined()) leaves[i] = out[i].detach().requires_grad_();
      at::AutoGradMode on(true);
      return (*error)(std::move(leaves));
    }
    return out;
  }
};

at::Tensor norm(const at::Tensor& x, const Optional& w, const Optional& b, const Optional& r, const Optional& o,
                const std::vector<int64_t>& sizes, int64_t dtype, int64_t pdtype, int64_t act, int64_t bytes, double eps,
                bool read) {
  const pybind11::gil_scoped_release nogil;
  // a dual tensor need not require a gradient, and autograd modes do not turn it off
  const auto dual = [](const Optional& t) { return t && t->_fw_grad(/*level=*/0).defined(); };
  TORCH_CHECK_NOT_IMPLEMENTED(!dual(x) && !dual(w) && !dual(b) && !dual(r) && !dual(o),
                              "group norm has no forward-mode derivative");
  const Plan p{sizes[0], sizes[1], sizes[2], sizes[3], dtype, pdtype, act, bytes, eps, read};
  const auto wants = [](const Optional& t) { return t && t->requires_grad(); };
  if (at::GradMode::is_enabled() && (x.requires_grad() || wants(w) || wants(b) || wants(r) || wants(o)))
    return Norm::apply(x, w, b, r, o, p);
  return run_forward(p, dense(x), dense(w), dense(b), dense(r), dense(o), nullptr);
}

}  // namespace

PYBIND11_MODULE(_torch, m) { m.def("norm", &norm); }
