// What the torch bindings share (ecc_torch.cpp, ecc_torch_block.cpp).
#pragma once

#include <ATen/hip/impl/HIPStreamMasqueradingAsCUDA.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/core/DeviceGuard.h>
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/csrc/jit/frontend/tracer.h>
#include <torch/csrc/utils/pybind.h>

#include <optional>
#include <string>
#include <vector>

#include "../../include/ecc.h"
#include "../../include/ecc_train.h"

namespace ecc_torch {

using torch::autograd::AutogradContext;
using torch::autograd::variable_list;
using Optional = std::optional<at::Tensor>;

inline const void* ptr(const at::Tensor& t) { return t.defined() ? t.const_data_ptr() : nullptr; }
inline void* out_ptr(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
// What a kernel reads: contiguous, and not the negative of what lies in memory,
// as the imaginary part of a conjugate is.
inline at::Tensor dense(const at::Tensor& t) {
  if (!t.defined()) return t;
  return t.is_neg() ? t.resolve_neg().contiguous() : t.contiguous();
}
inline at::Tensor dense(const Optional& t) { return t ? dense(*t) : at::Tensor(); }
inline void* stream_of(const at::Tensor& t) {
  return c10::hip::getCurrentHIPStreamMasqueradingAsCUDA(t.get_device()).stream();
}

inline void check(int status, const char* what) {
  if (status == ECC_OK) return;
  const std::string detail = ecc_last_error();
  pybind11::gil_scoped_acquire gil;  // backward runs on the engine's thread
  const auto error = pybind11::module_::import("euler_characteristic_curves_amd._lib").attr("EccError");
  const auto value = error(status, std::string(what) + ": " + ecc_status_string(status) + " (" + detail + ")");
  PyErr_SetObject(error.ptr(), value.ptr());
  throw pybind11::error_already_set();
}

// A dual tensor need not require a gradient, and autograd modes do not turn it off.
inline bool is_dual(const Optional& t) { return t && t->_fw_grad(/*level=*/0).defined(); }

// A traced call would leave its results' allocation in the graph, and nothing
// that writes them.
inline void refuse_tracing(const char* what) {
  TORCH_CHECK_NOT_IMPLEMENTED(!torch::jit::tracer::isTracing(), what, " cannot be traced");
}

// A gradient of these gradients is an error, not zero.
inline variable_list once_only(const variable_list& out, const char* what) {
  const auto error = std::make_shared<torch::autograd::DelayedError>(
      std::string(what) + "'s backward pass is differentiable once only", (int64_t)out.size());
  variable_list leaves(out.size());
  for (size_t i = 0; i < out.size(); ++i)
    if (out[i].defined()) leaves[i] = out[i].detach().requires_grad_();
  at::AutoGradMode on(true);
  return (*error)(std::move(leaves));
}

void define_block(pybind11::module_& m);

}  // namespace ecc_torch
