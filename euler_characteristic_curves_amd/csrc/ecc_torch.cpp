// Autograd nodes of the norm calls (include/ecc_train.h), for train.py.
//
// A node written in Python runs on the engine's thread, which has to wait for
// the interpreter: a training pass over a few voxels, three launches each way,
// took 127 us of host time so.  Arguments are checked in train.py; here
// tensors become pointers, and scratch comes from torch's allocator per call,
// on the current stream.

#include "ecc_torch.hpp"

namespace {

using namespace ecc_torch;

// What a call needs besides its tensors.
struct Plan {
  int64_t batch, voxels, channels, groups, dtype, pdtype, act, bytes;
  double eps;
  bool read;
};

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
    if (again && any) return once_only(out, "group norm");
    return out;
  }
};

at::Tensor norm(const at::Tensor& x, const Optional& w, const Optional& b, const Optional& r, const Optional& o,
                const std::vector<int64_t>& sizes, int64_t dtype, int64_t pdtype, int64_t act, int64_t bytes, double eps,
                bool read) {
  refuse_tracing("group norm");
  const pybind11::gil_scoped_release nogil;
  TORCH_CHECK_NOT_IMPLEMENTED(!is_dual(x) && !is_dual(w) && !is_dual(b) && !is_dual(r) && !is_dual(o),
                              "group norm has no forward-mode derivative");
  const Plan p{sizes[0], sizes[1], sizes[2], sizes[3], dtype, pdtype, act, bytes, eps, read};
  const auto wants = [](const Optional& t) { return t && t->requires_grad(); };
  if (at::GradMode::is_enabled() && (x.requires_grad() || wants(w) || wants(b) || wants(r) || wants(o)))
    return Norm::apply(x, w, b, r, o, p);
  return run_forward(p, dense(x), dense(w), dense(b), dense(r), dense(o), nullptr);
}

}  // namespace

PYBIND11_MODULE(_torch, m) {
  m.def("norm", &norm);
  ecc_torch::define_block(m);
}
