// Argument checks and autograd nodes of a residual block's operators
// (include/ecc_train.h), for block.py.
//
// One position of a sequence is a few microseconds of GPU time, so the checks
// are here too: in Python they took longer than the kernels.

#include <c10/hip/HIPGraphsC10Utils.h>

#include "ecc_torch.hpp"

namespace ecc_torch {
namespace {

int64_t type_of(at::ScalarType t) {
  return t == at::kFloat ? ECC_T_F32 : t == at::kHalf ? ECC_T_F16 : t == at::kBFloat16 ? ECC_T_BF16 : -1;
}

void on_device(const at::Tensor& t, const char* name, const c10::Device* where) {
  TORCH_CHECK_VALUE(t.is_cuda(), name, " must be on a ROCm device (got ", t.device(), ")");
  TORCH_CHECK_VALUE(t.layout() == at::kStrided, name, " must be a strided tensor");
  TORCH_CHECK_VALUE(!where || t.device() == *where, name, " is on ", t.device(), ", expected ", where ? *where : t.device());
}

void features(const at::Tensor& t, const char* name) {
  on_device(t, name, nullptr);
  TORCH_CHECK_TYPE(type_of(t.scalar_type()) >= 0, name, " dtype ", t.scalar_type(),
                   " not supported (float32, float16 or bfloat16)");
}

// A parameter that is `like` the others given before it: float32 or the features' type.
void parameter(const Optional& t, const char* name, const at::Tensor& x, at::ScalarType type, int64_t* pdtype) {
  if (!t) return;
  const c10::Device where = x.device();
  on_device(*t, name, &where);
  TORCH_CHECK_TYPE(t->scalar_type() == at::kFloat || t->scalar_type() == type, name, " must be torch.float32 or the features' ",
                   type, " (got ", t->scalar_type(), ")");
  const int64_t here = type_of(t->scalar_type());
  TORCH_CHECK_TYPE(*pdtype < 0 || *pdtype == here, name, " is ", t->scalar_type(), ", the parameters before it are not");
  *pdtype = here;
}

void vector(const Optional& t, const char* name, int64_t n) {
  TORCH_CHECK_VALUE(!t || (t->dim() == 1 && t->size(0) == n), name, " must be [", n, "] (got ", t->sizes(), ")");
}

bool capturing() {
  return c10::hip::currentStreamCaptureStatusMayInitCtx() != c10::hip::CaptureStatus::None;
}
// A leaf's gradient accumulator belongs to the stream it was made on, and lives
// as long as any graph that reaches the leaf.  A captured backward pass makes
// that stream wait for the capturing one: another stream joins the capture by
// it, the default one cannot, which ends the process.  `in`: a node's first
// inputs; what no gradient is wanted of has no say.  Absent inputs have no edge.
void refuse_foreign_capture(AutogradContext* ctx, const variable_list& in, size_t count) {
  if (!capturing()) return;
  for (size_t i = 0, edge = 0; i < count; ++i) {
    const at::Tensor& t = in[i];
    if (!t.defined() || !ctx->needs_input_grad(edge++) || !t.requires_grad() || !t.is_leaf()) continue;
    const auto node = torch::autograd::impl::try_get_grad_accumulator(t);
    if (!node) continue;
    const auto made = node->stream();
    TORCH_CHECK(!made || *made != c10::hip::getDefaultHIPStreamMasqueradingAsCUDA(t.get_device()).unwrap(),
                "a backward pass is captured while an eager graph of the same leaves is alive: free that graph first");
  }
}

at::Tensor bytes_like(const at::Tensor& x, int64_t bytes) {
  return at::empty({bytes}, x.options().dtype(at::kByte).requires_grad(false));
}
at::Tensor result_like(const at::Tensor& x) { return at::empty(x.sizes(), x.options().requires_grad(false)); }

bool wants(const Optional& t) { return t && t->requires_grad(); }

// Gradients of a node's first inputs: what is wanted of them, contiguous, 0 where nothing is summed.
// Absent inputs have no edge.
bool gradients(AutogradContext* ctx, const variable_list& in, variable_list& out, bool nothing) {
  bool any = false;
  for (size_t i = 0, edge = 0; i < out.size(); ++i) {
    if (!in[i].defined() || !ctx->needs_input_grad(edge++)) continue;
    out[i] = result_like(in[i]);
    any = true;
    if (nothing) out[i].zero_();
  }
  return any;
}

// ------------------------------------------------- norms around a block
struct ResPlan {
  int64_t batch, inner, channels, xdtype, dtype, pdtype, per_sample, norm_branch;
  double scale, eps;
  at::ScalarType ztype;
};

// Tensors are contiguous, absent ones undefined.
variable_list residual_forward(const ResPlan& p, const at::Tensor& x, const at::Tensor& b, const at::Tensor& g,
                               const at::Tensor& w, const at::Tensor& bw, at::Tensor* keep) {
  const c10::DeviceGuard guard(x.device());
  at::Tensor y, z = at::empty(x.sizes(), x.options().dtype(p.ztype).requires_grad(false));
  if (b.defined()) y = result_like(x);
  if (keep) *keep = at::empty({p.batch * p.inner, 2}, x.options().dtype(at::kFloat).requires_grad(false));
  if (x.numel())
    check(ecc_residual_norm_fwd(ptr(x), (int)p.xdtype, ptr(b), (int)p.dtype, p.batch, p.inner, p.channels, ptr(g),
                                (int)p.per_sample, ptr(w), ptr(bw), (int)p.pdtype, (int)p.norm_branch, (float)p.scale,
                                (float)p.eps, out_ptr(y), out_ptr(z), keep ? keep->data_ptr<float>() : nullptr, stream_of(x)),
          "ecc_residual_norm_fwd");
  if (!y.defined()) return {z};
  return {y, z};
}

struct Residual : torch::autograd::Function<Residual> {
  static variable_list forward(AutogradContext* ctx, const at::Tensor& x, const Optional& b, const Optional& g,
                               const Optional& w, const Optional& bw, const ResPlan& p) {
    at::Tensor stats;
    variable_list out = residual_forward(p, dense(x), dense(b), dense(g), dense(w), dense(bw), &stats);
    ctx->set_materialize_grads(false);
    ctx->save_for_backward({x, b.value_or(at::Tensor()), g.value_or(at::Tensor()), w.value_or(at::Tensor()),
                            bw.value_or(at::Tensor()), stats});
    ctx->saved_data["plan"] = std::vector<int64_t>{p.batch, p.inner, p.channels, p.xdtype, p.dtype, p.pdtype, p.per_sample,
                                                   p.norm_branch};
    ctx->saved_data["scale"] = p.scale;
    return out;
  }

  static variable_list backward(AutogradContext* ctx, const variable_list& grads) {
    const std::vector<int64_t> s = ctx->saved_data["plan"].toIntVector();
    const bool again = at::GradMode::is_enabled();
    at::AutoGradMode off(false);
    const variable_list saved = ctx->get_saved_variables();
    variable_list in(5), out(6);
    refuse_foreign_capture(ctx, saved, 5);
    for (int i = 0; i < 5; ++i) in[i] = dense(saved[i]);
    variable_list wanted(5);
    const at::Tensor& x = in[0];
    const c10::DeviceGuard guard(x.device());
    const at::Tensor gy = in[1].defined() ? dense(grads[0]) : at::Tensor(), gz = dense(grads.back());
    const bool nothing = !x.numel() || (!gy.defined() && !gz.defined());
    const bool any = gradients(ctx, in, wanted, nothing);
    if (any && !nothing) {
      const int64_t bytes = ecc_residual_norm_workspace_bytes(s[0], s[1], s[2], (int)s[6]);
      at::Tensor ws = bytes_like(x, bytes);
      check(ecc_residual_norm_bwd(ptr(x), (int)s[3], ptr(in[1]), (int)s[4], s[0], s[1], s[2], ptr(in[2]), (int)s[6],
                                  ptr(in[3]), ptr(in[4]), (int)s[5], (int)s[7], (float)ctx->saved_data["scale"].toDouble(),
                                  saved[5].const_data_ptr<float>(), ptr(gy), ptr(gz), out_ptr(wanted[0]),
                                  out_ptr(wanted[1]), out_ptr(wanted[2]), out_ptr(wanted[3]), out_ptr(wanted[4]),
                                  ws.data_ptr(), bytes, stream_of(x)),
            "ecc_residual_norm_bwd");
    }
    for (int i = 0; i < 5; ++i) out[i] = wanted[i];
    if (again && any) return once_only(out, "residual norm");
    return out;
  }
};

variable_list residual_norm(const at::Tensor& x, const Optional& b, const Optional& g, const Optional& w, const Optional& bw,
                            double scale, double eps, bool norm_branch, const std::optional<at::ScalarType>& ztype) {
  refuse_tracing("residual norm");
  const pybind11::gil_scoped_release nogil;
  features(x, "x");
  TORCH_CHECK_VALUE(x.dim() >= 2, "x must be [batch, *space, channels] (got ", x.sizes(), ")");
  const c10::Device where = x.device();
  ResPlan p{};
  p.channels = x.size(-1);
  p.batch = x.size(0);
  p.ztype = ztype.value_or(b ? b->scalar_type() : x.scalar_type());
  TORCH_CHECK_VALUE(p.channels >= 1, "x has no channels");
  if (b) {
    features(*b, "branch");
    on_device(*b, "branch", &where);
    TORCH_CHECK_VALUE(b->sizes() == x.sizes(), "branch must have x's shape ", x.sizes(), " (got ", b->sizes(), ")");
  }
  p.xdtype = type_of(x.scalar_type());
  p.dtype = type_of(p.ztype);
  TORCH_CHECK_TYPE(p.dtype >= 0 && (x.scalar_type() == at::kFloat || x.scalar_type() == p.ztype), b ? "branch" : "dtype",
                   " must be x's ", x.scalar_type(), ", or 16-bit beside a float32 x (got ", p.ztype, ")");
  p.pdtype = -1;
  parameter(g, "gate", x, p.ztype, &p.pdtype);
  parameter(w, "weight", x, p.ztype, &p.pdtype);
  parameter(bw, "branch_weight", x, p.ztype, &p.pdtype);
  if (p.pdtype < 0) p.pdtype = ECC_T_F32;
  vector(w, "weight", p.channels);
  vector(bw, "branch_weight", p.channels);
  if (g && g->dim() == 2) {
    TORCH_CHECK_VALUE(g->size(0) == p.batch && g->size(1) == p.channels, "gate must be [", p.channels, "] or [", p.batch, ", ",
                      p.channels, "] (got ", g->sizes(), ")");
    p.per_sample = 1;
  } else {
    vector(g, "gate", p.channels);
  }
  TORCH_CHECK_VALUE(!bw || norm_branch, "branch_weight is given, but norm_branch is False");
  TORCH_CHECK_NOT_IMPLEMENTED(!is_dual(x) && !is_dual(b) && !is_dual(g) && !is_dual(w) && !is_dual(bw),
                              "residual norm has no forward-mode derivative");
  p.inner = x.numel() ? x.numel() / (p.batch * p.channels) : 0;
  p.norm_branch = norm_branch;
  p.scale = scale;
  p.eps = eps;
  if (at::GradMode::is_enabled() && (x.requires_grad() || wants(b) || wants(g) || wants(w) || wants(bw)))
    return Residual::apply(x, b, g, w, bw, p);
  return residual_forward(p, dense(x), dense(b), dense(g), dense(w), dense(bw), nullptr);
}

// ------------------------------------------- gated pair of projections
struct GluPlan {
  int64_t rows, channels, hidden, dtype, act;
};

// Tensors are contiguous, absent ones undefined.
at::Tensor glu_forward(const GluPlan& p, const at::Tensor& x, const at::Tensor& wg, const at::Tensor& wu, const at::Tensor& bg,
                       const at::Tensor& bu) {
  const c10::DeviceGuard guard(x.device());
  std::vector<int64_t> sizes = x.sizes().vec();
  sizes.back() = p.hidden;
  at::Tensor h = at::empty(sizes, x.options().requires_grad(false));
  if (!h.numel()) return h;
  const int64_t bytes = ecc_gated_linear_workspace_bytes(p.rows, p.channels, p.hidden, (int)p.dtype, 0);
  at::Tensor ws;
  if (bytes > 256) ws = bytes_like(x, bytes);  // no workspace otherwise
  check(ecc_gated_linear_fwd(ptr(x), (int)p.dtype, p.rows, p.channels, p.hidden, ptr(wg), ptr(wu), ptr(bg), ptr(bu),
                             (int)p.act, h.data_ptr(), out_ptr(ws), ws.defined() ? bytes : 0, stream_of(x)),
        "ecc_gated_linear_fwd");
  return h;
}

struct Glu : torch::autograd::Function<Glu> {
  static at::Tensor forward(AutogradContext* ctx, const at::Tensor& x, const at::Tensor& wg, const at::Tensor& wu,
                            const Optional& bg, const Optional& bu, const GluPlan& p) {
    at::Tensor h = glu_forward(p, dense(x), dense(wg), dense(wu), dense(bg), dense(bu));
    ctx->save_for_backward({x, wg, wu, bg.value_or(at::Tensor()), bu.value_or(at::Tensor())});
    ctx->saved_data["plan"] = std::vector<int64_t>{p.rows, p.channels, p.hidden, p.dtype, p.act};
    return h;
  }

  static variable_list backward(AutogradContext* ctx, const variable_list& grads) {
    const std::vector<int64_t> p = ctx->saved_data["plan"].toIntVector();
    const bool again = at::GradMode::is_enabled();
    at::AutoGradMode off(false);
    const variable_list saved = ctx->get_saved_variables();
    refuse_foreign_capture(ctx, saved, 5);
    variable_list in(5), wanted(5), out(6);
    for (int i = 0; i < 5; ++i) in[i] = dense(saved[i]);
    const at::Tensor &x = in[0], g = dense(grads[0]);
    const c10::DeviceGuard guard(x.device());
    const bool any = gradients(ctx, in, wanted, !p[0]);
    if (any && p[0]) {
      const int64_t bytes = ecc_gated_linear_workspace_bytes(p[0], p[1], p[2], (int)p[3], 1);
      at::Tensor ws = bytes_like(x, bytes);
      check(ecc_gated_linear_bwd(ptr(x), (int)p[3], p[0], p[1], p[2], ptr(in[1]), ptr(in[2]), ptr(in[3]), ptr(in[4]),
                                 (int)p[4], ptr(g), out_ptr(wanted[0]), out_ptr(wanted[1]), out_ptr(wanted[2]),
                                 out_ptr(wanted[3]), out_ptr(wanted[4]), ws.data_ptr(), bytes, stream_of(x)),
            "ecc_gated_linear_bwd");
    }
    for (int i = 0; i < 5; ++i) out[i] = wanted[i];
    if (again && any) return once_only(out, "gated linear");
    return out;
  }
};

at::Tensor gated_linear(const at::Tensor& x, const at::Tensor& wg, const at::Tensor& wu, const Optional& bg,
                        const Optional& bu, int64_t act) {
  refuse_tracing("gated linear");
  const pybind11::gil_scoped_release nogil;
  features(x, "x");
  TORCH_CHECK_VALUE(x.dim() >= 1, "x must be [*space, channels]");
  const c10::Device where = x.device();
  GluPlan p{};
  p.channels = x.size(-1);
  TORCH_CHECK_VALUE(p.channels >= 1, "x has no channels");
  p.rows = x.numel() / p.channels;
  p.dtype = type_of(x.scalar_type());
  p.act = act;
  const auto like = [&](const Optional& t, const char* name, int64_t dim) {
    if (!t) return;
    on_device(*t, name, &where);
    TORCH_CHECK_TYPE(t->scalar_type() == x.scalar_type(), name, " must be ", x.scalar_type(), " (got ", t->scalar_type(), ")");
    TORCH_CHECK_VALUE(t->dim() == dim, name, " must be ", dim == 2 ? "[hidden, channels]" : "[hidden]", " (got ", t->sizes(), ")");
  };
  like(wg, "w_gate", 2);
  like(wu, "w_up", 2);
  like(bg, "b_gate", 1);
  like(bu, "b_up", 1);
  p.hidden = wg.size(0);
  TORCH_CHECK_VALUE(p.hidden >= 1 && wg.size(1) == p.channels, "w_gate must be [hidden, ", p.channels, "] (got ", wg.sizes(), ")");
  TORCH_CHECK_VALUE(wu.sizes() == wg.sizes(), "w_up must have w_gate's shape ", wg.sizes(), " (got ", wu.sizes(), ")");
  vector(bg, "b_gate", p.hidden);
  vector(bu, "b_up", p.hidden);
  TORCH_CHECK_NOT_IMPLEMENTED(!is_dual(x) && !is_dual(wg) && !is_dual(wu) && !is_dual(bg) && !is_dual(bu),
                              "gated linear has no forward-mode derivative");
  if (at::GradMode::is_enabled() &&
      (x.requires_grad() || wg.requires_grad() || wu.requires_grad() || wants(bg) || wants(bu)))
    return Glu::apply(x, wg, wu, bg, bu, p);
  return glu_forward(p, dense(x), dense(wg), dense(wu), dense(bg), dense(bu));
}

// -------------------------------------------------------- gated recurrence
struct RecPlan {
  int64_t batch, steps, channels, dtype;
};

// Tensors are contiguous, absent ones undefined.
variable_list recurrence_forward(const RecPlan& p, const at::Tensor& x, const at::Tensor& f, const at::Tensor& s,
                                 const at::Tensor& n, at::Tensor* keep) {
  const c10::DeviceGuard guard(x.device());
  const auto f32 = x.options().dtype(at::kFloat).requires_grad(false);
  at::Tensor h = result_like(x), last = at::empty({p.batch, p.channels}, f32);
  if (!x.numel()) {
    if (s.defined())
      last.copy_(s);
    else
      last.zero_();
    return {h, last};
  }
  const int64_t bytes = ecc_gated_recurrence_workspace_bytes(p.batch, p.steps, p.channels, (int)p.dtype);
  const int64_t saved = ecc_gated_recurrence_saved_bytes(p.batch, p.steps, p.channels, (int)p.dtype);
  if (keep) *keep = at::empty({saved / 4}, f32);
  at::Tensor ws = bytes_like(x, bytes);
  check(ecc_gated_recurrence_fwd(ptr(x), ptr(f), (int)p.dtype, p.batch, p.steps, p.channels,
                                 s.defined() ? s.const_data_ptr<float>() : nullptr,
                                 n.defined() ? n.const_data_ptr<int64_t>() : nullptr, h.data_ptr(), last.data_ptr<float>(),
                                 keep ? keep->data_ptr<float>() : nullptr, ws.data_ptr(), bytes, stream_of(x)),
        "ecc_gated_recurrence_fwd");
  return {h, last};
}

struct Recurrence : torch::autograd::Function<Recurrence> {
  static variable_list forward(AutogradContext* ctx, const at::Tensor& x, const at::Tensor& f, const Optional& s,
                               const Optional& n, const RecPlan& p) {
    at::Tensor keep;
    variable_list out = recurrence_forward(p, dense(x), dense(f), dense(s), dense(n), &keep);
    ctx->set_materialize_grads(false);
    ctx->save_for_backward({x, f, s.value_or(at::Tensor()), n.value_or(at::Tensor()), keep});
    ctx->saved_data["plan"] = std::vector<int64_t>{p.batch, p.steps, p.channels, p.dtype};
    return out;
  }

  static variable_list backward(AutogradContext* ctx, const variable_list& grads) {
    const std::vector<int64_t> p = ctx->saved_data["plan"].toIntVector();
    const bool again = at::GradMode::is_enabled();
    at::AutoGradMode off(false);
    const variable_list saved = ctx->get_saved_variables();
    refuse_foreign_capture(ctx, saved, 3);
    variable_list in(3), wanted(3), out(5);
    for (int i = 0; i < 3; ++i) in[i] = dense(saved[i]);
    const at::Tensor &x = in[0], n = dense(saved[3]), gh = dense(grads[0]), gl = dense(grads[1]);
    const c10::DeviceGuard guard(x.device());
    const bool nothing = !x.numel() || (!gh.defined() && !gl.defined());
    const bool any = gradients(ctx, in, wanted, nothing);
    if (nothing && wanted[2].defined() && gl.defined()) wanted[2].copy_(gl);  // no steps: the state is the last one
    if (any && !nothing) {
      const int64_t bytes = ecc_gated_recurrence_workspace_bytes(p[0], p[1], p[2], (int)p[3]);
      at::Tensor ws = bytes_like(x, bytes);
      check(ecc_gated_recurrence_bwd(ptr(x), ptr(in[1]), (int)p[3], p[0], p[1], p[2],
                                     n.defined() ? n.const_data_ptr<int64_t>() : nullptr, saved[4].const_data_ptr<float>(),
                                     ptr(gh), gl.defined() ? gl.const_data_ptr<float>() : nullptr, out_ptr(wanted[0]),
                                     out_ptr(wanted[1]), wanted[2].defined() ? wanted[2].data_ptr<float>() : nullptr,
                                     ws.data_ptr(), bytes, stream_of(x)),
            "ecc_gated_recurrence_bwd");
    }
    for (int i = 0; i < 3; ++i) out[i] = wanted[i];
    if (again && any) return once_only(out, "gated recurrence");
    return out;
  }
};

std::tuple<at::Tensor, at::Tensor> gated_recurrence(const at::Tensor& x, const at::Tensor& f, const Optional& s,
                                                    const Optional& n) {
  refuse_tracing("gated recurrence");
  const pybind11::gil_scoped_release nogil;
  features(x, "x");
  TORCH_CHECK_VALUE(x.dim() == 3, "x must be [batch, steps, channels] (got ", x.sizes(), ")");
  TORCH_CHECK_VALUE(x.size(2) >= 1, "x has no channels");
  const c10::Device where = x.device();
  on_device(f, "gate", &where);
  TORCH_CHECK_TYPE(f.scalar_type() == x.scalar_type(), "gate must be ", x.scalar_type(), " (got ", f.scalar_type(), ")");
  TORCH_CHECK_VALUE(f.sizes() == x.sizes(), "gate must have x's shape ", x.sizes(), " (got ", f.sizes(), ")");
  const RecPlan p{x.size(0), x.size(1), x.size(2), type_of(x.scalar_type())};
  if (s) {
    on_device(*s, "state", &where);
    TORCH_CHECK_TYPE(s->scalar_type() == at::kFloat, "state must be torch.float32 (got ", s->scalar_type(), ")");
    TORCH_CHECK_VALUE(s->dim() == 2 && s->size(0) == p.batch && s->size(1) == p.channels, "state must be [", p.batch, ", ",
                      p.channels, "] (got ", s->sizes(), ")");
  }
  if (n) {
    on_device(*n, "lengths", &where);
    TORCH_CHECK_TYPE(n->scalar_type() == at::kLong, "lengths must be torch.int64 (got ", n->scalar_type(), ")");
    TORCH_CHECK_VALUE(n->dim() == 1 && n->size(0) == p.batch, "lengths must be [", p.batch, "] (got ", n->sizes(), ")");
  }
  TORCH_CHECK_NOT_IMPLEMENTED(!is_dual(x) && !is_dual(f) && !is_dual(s), "gated recurrence has no forward-mode derivative");
  variable_list out;
  if (at::GradMode::is_enabled() && (x.requires_grad() || f.requires_grad() || wants(s)))
    out = Recurrence::apply(x, f, s, n, p);
  else
    out = recurrence_forward(p, dense(x), dense(f), dense(s), dense(n), nullptr);
  return {out[0], out[1]};
}

}  // namespace

void define_block(pybind11::module_& m) {
  m.def("residual_norm", [](const at::Tensor& x, const at::Tensor& b, const Optional& g, const Optional& w,
                            const Optional& bw, double scale, double eps, bool norm_branch) {
    const variable_list out = residual_norm(x, b, g, w, bw, scale, eps, norm_branch, std::nullopt);
    return std::make_tuple(out[0], out[1]);
  });
  m.def("gated_linear", &gated_linear);
  m.def("gated_recurrence", &gated_recurrence);
  m.def("rms_norm", [](const at::Tensor& x, const Optional& w, double eps, const std::optional<at::ScalarType>& dtype) {
    return residual_norm(x, std::nullopt, std::nullopt, w, std::nullopt, 1.0, eps, false, dtype)[0];
  });
}

}  // namespace ecc_torch
