// The frame-encoder operators as functions on tensors: argument checks,
// outputs, workspaces, the current stream and autograd nodes around the C ABI
// of fm_ops.h. In C++ because the smallest calls take less time on the GPU than
// Python takes to prepare them; every computation is in libfm_mel.so.
#include <ATen/ATen.h>
#include <c10/core/AutogradState.h>
#include <c10/core/impl/TorchDispatchModeTLS.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/csrc/autograd/functions/utils.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/jit/frontend/tracer.h>

#include <cmath>
#include <map>
#include <mutex>
#include <tuple>

#include "fm_ops.h"

using at::Tensor;
using torch::autograd::AutogradContext;
using torch::autograd::variable_list;

namespace {

PyObject* g_fm_error = nullptr;  // the package's FmError class

// a status other than FM_OK; becomes FmError at the Python boundary
struct Failure : std::runtime_error {
  int status;
  Failure(int s, const char* call)
      : std::runtime_error(std::string(call) + ": " + fm_status_string((fm_status)s)), status(s) {}
};

int type_of(const Tensor& t, const char* name) {
  switch (t.scalar_type()) {
    case at::kFloat: return FM_F32;
    case at::kHalf: return FM_F16;
    case at::kBFloat16: return FM_BF16;
    default: break;
  }
  TORCH_CHECK_TYPE(false, name, ": dtype ", t.scalar_type(), " not supported (float32, float16, bfloat16)");
}
// A tensor's memory, NULL for an absent tensor. One without memory of its own (a
// fake tensor, a wrapper around others) is refused: the library would take it for
// absent.
template <typename P>
P* its_memory(P* p, const Tensor& t) {
  TORCH_CHECK_VALUE(p != nullptr || t.numel() == 0, "a tensor of ", t.numel(),
                    " elements has no memory of its own (a fake or wrapper tensor): the operators need the data");
  return p;
}
const void* ptr(const Tensor& t) { return t.defined() ? its_memory(t.const_data_ptr(), t) : nullptr; }
void* mut(const Tensor& t) { return t.defined() ? its_memory(t.mutable_data_ptr(), t) : nullptr; }

void need_cuda(const Tensor& t, const char* name, const Tensor& like) {
  if (!t.defined()) return;
  TORCH_CHECK_VALUE(t.is_cuda(), name, " must be a CUDA tensor (the operators run only on the GPU)");
  TORCH_CHECK_VALUE(t.get_device() == like.get_device(), name, " is on ", t.device(), ", the other inputs on ",
                    like.device());
}

// makes the tensor's device current for a call, and gives its current stream
struct OnDevice {
  c10::cuda::OptionalCUDAGuard guard;
  fm_stream_t stream;
  explicit OnDevice(const Tensor& t) {
    if (t.get_device() != c10::cuda::current_device()) guard.set_index(t.get_device());
    stream = (fm_stream_t)c10::cuda::getCurrentCUDAStream(t.get_device()).stream();
  }
};
void run(fm_status s, const char* call) {
  if (s != FM_OK) throw Failure(s, call);
}
Tensor bytes_on(const Tensor& t, int64_t n) {
  return at::empty({n}, t.options().dtype(at::kByte).requires_grad(false));
}
// autograd takes an absent input as an empty optional (it has no edge then)
using Maybe = std::optional<Tensor>;
Maybe maybe(const Tensor& t) { return t.defined() ? Maybe(t) : Maybe(); }
Tensor or_none(const Maybe& t) { return t ? *t : Tensor(); }
bool wants_grad(const Tensor& t) { return t.defined() && t.requires_grad(); }

// t with the signs that its values have: a view of a conjugate's imaginary part
// may hold them as a flag, which its memory does not show.
Tensor signed_as_is(const Tensor& t) { return t.defined() && t.is_neg() ? t.resolve_neg() : t; }

// Traces are refused: the calls are no operators of torch's own registry, so that
// a trace would hold their outputs' allocations, or one call's results, alone.
void no_trace(const char* name) {
  using c10::impl::TorchDispatchModeKey, c10::impl::TorchDispatchModeTLS;
  const bool traced = torch::jit::tracer::isTracing() || TorchDispatchModeTLS::get_mode(TorchDispatchModeKey::PROXY);
  TORCH_CHECK_NOT_IMPLEMENTED(!traced, name, " cannot be traced");
}

// Forward-mode derivatives are refused: a result without a tangent would read as
// one whose tangent is zero.
template <typename... Inputs>
void no_tangents(const char* name, const Inputs&... inputs) {
  if (!c10::AutogradState::get_tls_state().get_fw_grad_mode()) return;
  auto has = [](const Tensor& t) { return t.defined() && t._fw_grad(0).defined(); };
  TORCH_CHECK_NOT_IMPLEMENTED(!(has(inputs) || ...), name, " has no forward-mode derivative");
}

// What a backward pass returns where the caller asked for a graph of it: the
// gradients, whose own history is an error that leads to everything they were
// made `from`, so that whoever derives through them to one of those meets it.
template <typename... From>
variable_list once(variable_list out, const char* name, const From&... from) {
  using namespace torch::autograd;
  if (!compute_requires_grad(from...)) return out;  // also where no graph is wanted
  const std::shared_ptr<Node> error(
      new Error(std::string(name) + ": its gradient is differentiable once, no second gradient is built",
                collect_next_edges(from...)),
      deleteNode);
  for (Tensor& t : out)
    if (t.defined()) set_history(t, error);
  return out;
}

// ---- layer norm ---------------------------------------------------------------
// t as rows of `width` adjacent elements at one stride: a view where the
// strides allow one, a copy otherwise
std::pair<Tensor, int64_t> rows_of(const Tensor& t, int64_t width) {
  if (t.is_contiguous()) return {t, width};
  Tensor r = t.reshape({-1, width});
  if ((width > 1 && r.stride(1) != 1) || (r.size(0) > 1 && r.stride(0) < width)) r = r.contiguous();
  return {r, std::max(r.stride(0), width)};
}

std::tuple<Tensor, Tensor> norm_forward(const Tensor& x, const Tensor& weight, const Tensor& bias, double eps,
                                        bool stats) {
  const int64_t width = x.size(-1), rows = x.numel() / width;
  Tensor y = at::empty(x.sizes(), x.options().requires_grad(false).memory_format(at::MemoryFormat::Contiguous));
  auto [x2, xs] = rows_of(x, width);
  Tensor st;
  if (stats) st = at::empty({2, rows}, x.options().dtype(at::kFloat).requires_grad(false));
  fm_layer_norm_args a{};
  a.rows = rows, a.width = width;
  a.dtype = type_of(x, "x");
  a.param_dtype = weight.defined() ? type_of(weight, "weight") : bias.defined() ? type_of(bias, "bias") : a.dtype;
  a.x_stride = xs, a.y_stride = width;
  a.eps = eps;
  a.x = ptr(x2), a.weight = ptr(weight), a.bias = ptr(bias), a.y = mut(y);
  if (stats) a.mean = (float*)mut(st), a.rstd = a.mean + rows;
  OnDevice on(x);
  run(fm_layer_norm_forward(&a, on.stream), "fm_layer_norm_forward");
  return {y, st};
}

struct NormNode : torch::autograd::Function<NormNode> {
  static Tensor forward(AutogradContext* ctx, const Tensor& x, const Maybe& w, const Maybe& b, double eps) {
    const Tensor weight = or_none(w), bias = or_none(b);
    auto [y, st] = norm_forward(x, weight, bias, eps, true);
    ctx->save_for_backward({x, weight, st});
    ctx->saved_data["eps"] = eps;
    ctx->saved_data["has_bias"] = bias.defined();
    ctx->saved_data["bias_f32"] = bias.defined() && bias.scalar_type() == at::kFloat;
    return y;
  }
  static variable_list backward(AutogradContext* ctx, variable_list grads) {
    const auto saved = ctx->get_saved_variables();
    const Tensor &x = saved[0], &weight = saved[1], &st = saved[2];
    if (!grads[0].defined()) return {Tensor(), Tensor(), Tensor(), Tensor()};
    Tensor dx, dw, db;
    {
      at::NoGradGuard no_grad;
      const int64_t width = x.size(-1), rows = x.numel() / width;
      auto [x2, xs] = rows_of(x, width);
      auto [dy2, dys] = rows_of(signed_as_is(grads[0]), width);
      const auto options = x.options().requires_grad(false);
      const bool f32 = weight.defined() ? weight.scalar_type() == at::kFloat : ctx->saved_data["bias_f32"].toBool();
      const auto ptype = f32 ? options.dtype(at::kFloat) : options;
      if (ctx->needs_input_grad(0)) dx = at::empty(x.sizes(), options.memory_format(at::MemoryFormat::Contiguous));
      const bool has_weight = weight.defined(), has_bias = ctx->saved_data["has_bias"].toBool();
      if (has_weight && ctx->needs_input_grad(1)) dw = at::empty({width}, ptype);
      if (has_bias && ctx->needs_input_grad(has_weight ? 2 : 1)) db = at::empty({width}, ptype);
      fm_layer_norm_args a{};
      a.rows = rows, a.width = width;
      a.dtype = type_of(x, "x");
      a.param_dtype = f32 ? (int64_t)FM_F32 : a.dtype;
      a.x_stride = xs, a.dy_stride = dys, a.dx_stride = width;
      a.eps = ctx->saved_data["eps"].toDouble();
      a.x = ptr(x2), a.weight = ptr(weight), a.dy = ptr(dy2);
      a.mean = (float*)ptr(st), a.rstd = a.mean + rows;
      a.dx = mut(dx), a.dweight = mut(dw), a.dbias = mut(db);
      OnDevice on(x);
      Tensor work;
      if (dw.defined() || db.defined()) {
        a.workspace_bytes = fm_layer_norm_workspace(&a);
        work = bytes_on(x, a.workspace_bytes);
        a.workspace = mut(work);
      }
      run(fm_layer_norm_backward(&a, on.stream), "fm_layer_norm_backward");
    }
    return once({dx, dw, db, Tensor()}, "layer_norm", grads[0], x, weight);
  }
};

Tensor layer_norm(Tensor x, Tensor weight, Tensor bias, double eps) {
  no_trace("layer_norm");
  no_tangents("layer_norm", x, weight, bias);
  x = signed_as_is(x), weight = signed_as_is(weight), bias = signed_as_is(bias);
  TORCH_CHECK_VALUE(x.is_cuda(), "x must be a CUDA tensor (the operators run only on the GPU)");
  need_cuda(weight, "weight", x);
  need_cuda(bias, "bias", x);
  type_of(x, "x");
  TORCH_CHECK_VALUE(x.dim() >= 1 && x.size(-1) >= 1, "x needs a last dimension of at least one element");
  const int64_t width = x.size(-1);
  auto param = [&](Tensor& t, const char* name) {
    if (!t.defined()) return;
    TORCH_CHECK_VALUE(t.dim() == 1 && t.size(0) == width, name, " has shape ", t.sizes(), ", expected (", width, ",)");
    TORCH_CHECK_TYPE(t.scalar_type() == x.scalar_type() || t.scalar_type() == at::kFloat, name, ": dtype ",
                     t.scalar_type(), ", expected ", x.scalar_type(), " or float32");
    t = t.contiguous();
  };
  param(weight, "weight");
  param(bias, "bias");
  TORCH_CHECK_TYPE(!weight.defined() || !bias.defined() || weight.scalar_type() == bias.scalar_type(),
                   "weight and bias need the same dtype");
  TORCH_CHECK_VALUE(eps >= 0, "eps must not be negative");
  if (at::GradMode::is_enabled() && (wants_grad(x) || wants_grad(weight) || wants_grad(bias)))
    return NormNode::apply(x, maybe(weight), maybe(bias), eps);
  return std::get<0>(norm_forward(x, weight, bias, eps, false));
}

// ---- distance buckets -----------------------------------------------------------
// One map per device and configuration, made once and kept (a few kilobytes).
fm_buckets* buckets_for(const c10::Device& device, int64_t num, int64_t far, bool both) {
  static std::mutex mu;
  static std::map<std::tuple<int, int64_t, int64_t, bool>, fm_buckets*> known;
  std::lock_guard<std::mutex> lock(mu);
  fm_buckets*& b = known[{(int)device.index(), num, far, both}];
  if (b == nullptr) {
    c10::cuda::CUDAGuard guard(device);
    const auto fits = [](int64_t v) { return (int)std::min<int64_t>(std::max<int64_t>(v, -1), 1 << 30); };
    const fm_status s = fm_buckets_create(&b, fits(num), fits(far), both);
    TORCH_CHECK_VALUE(s != FM_ERR_INVALID_ARG, num, " buckets up to distance ", far,
                      ": needs 2 to 4096 buckets (even and at least 4 where bidirectional) and a max_distance of at "
                      "most 2048 that is beyond the buckets of single distances");
    run(s, "fm_buckets_create");
  }
  return b;
}

void check_table(const Tensor& table) {
  TORCH_CHECK_VALUE(table.dim() == 2, "table has shape ", table.sizes(), ", expected (num_buckets, heads)");
  type_of(table, "table");
}

Tensor bias_forward(const Tensor& table, const fm_buckets* b, int64_t q_len, int64_t k_len, int64_t q_start) {
  Tensor out = at::empty({table.size(1), q_len, k_len}, table.options().requires_grad(false));
  fm_relative_bias_args a{};
  a.heads = table.size(1), a.q_len = q_len, a.k_len = k_len, a.q_start = q_start;
  a.dtype = type_of(table, "table");
  a.buckets = b;
  a.table = ptr(table), a.out = mut(out);
  OnDevice on(table);
  run(fm_relative_bias_forward(&a, on.stream), "fm_relative_bias_forward");
  return out;
}

struct BiasNode : torch::autograd::Function<BiasNode> {
  static Tensor forward(AutogradContext* ctx, const Tensor& table, int64_t handle, int64_t q_len, int64_t k_len,
                        int64_t q_start) {
    ctx->saved_data["args"] = std::vector<int64_t>{handle, q_len, k_len, q_start, table.size(0), table.size(1)};
    return bias_forward(table, (const fm_buckets*)handle, q_len, k_len, q_start);
  }
  static variable_list backward(AutogradContext* ctx, variable_list grads) {
    if (!grads[0].defined()) return {Tensor(), Tensor(), Tensor(), Tensor(), Tensor()};
    const auto v = ctx->saved_data["args"].toIntVector();
    Tensor dtable;
    {
      at::NoGradGuard no_grad;
      const Tensor dout = signed_as_is(grads[0]).contiguous();
      dtable = at::empty({v[4], v[5]}, dout.options().requires_grad(false));
      fm_relative_bias_args a{};
      a.heads = v[5], a.q_len = v[1], a.k_len = v[2], a.q_start = v[3];
      a.dtype = type_of(dout, "gradient");
      a.buckets = (const fm_buckets*)v[0];
      a.dout = ptr(dout), a.dtable = mut(dtable);
      a.workspace_bytes = fm_relative_bias_workspace(&a);
      const Tensor work = bytes_on(dout, std::max<int64_t>(a.workspace_bytes, 0));
      a.workspace = mut(work);
      OnDevice on(dout);
      run(fm_relative_bias_backward(&a, on.stream), "fm_relative_bias_backward");
    }
    // linear in the gradient that came in, whatever the table holds
    return once({dtable, Tensor(), Tensor(), Tensor(), Tensor()}, "relative_bias", grads[0]);
  }
};

Tensor relative_bias(Tensor table, int64_t q_len, int64_t k_len, int64_t q_start, int64_t far, bool both) {
  no_trace("relative_bias");
  no_tangents("relative_bias", table);
  table = signed_as_is(table);
  TORCH_CHECK_VALUE(table.is_cuda(), "table must be a CUDA tensor (the operators run only on the GPU)");
  check_table(table);
  TORCH_CHECK_VALUE(q_len >= 0 && k_len >= 0, "q_len and k_len must not be negative");
  const fm_buckets* b = buckets_for(table.device(), table.size(0), far, both);
  table = table.contiguous();
  if (at::GradMode::is_enabled() && table.requires_grad())
    return BiasNode::apply(table, (int64_t)b, q_len, k_len, q_start);
  return bias_forward(table, b, q_len, k_len, q_start);
}

// ---- attention ------------------------------------------------------------------
// What one call's passes share besides q, k, v and the table.
struct Call : torch::CustomClassHolder {
  double scale, softcap;
  bool causal;
  int64_t start_all;
  const fm_buckets* buckets = nullptr;
};
// The masks and slopes: like q, k and v saved for the backward pass, which
// would otherwise answer for what has been written over them since.
struct Masks {
  Tensor slopes, q_docs, k_docs, k_lens, q_start, prefix;
};

void set_strides(int64_t (&to)[3], const Tensor& t) { to[0] = t.stride(0), to[1] = t.stride(1), to[2] = t.stride(2); }

fm_attention_args attention_args(const Call& c, const Masks& m, const Tensor& q, const Tensor& k, const Tensor& v,
                                 const Tensor& out, const Tensor& rest, const Tensor& lse, const Tensor& table) {
  fm_attention_args a{};
  a.batch = q.size(0), a.q_len = q.size(1), a.k_len = k.size(1);
  a.heads = q.size(2), a.kv_heads = k.size(2), a.dim = q.size(3);
  a.dtype = type_of(q, "q");
  a.causal = c.causal;
  a.scale = c.scale, a.softcap = c.softcap;
  a.q = ptr(q), a.k = ptr(k), a.v = ptr(v), a.out = mut(out);
  set_strides(a.q_s, q);
  set_strides(a.k_s, k);
  set_strides(a.v_s, v);
  set_strides(a.out_s, out);
  a.lse = (float*)mut(lse);
  a.out_rest = mut(rest);
  a.q_docs = (const int32_t*)ptr(m.q_docs), a.k_docs = (const int32_t*)ptr(m.k_docs);
  a.k_lens = (const int32_t*)ptr(m.k_lens), a.q_start = (const int32_t*)ptr(m.q_start);
  a.prefix = (const int32_t*)ptr(m.prefix);
  a.q_start_all = c.start_all;
  a.buckets = c.buckets;
  if (table.defined()) a.table = ptr(table), a.table_dtype = type_of(table, "table");
  a.slopes = (const float*)ptr(m.slopes);
  return a;
}

void workspace_for(fm_attention_args& a, int backward, const Tensor& like, Tensor& work) {
  a.workspace_bytes = fm_attention_workspace(&a, backward);
  if (a.workspace_bytes > 0) {
    work = bytes_on(like, a.workspace_bytes);
    a.workspace = mut(work);
  }
}

// rest: what rounding took from the output (16-bit types, where a backward
// pass will want its exact product with the gradient)
std::tuple<Tensor, Tensor, Tensor> attention_forward(const Call& c, const Masks& m, const Tensor& q, const Tensor& k,
                                                     const Tensor& v, const Tensor& table, bool want_lse,
                                                     bool want_rest) {
  const auto options = q.options().requires_grad(false);
  Tensor out = at::empty(q.sizes(), options.memory_format(at::MemoryFormat::Contiguous)), rest, lse;
  if (want_rest && q.scalar_type() != at::kFloat)
    rest = at::empty(q.sizes(), options.memory_format(at::MemoryFormat::Contiguous));
  if (want_lse) lse = at::empty({q.size(0), q.size(2), q.size(1)}, options.dtype(at::kFloat));
  fm_attention_args a = attention_args(c, m, q, k, v, out, rest, lse, table);
  OnDevice on(q);
  Tensor work;
  workspace_for(a, 0, q, work);
  run(fm_attention_forward(&a, on.stream), "fm_attention_forward");
  return {out, rest, lse};
}

// the gradient arrives in any layout: the kernels want the elements of a
// token's head adjacent, and tokens apart
Tensor gradient_rows(const Tensor& t) {
  if (t.stride(3) != 1) return t.contiguous();
  for (int d = 0; d < 3; ++d)
    if (t.size(d) > 1 && t.stride(d) <= 0) return t.contiguous();
  return t;
}

struct AttentionNode : torch::autograd::Function<AttentionNode> {
  static variable_list forward(AutogradContext* ctx, const Tensor& q, const Tensor& k, const Tensor& v,
                               const Maybe& maybe_table, const c10::intrusive_ptr<Call>& c, const Masks& m) {
    const Tensor table = or_none(maybe_table);
    auto [out, rest, lse] = attention_forward(*c, m, q, k, v, table, true, true);
    ctx->save_for_backward({q, k, v, table, out, rest, lse, m.slopes, m.q_docs, m.k_docs, m.k_lens, m.q_start,
                            m.prefix});
    ctx->saved_data["call"] = c10::IValue::make_capsule(c);
    ctx->mark_non_differentiable({lse});
    ctx->set_materialize_grads(false);
    return {out, lse};
  }
  static variable_list backward(AutogradContext* ctx, variable_list grads) {
    if (!grads[0].defined()) return {Tensor(), Tensor(), Tensor(), Tensor(), Tensor(), Tensor()};
    const auto saved = ctx->get_saved_variables();
    const Masks m{saved[7], saved[8], saved[9], saved[10], saved[11], saved[12]};
    const Tensor &q = saved[0], &k = saved[1], &v = saved[2], &table = saved[3];
    const auto capsule = ctx->saved_data["call"].toCapsule();
    const Call& c = *static_cast<Call*>(capsule.get());
    Tensor dq, dk, dv, dtable;
    {
      at::NoGradGuard no_grad;
      const Tensor dout = gradient_rows(signed_as_is(grads[0]));
      const auto dense = q.options().requires_grad(false).memory_format(at::MemoryFormat::Contiguous);
      dq = at::empty(q.sizes(), dense);
      dk = at::empty(k.sizes(), dense);
      dv = at::empty(v.sizes(), dense);
      if (table.defined() && ctx->needs_input_grad(3)) dtable = at::empty(table.sizes(), table.options().requires_grad(false));
      fm_attention_args a = attention_args(c, m, q, k, v, saved[4], saved[5], saved[6], table);
      a.dout = ptr(dout), a.dq = mut(dq), a.dk = mut(dk), a.dv = mut(dv), a.dtable = mut(dtable);
      set_strides(a.dout_s, dout);
      set_strides(a.dq_s, dq);
      set_strides(a.dk_s, dk);
      set_strides(a.dv_s, dv);
      OnDevice on(q);
      Tensor work;
      workspace_for(a, 1, q, work);
      run(fm_attention_backward(&a, on.stream), "fm_attention_backward");
    }
    return once({dq, dk, dv, dtable, Tensor(), Tensor()}, "attention", grads[0], q, k, v, table);
  }
};

Tensor int32_of(const Tensor& t, const char* name, at::IntArrayRef shape, const Tensor& q) {
  if (!t.defined()) return t;
  need_cuda(t, name, q);
  TORCH_CHECK_TYPE(t.scalar_type() == at::kInt, name, ": dtype ", t.scalar_type(), ", expected int32");
  TORCH_CHECK_VALUE(t.sizes() == shape, name, " has shape ", t.sizes(), ", expected ", shape);
  return signed_as_is(t).contiguous();
}

std::tuple<Tensor, Tensor> attention(Tensor q, Tensor k, Tensor v, Tensor table, const c10::intrusive_ptr<Call>& c,
                                     Masks m, int64_t far, bool both, bool want_lse) {
  no_trace("attention");
  no_tangents("attention", q, k, v, table, m.slopes);
  q = signed_as_is(q), k = signed_as_is(k), v = signed_as_is(v), table = signed_as_is(table);
  m.slopes = signed_as_is(m.slopes);
  TORCH_CHECK_VALUE(q.is_cuda(), "q must be a CUDA tensor (the operators run only on the GPU)");
  need_cuda(k, "k", q);
  need_cuda(v, "v", q);
  need_cuda(table, "table", q);
  need_cuda(m.slopes, "slopes", q);
  type_of(q, "q");
  TORCH_CHECK_TYPE(k.scalar_type() == q.scalar_type() && v.scalar_type() == q.scalar_type(),
                   "q, k and v need one dtype, got ", q.scalar_type(), ", ", k.scalar_type(), ", ", v.scalar_type());
  TORCH_CHECK_VALUE(q.dim() == 4 && k.dim() == 4 && k.sizes() == v.sizes(), "q, k, v have shapes ", q.sizes(), ", ",
                    k.sizes(), ", ", v.sizes(),
                    "; expected (batch, q_len, heads, dim) and twice (batch, k_len, kv_heads, dim)");
  const int64_t B = q.size(0), Tq = q.size(1), H = q.size(2), D = q.size(3), Tk = k.size(1), Hk = k.size(2);
  TORCH_CHECK_VALUE(k.size(0) == B && k.size(3) == D && D >= 1 && Hk >= 1 && H >= 1 && H % Hk == 0, "q ", q.sizes(),
                    " does not fit k and v ", k.sizes(), ": same batch and dim, heads a multiple of the keys' heads");
  TORCH_CHECK_VALUE(D <= 256, "dim ", D, " is not supported (at most 256)");
  if (std::isnan(c->scale)) c->scale = 1.0 / std::sqrt((double)D);
  TORCH_CHECK_VALUE(std::isfinite(c->scale) && c->softcap >= 0 && std::isfinite(c->softcap),
                    "scale must be finite, softcap finite and not negative");
  TORCH_CHECK_VALUE(!m.prefix.defined() || c->causal, "prefix needs causal=True");
  TORCH_CHECK_VALUE(m.q_docs.defined() == m.k_docs.defined(), "q_docs and k_docs go together");
  m.q_docs = int32_of(m.q_docs, "q_docs", {B, Tq}, q);
  m.k_docs = int32_of(m.k_docs, "k_docs", {B, Tk}, q);
  m.k_lens = int32_of(m.k_lens, "k_lens", {B}, q);
  m.prefix = int32_of(m.prefix, "prefix", {B}, q);
  m.q_start = int32_of(m.q_start, "q_start", {B}, q);
  const bool grad = at::GradMode::is_enabled();
  if (m.slopes.defined()) {
    TORCH_CHECK_VALUE(m.slopes.scalar_type() == at::kFloat && m.slopes.dim() == 1 && m.slopes.size(0) == H,
                      "slopes must be float32 of shape (", H, ",)");
    TORCH_CHECK(!(grad && m.slopes.requires_grad()), "slopes are constants: no gradient is computed for them");
    m.slopes = m.slopes.contiguous();
  }
  if (table.defined()) {
    check_table(table);
    TORCH_CHECK_VALUE(table.size(1) == H, "table has ", table.size(1), " heads, q has ", H);
    TORCH_CHECK_TYPE(table.scalar_type() == q.scalar_type() || table.scalar_type() == at::kFloat, "table: dtype ",
                     table.scalar_type(), ", expected ", q.scalar_type(), " or float32");
    c->buckets = buckets_for(q.device(), table.size(0), far, both);
    table = table.contiguous();
  }
  auto rows = [](Tensor& t) {
    if (t.size(3) > 1 && t.stride(3) != 1) t = t.contiguous();
  };
  rows(q);
  rows(k);
  rows(v);
  if (grad && (wants_grad(q) || wants_grad(k) || wants_grad(v) || wants_grad(table))) {
    auto r = AttentionNode::apply(q, k, v, maybe(table), c, m);
    return {r[0], r[1]};
  }
  auto [out, rest, lse] = attention_forward(*c, m, q, k, v, table, want_lse, false);
  return {out, lse};
}

// ---- Python ---------------------------------------------------------------------
Tensor tensor_arg(PyObject* o, const char* name, bool optional) {
  if (optional && o == Py_None) return Tensor();
  TORCH_CHECK_VALUE(THPVariable_Check(o), name, " must be a CUDA tensor (the operators run only on the GPU)");
  return THPVariable_Unpack(o);
}
double real_arg(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}
int64_t whole_arg(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
bool flag_arg(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();  // it has no truth value
  return v != 0;
}
void count_args(Py_ssize_t got, Py_ssize_t want) {
  TORCH_CHECK_TYPE(got == want, "expected ", want, " arguments, got ", got);
}
struct NoGil {
  PyThreadState* state = PyEval_SaveThread();
  ~NoGil() { PyEval_RestoreThread(state); }
};
PyObject* raise(const Failure& e) {
  PyObject* args = Py_BuildValue("(is)", e.status, e.what());
  PyObject* v = args && g_fm_error ? PyObject_CallObject(g_fm_error, args) : nullptr;
  Py_XDECREF(args);
  if (v) PyErr_SetObject(g_fm_error, v);
  else if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  Py_XDECREF(v);
  return nullptr;
}

PyObject* py_layer_norm(PyObject*, PyObject* const* v, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    count_args(n, 4);
    const Tensor x = tensor_arg(v[0], "x", false), w = tensor_arg(v[1], "weight", true), b = tensor_arg(v[2], "bias", true);
    const double eps = real_arg(v[3]);
    Tensor y;
    {
      NoGil free;
      y = layer_norm(x, w, b, eps);
    }
    return THPVariable_Wrap(y);
  } catch (const Failure& e) {
    return raise(e);
  }
  END_HANDLE_TH_ERRORS
}

PyObject* py_relative_bias(PyObject*, PyObject* const* v, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    count_args(n, 6);
    const Tensor table = tensor_arg(v[0], "table", false);
    const int64_t q = whole_arg(v[1]), k = whole_arg(v[2]);
    const int64_t start = v[3] == Py_None ? k - q : whole_arg(v[3]), far = whole_arg(v[4]);
    const bool both = flag_arg(v[5]);
    Tensor y;
    {
      NoGil free;
      y = relative_bias(table, q, k, start, far, both);
    }
    return THPVariable_Wrap(y);
  } catch (const Failure& e) {
    return raise(e);
  }
  END_HANDLE_TH_ERRORS
}

// q, k, v, scale, causal, prefix, softcap, table, max_distance, bidirectional,
// slopes, q_docs, k_docs, k_lens, q_start, return_lse
PyObject* py_attention(PyObject*, PyObject* const* v, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    count_args(n, 16);
    const Tensor q = tensor_arg(v[0], "q", false), k = tensor_arg(v[1], "k", false), w = tensor_arg(v[2], "v", false);
    auto c = c10::make_intrusive<Call>();
    Masks m;
    c->scale = v[3] == Py_None ? NAN : real_arg(v[3]);
    TORCH_CHECK_VALUE(v[3] == Py_None || std::isfinite(c->scale), "scale must be finite");
    c->causal = flag_arg(v[4]);
    m.prefix = tensor_arg(v[5], "prefix", true);
    c->softcap = real_arg(v[6]);
    const Tensor table = tensor_arg(v[7], "table", true);
    const int64_t far = whole_arg(v[8]);
    const bool both = flag_arg(v[9]), want_lse = flag_arg(v[15]);
    m.slopes = tensor_arg(v[10], "slopes", true);
    m.q_docs = tensor_arg(v[11], "q_docs", true);
    m.k_docs = tensor_arg(v[12], "k_docs", true);
    m.k_lens = tensor_arg(v[13], "k_lens", true);
    c->start_all = FM_Q_START_END;
    if (THPVariable_Check(v[14])) m.q_start = THPVariable_Unpack(v[14]);
    else if (v[14] != Py_None)
      c->start_all = std::max<int64_t>(-((int64_t)1 << 40), std::min<int64_t>((int64_t)1 << 40, whole_arg(v[14])));
    Tensor out, lse;
    {
      NoGil free;
      std::tie(out, lse) = attention(q, k, w, table, c, m, far, both, want_lse);
    }
    if (!want_lse) return THPVariable_Wrap(out);
    PyObject *a = THPVariable_Wrap(out), *b = THPVariable_Wrap(lse);
    PyObject* both_out = a && b ? PyTuple_Pack(2, a, b) : nullptr;
    Py_XDECREF(a);
    Py_XDECREF(b);
    return both_out;
  } catch (const Failure& e) {
    return raise(e);
  }
  END_HANDLE_TH_ERRORS
}

// device index, num_buckets, max_distance, bidirectional -> handle
PyObject* py_buckets(PyObject*, PyObject* const* v, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    count_args(n, 4);
    const c10::Device device(c10::kCUDA, (c10::DeviceIndex)whole_arg(v[0]));
    const int64_t num = whole_arg(v[1]), far = whole_arg(v[2]);
    return PyLong_FromVoidPtr(buckets_for(device, num, far, flag_arg(v[3])));
  } catch (const Failure& e) {
    return raise(e);
  }
  END_HANDLE_TH_ERRORS
}

PyObject* py_set_error(PyObject*, PyObject* type) {
  Py_INCREF(type);
  Py_XDECREF(g_fm_error);
  g_fm_error = type;
  Py_RETURN_NONE;
}

PyMethodDef kMethods[] = {
    {"layer_norm", (PyCFunction)(void (*)())py_layer_norm, METH_FASTCALL, nullptr},
    {"relative_bias", (PyCFunction)(void (*)())py_relative_bias, METH_FASTCALL, nullptr},
    {"attention", (PyCFunction)(void (*)())py_attention, METH_FASTCALL, nullptr},
    {"buckets", (PyCFunction)(void (*)())py_buckets, METH_FASTCALL, nullptr},
    {"set_error", py_set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_fm_torch", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};
}  // namespace

PyMODINIT_FUNC PyInit__fm_torch() { return PyModule_Create(&kModule); }
