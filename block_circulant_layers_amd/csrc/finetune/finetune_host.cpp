// finetune_host.cpp -- Python module _finetune_host: the calls of finetune.h on
// torch tensors.
//
// Argument marshalling only: checks of dtypes, shapes and devices, outputs and
// workspaces from torch's allocator, the current stream of the tensors' device.
// A pass over a few kilobytes takes the GPU 3 us; the same marshalling through
// ctypes took the host 16 us a call, most of it allocation, stream lookup and
// shape objects made in Python.
#include "host.hpp"

namespace finetune_host {
void define_attention(pybind11::module_& m);  // attention_host.cpp
}

namespace {

using namespace finetune_host;

// ---- layer normalisation --------------------------------------------------

std::tuple<Tensor, Tensor, Tensor> layer_norm_fwd_(const Tensor& x, const Opt& weight, const Opt& bias, double eps,
                                                   const Opt& y) {
  const RowsOf r = rows_of("x", x);
  const int code = dtype_code(x);
  const float* w = f32("weight", weight, {r.d}, x);
  const float* b = f32("bias", bias, {r.d}, x);
  const int64_t ys = y ? same_rows("y", *y, x) : r.d;
  const c10::DeviceGuard guard(x.device());
  Tensor out = y ? *y : at::empty(x.sizes(), x.options());
  const auto lead = x.sizes().slice(0, x.dim() - 1);
  Results res(x, {r.rows, r.rows});
  Tensor mean = res.next(lead), rstd = res.next(lead);
  check("layer_norm_fwd",
        layer_norm_fwd(x.data_ptr(), w, b, out.data_ptr(), static_cast<float*>(mean.data_ptr()),
                       static_cast<float*>(rstd.data_ptr()), r.rows, r.d, r.stride, ys, eps, code, stream_of(x)));
  written(y);
  return {out, mean, rstd};
}

std::tuple<Opt, Opt, Opt> layer_norm_bwd_(const Tensor& x, const Opt& weight, const Tensor& mean, const Tensor& rstd,
                                          const Tensor& dy, const Opt& dx, const Opt& dw, const Opt& db, bool need_dx,
                                          bool need_dw, bool need_db, const Opt& ws) {
  const RowsOf r = rows_of("x", x);
  const int code = dtype_code(x);
  const int64_t dys = same_rows("dy", dy, x);
  const float* w = f32("weight", weight, {r.d}, x);
  const auto lead = x.sizes().slice(0, x.dim() - 1);
  const float* m = f32("mean", mean, lead, x);
  const float* s = f32("rstd", rstd, lead, x);
  const int64_t dxs = need_dx && dx ? same_rows("dx", *dx, x) : r.d;
  f32("dw", dw, {r.d}, x);
  f32("db", db, {r.d}, x);
  const c10::DeviceGuard guard(x.device());
  Opt odx, odw, odb;
  if (need_dx) odx = dx ? *dx : at::empty(x.sizes(), x.options());
  if (need_dw) odw = dw ? *dw : new_f32({r.d}, x);
  if (need_db) odb = db ? *db : new_f32({r.d}, x);
  std::optional<Workspace> work;
  if (need_dw || need_db) {
    int64_t need = 0;
    check("layer_norm_bwd_workspace", layer_norm_bwd_workspace(r.rows, r.d, &need));
    work.emplace(x, need, ws);
  }
  const auto ptr = [](const Opt& t) { return t ? t->data_ptr() : nullptr; };
  check("layer_norm_bwd",
        layer_norm_bwd(x.data_ptr(), w, m, s, dy.data_ptr(), ptr(odx), static_cast<float*>(ptr(odw)),
                       static_cast<float*>(ptr(odb)), work ? work->p() : nullptr, work ? work->bytes() : 0, r.rows,
                       r.d, r.stride, dys, dxs, code, stream_of(x)));
  if (need_dx) written(dx);
  if (need_dw) written(dw);
  if (need_db) written(db);
  return {odx, odw, odb};
}

// ---- logits ---------------------------------------------------------------

finetune_logits logits_of(const Tensor& logits, const Tensor& labels) {
  check_gpu(logits);
  check_gpu(labels);
  CHECK_VALUE(logits.dim() == 3, "logits must have shape (sequences, positions, vocabulary)");
  const int64_t n = logits.size(0), t = logits.size(1), v = logits.size(2);
  CHECK_VALUE(labels.scalar_type() == at::kLong && labels.dim() == 2 && labels.size(0) == n && labels.size(1) == t,
              "labels must be int64 of shape (sequences, positions)");
  CHECK_VALUE(labels.device() == logits.device(), "tensors must be on one device");
  CHECK_VALUE(labels.is_contiguous(), "labels must be contiguous");
  CHECK_VALUE(logits.stride(2) == 1 || v <= 1, "the vocabulary axis of logits must be contiguous");
  return {logits.data_ptr(),  static_cast<const int64_t*>(labels.data_ptr()), n, t, v, logits.stride(0),
          logits.stride(1), dtype_code(logits)};
}

// the gradient's buffer, checked before anything is allocated
void check_dlogits(const Tensor& logits, const Opt& out) {
  if (!out) return;
  CHECK_VALUE(out->sizes() == logits.sizes() && out->scalar_type() == logits.scalar_type() &&
                  out->device() == logits.device(),
              "dlogits must have the shape, dtype and device of logits");
  CHECK_VALUE(out->stride(2) == 1 || out->size(2) <= 1, "the vocabulary axis of dlogits must be contiguous");
}
Tensor dlogits_of(const Tensor& logits, const Opt& out) {
  return out ? *out : at::empty(logits.sizes(), logits.options());
}
finetune_dlogits dlogits_args(const Tensor& out) { return {out.data_ptr(), out.stride(0), out.stride(1)}; }

// the caller's workspace or a new one of the size the call needs
Workspace logits_workspace(const Tensor& logits, const finetune_logits& in, const Opt& ws) {
  int64_t need = 0;
  if (!ws) check("finetune_logits_workspace", finetune_logits_workspace(&in, &need));
  return Workspace(logits, need, ws);
}

std::tuple<Tensor, Tensor> token_logprob_(const Tensor& logits, const Tensor& labels, const Opt& ws) {
  const finetune_logits in = logits_of(logits, labels);
  const c10::DeviceGuard guard(logits.device());
  const Workspace work = logits_workspace(logits, in, ws);
  const int64_t rows = labels.numel();
  Results res(logits, {rows, rows});
  Tensor logp = res.next(labels.sizes()), lse = res.next(labels.sizes());
  check("token_logprob", token_logprob(&in, ptr(logp), ptr(lse), work.p(), work.bytes(), stream_of(logits)));
  return {logp, lse};
}

Tensor token_logprob_bwd_(const Tensor& logits, const Tensor& labels, const Tensor& lse, const Tensor& dlogp,
                          const Opt& dlogits) {
  const finetune_logits in = logits_of(logits, labels);
  const float *l = f32("lse", lse, labels.sizes(), logits), *d = f32("dlogp", dlogp, labels.sizes(), logits);
  check_dlogits(logits, dlogits);
  const c10::DeviceGuard guard(logits.device());
  Tensor out = dlogits_of(logits, dlogits);
  const finetune_dlogits args = dlogits_args(out);
  check("token_logprob_bwd", token_logprob_bwd(&in, l, d, &args, stream_of(logits)));
  written(dlogits);
  return out;
}

// forward (scale absent) or step; returns loss, logratio, logp, lse, slope and the gradient or None
std::tuple<Tensor, Tensor, Tensor, Tensor, Tensor, Opt> preference_loss_(
    const Tensor& logits, const Tensor& labels, const Tensor& ref_logp, double beta, int64_t kind, double smoothing,
    bool average, std::optional<double> scale, const Opt& dlogits, const Opt& ws) {
  const finetune_logits in = logits_of(logits, labels);
  CHECK_VALUE(in.seqs % 2 == 0, "logits hold the chosen sequences and then as many rejected ones");
  const float* ref = f32("ref_logp", ref_logp, labels.sizes(), logits);
  check_dlogits(logits, dlogits);
  const c10::DeviceGuard guard(logits.device());
  const Workspace work = logits_workspace(logits, in, ws);
  const int64_t rows = labels.numel();
  Results res(logits, {in.seqs / 2, in.seqs, in.seqs, rows, rows});
  Tensor loss = res.next({in.seqs / 2}), ratio = res.next({in.seqs}), slope = res.next({in.seqs}),
         logp = res.next(labels.sizes()), lse = res.next(labels.sizes());
  const finetune_preference how{kind, average, beta, smoothing};
  if (!scale) {
    check("preference_loss_fwd", preference_loss_fwd(&in, ref, &how, ptr(loss), ptr(ratio), ptr(logp), ptr(lse),
                                                     ptr(slope), work.p(), work.bytes(), stream_of(logits)));
    return {loss, ratio, logp, lse, slope, std::nullopt};
  }
  Tensor out = dlogits_of(logits, dlogits);
  const finetune_dlogits args = dlogits_args(out);
  check("preference_loss_step",
        preference_loss_step(&in, ref, &how, *scale, ptr(loss), ptr(ratio), ptr(logp), ptr(lse), ptr(slope), &args,
                             work.p(), work.bytes(), stream_of(logits)));
  written(dlogits);
  return {loss, ratio, logp, lse, slope, out};
}

Tensor preference_loss_bwd_(const Tensor& logits, const Tensor& labels, const Tensor& lse, const Tensor& slope,
                            const Tensor& dloss, const Opt& dlogits) {
  const finetune_logits in = logits_of(logits, labels);
  const float *l = f32("lse", lse, labels.sizes(), logits), *s = f32("slope", slope, {in.seqs}, logits),
              *d = f32("dloss", dloss, {in.seqs / 2}, logits);
  check_dlogits(logits, dlogits);
  const c10::DeviceGuard guard(logits.device());
  Tensor out = dlogits_of(logits, dlogits);
  const finetune_dlogits args = dlogits_args(out);
  check("preference_loss_bwd", preference_loss_bwd(&in, l, s, d, &args, stream_of(logits)));
  written(dlogits);
  return out;
}

// forward (scale absent) or step; returns loss, kl, logp, lse, slope and the gradient or None
std::tuple<Tensor, Tensor, Tensor, Tensor, Tensor, Opt> policy_loss_(
    const Tensor& logits, const Tensor& labels, const Tensor& old_logp, const Tensor& advantages, const Opt& ref_logp,
    double clip_low, double clip_high, double kl_coef, int64_t reduction, std::optional<double> scale,
    const Opt& dlogits, const Opt& ws) {
  const finetune_logits in = logits_of(logits, labels);
  const float* old = f32("old_logp", old_logp, labels.sizes(), logits);
  const float* ref = f32("ref_logp", ref_logp, labels.sizes(), logits);
  const bool per_token = advantages.dim() == 2 && advantages.sizes() == labels.sizes();
  CHECK_VALUE(per_token || (advantages.dim() == 1 && advantages.size(0) == in.seqs) ||
                  (advantages.dim() == 2 && advantages.size(0) == in.seqs && advantages.size(1) == 1),
              "advantages must have shape (sequences,), (sequences, 1) or (sequences, positions)");
  const float* adv = f32("advantages", advantages, advantages.sizes(), logits);
  check_dlogits(logits, dlogits);
  const c10::DeviceGuard guard(logits.device());
  const Workspace work = logits_workspace(logits, in, ws);
  const int64_t rows = labels.numel();
  Results res(logits, {1, 1, rows, rows, rows});
  Tensor loss = res.next({}), kl = res.next({}),  // next to each other: the call's stats
      logp = res.next(labels.sizes()), lse = res.next(labels.sizes()), slope = res.next(labels.sizes());
  const finetune_policy how{reduction, per_token, clip_low, clip_high, kl_coef};
  if (!scale) {
    check("policy_loss_fwd", policy_loss_fwd(&in, old, ref, adv, &how, ptr(loss), ptr(logp), ptr(lse), ptr(slope),
                                             work.p(), work.bytes(), stream_of(logits)));
    return {loss, kl, logp, lse, slope, std::nullopt};
  }
  Tensor out = dlogits_of(logits, dlogits);
  const finetune_dlogits args = dlogits_args(out);
  check("policy_loss_step",
        policy_loss_step(&in, old, ref, adv, &how, *scale, ptr(loss), ptr(logp), ptr(lse), ptr(slope), &args,
                         work.p(), work.bytes(), stream_of(logits)));
  written(dlogits);
  return {loss, kl, logp, lse, slope, out};
}

Tensor policy_loss_bwd_(const Tensor& logits, const Tensor& labels, const Tensor& lse, const Tensor& slope,
                        const Tensor& dloss, const Opt& dlogits) {
  const finetune_logits in = logits_of(logits, labels);
  const float *l = f32("lse", lse, labels.sizes(), logits), *s = f32("slope", slope, labels.sizes(), logits);
  CHECK_VALUE(dloss.numel() == 1, "dloss must hold one value");
  const float* d = f32("dloss", dloss, dloss.sizes(), logits);
  check_dlogits(logits, dlogits);
  const c10::DeviceGuard guard(logits.device());
  Tensor out = dlogits_of(logits, dlogits);
  const finetune_dlogits args = dlogits_args(out);
  check("policy_loss_bwd", policy_loss_bwd(&in, l, s, d, &args, stream_of(logits)));
  written(dlogits);
  return out;
}

// ---- gradient tensors -----------------------------------------------------

// the tensors of a Python list, by reference
struct TensorList {
  PyObject* list;
  explicit TensorList(const py::list& l) : list(l.ptr()) {}
  size_t size() const { return static_cast<size_t>(PyList_GET_SIZE(list)); }
  const Tensor& operator[](size_t i) const {
    PyObject* o = PyList_GET_ITEM(list, static_cast<Py_ssize_t>(i));
    TORCH_CHECK_TYPE(THPVariable_Check(o), "gradients must be tensors");
    return THPVariable_Unpack(o);
  }
};

// max_norm absent: the norm alone.  `out` absent: in place.
Tensor clip_grad_norm_(const py::list& grad_list, std::optional<double> max_norm, double eps,
                       const std::optional<py::list>& out_list, const Opt& norm, const Opt& ws) {
  const TensorList grads(grad_list);
  CHECK_VALUE(grads.size() > 0, "there are no gradient tensors");
  std::optional<TensorList> out;
  if (out_list) out.emplace(*out_list);
  CHECK_VALUE(!out || out->size() == grads.size(), "out must have one tensor per gradient");
  const Tensor& first = grads[0];
  check_gpu(first);
  const at::Device device = first.device();
  std::vector<finetune_tensor> table(grads.size());
  for (size_t i = 0; i < grads.size(); ++i) {
    const Tensor& g = grads[i];
    CHECK_VALUE(g.layout() == at::kStrided && g.device() == device,
                "gradients must be dense and on one GPU (there is no CPU path)");
    const bool packed = g.is_contiguous();
    CHECK_VALUE(packed || g.is_non_overlapping_and_dense(), "gradients must fill one block of memory each");
    table[i] = {g.data_ptr(), nullptr, g.numel(), dtype_code(g)};
    table[i].out = const_cast<void*>(table[i].grad);
    if (out) {
      const Tensor& o = (*out)[i];
      CHECK_VALUE(o.layout() == at::kStrided && o.device() == device && o.scalar_type() == g.scalar_type() &&
                      o.sizes() == g.sizes() && ((packed && o.is_contiguous()) || o.strides() == g.strides()),
                  "out must match the gradients in dtype, device, shape and strides");
      table[i].out = o.data_ptr();
    }
  }
  const int64_t n = static_cast<int64_t>(grads.size());
  CHECK_VALUE(!norm || (norm->scalar_type() == at::kFloat && norm->numel() == 1 && norm->device() == device),
              "norm must hold one float32 on the gradients' device");
  const c10::DeviceGuard guard(device);
  Tensor result = norm ? *norm : new_f32({}, first);
  int64_t need = 0;
  check("grad_norm_workspace", grad_norm_workspace(table.data(), n, &need));
  const Workspace work(first, need, ws);
  if (max_norm) {
    check("clip_grad_norm", clip_grad_norm(table.data(), n, *max_norm, eps, ptr(result), work.p(), work.bytes(),
                                           stream_of(first)));
    const TensorList& changed = out ? *out : grads;
    for (size_t i = 0; i < changed.size(); ++i) written(changed[i]);
  } else {
    check("grad_norm", grad_norm(table.data(), n, ptr(result), work.p(), work.bytes(), stream_of(first)));
  }
  written(norm);
  return result;
}

}  // namespace

PYBIND11_MODULE(_finetune_host, m) {
  m.doc() = "calls of libfinetune.so on torch tensors";
  py::register_exception_translator([](std::exception_ptr p) {
    try {
      if (p) std::rethrow_exception(p);
    } catch (const StatusError& e) {
      const py::object type = py::module_::import("block_circulant_layers_amd.finetune").attr("FinetuneError");
      const py::object error = type(e.func, e.status);
      PyErr_SetObject(type.ptr(), error.ptr());
    }
  });
  m.def("status_string", &finetune_status_string);
  m.def("abi_version", &finetune_abi_version);
  m.def("layer_norm_fwd", &layer_norm_fwd_);
  m.def("layer_norm_bwd", &layer_norm_bwd_);
  m.def("token_logprob", &token_logprob_);
  m.def("token_logprob_bwd", &token_logprob_bwd_);
  m.def("preference_loss", &preference_loss_);
  m.def("preference_loss_bwd", &preference_loss_bwd_);
  m.def("policy_loss", &policy_loss_);
  m.def("policy_loss_bwd", &policy_loss_bwd_);
  m.def("clip_grad_norm", &clip_grad_norm_);
  finetune_host::define_attention(m);
}
