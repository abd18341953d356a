// attention_host.cpp -- the calls of attention.h on torch tensors, for the Python module _finetune_host.
#include <array>
#include <cmath>

#include "attention.h"
#include "host.hpp"

namespace finetune_host {
namespace {

namespace py = pybind11;

attention_buckets buckets_of(int64_t count, int64_t max_distance, bool two_sided) {
  return {count, max_distance, two_sided};
}

// a table of biases, float32 [buckets, heads]
const float* table_of(const Tensor& t, int64_t heads, const Tensor& like) {
  CHECK_VALUE(t.scalar_type() == at::kFloat && t.dim() == 2 && t.size(1) == heads && t.is_contiguous(),
              "bias must be contiguous float32 of shape (buckets, ", heads, ")");
  CHECK_VALUE(t.device() == like.device(), "tensors must be on one device");
  return static_cast<const float*>(t.data_ptr());
}

// (batch, tokens, heads, head size) with a contiguous last axis
attention_tensor rows4(const char* name, const Tensor& t, at::IntArrayRef shape, const Tensor& like) {
  CHECK_VALUE(t.scalar_type() == like.scalar_type() && t.device() == like.device(), name,
              " must have the dtype and device of q");
  CHECK_VALUE(t.sizes() == shape, name, " must have shape ", shape);
  CHECK_VALUE(t.stride(3) == 1 || t.size(3) <= 1 || t.numel() == 0, "the last axis of ", name, " must be contiguous");
  return {t.data_ptr(), t.stride(0), t.stride(1), t.stride(2)};
}

const int32_t* span_of(const char* name, const Opt& t, int64_t batch, const Tensor& like) {
  if (!t) return nullptr;
  CHECK_VALUE(t->scalar_type() == at::kInt && t->dim() == 1 && t->size(0) == batch && t->is_contiguous() &&
                  t->device() == like.device(),
              name, " must be contiguous int32 of shape (", batch, ",) on the tensors' device");
  return static_cast<const int32_t*>(t->data_ptr());
}

struct Call {
  attention_problem a;
  attention_tensor q, k, v;
};

Call call_of(const Tensor& q, const Tensor& k, const Tensor& v, std::optional<double> scale, bool causal,
             const Opt& begin, const Opt& end, const Opt& bias, int64_t max_distance, bool two_sided) {
  check_gpu(q);
  CHECK_VALUE(q.dim() == 4 && k.dim() == 4, "q, k and v must have shape (batch, tokens, heads, head size)");
  const int64_t b = q.size(0), d = q.size(3);
  Call c{};
  c.a.batch = b, c.a.queries = q.size(1), c.a.keys = k.size(1);
  c.a.heads = q.size(2), c.a.kv_heads = k.size(2), c.a.head_dim = d;
  c.a.dtype = dtype_code(q);
  c.a.scale = scale ? *scale : d > 0 ? 1.0 / std::sqrt(static_cast<double>(d)) : 1.0;
  c.a.causal = causal;
  c.q = rows4("q", q, q.sizes(), q);
  c.k = rows4("k", k, {b, c.a.keys, c.a.kv_heads, d}, q);
  c.v = rows4("v", v, {b, c.a.keys, c.a.kv_heads, d}, q);
  c.a.key_begin = span_of("key_begin", begin, b, q);
  c.a.key_end = span_of("key_end", end, b, q);
  if (bias) {
    c.a.bias = table_of(*bias, c.a.heads, q);
    c.a.buckets = buckets_of(bias->size(0), max_distance, two_sided);
    if (c.a.bias == nullptr) CHECK_VALUE(false, "bias must not be empty");
  }
  return c;
}

Workspace workspace_of(const Tensor& like, const attention_problem& a, int backward, const Opt& ws) {
  int64_t need = 0;
  check("attention_workspace", attention_workspace(&a, backward, &need));
  return Workspace(like, need, ws);
}

std::tuple<Tensor, Tensor> attention_fwd_(const Tensor& q, const Tensor& k, const Tensor& v,
                                          std::optional<double> scale, bool causal, const Opt& begin, const Opt& end,
                                          const Opt& bias, int64_t max_distance, bool two_sided, const Opt& o,
                                          const Opt& ws) {
  const Call c = call_of(q, k, v, scale, causal, begin, end, bias, max_distance, two_sided);
  if (o) rows4("o", *o, q.sizes(), q);
  const c10::DeviceGuard guard(q.device());
  const Workspace work = workspace_of(q, c.a, 0, ws);
  Tensor out = o ? *o : at::empty(q.sizes(), q.options());
  Tensor lse = new_f32({c.a.batch, c.a.heads, c.a.queries}, q);
  const attention_tensor to = rows4("o", out, q.sizes(), q);
  check("attention_fwd",
        attention_fwd(&c.a, &c.q, &c.k, &c.v, &to, ptr(lse), work.p(), work.bytes(), stream_of(q)));
  written(o);
  return {out, lse};
}

std::tuple<Tensor, Tensor, Tensor, Opt> attention_bwd_(
    const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& o, const Tensor& lse, const Tensor& dout,
    std::optional<double> scale, bool causal, const Opt& begin, const Opt& end, const Opt& bias, int64_t max_distance,
    bool two_sided, bool need_dbias, const Opt& dq, const Opt& dk, const Opt& dv, const Opt& ws) {
  const Call c = call_of(q, k, v, scale, causal, begin, end, bias, max_distance, two_sided);
  const attention_tensor ot = rows4("o", o, q.sizes(), q), dt = rows4("dout", dout, q.sizes(), q);
  const float* l = f32("lse", lse, {c.a.batch, c.a.heads, c.a.queries}, q);
  if (dq) rows4("dq", *dq, q.sizes(), q);
  if (dk) rows4("dk", *dk, k.sizes(), q);
  if (dv) rows4("dv", *dv, k.sizes(), q);
  const c10::DeviceGuard guard(q.device());
  const Workspace work = workspace_of(q, c.a, 1, ws);
  Tensor gq = dq ? *dq : at::empty(q.sizes(), q.options());
  Tensor gk = dk ? *dk : at::empty(k.sizes(), q.options());
  Tensor gv = dv ? *dv : at::empty(k.sizes(), q.options());
  Opt gb;
  if (bias && need_dbias) gb = new_f32(bias->sizes(), q);
  const attention_tensor tq = rows4("dq", gq, q.sizes(), q), tk = rows4("dk", gk, k.sizes(), q),
                         tv = rows4("dv", gv, k.sizes(), q);
  check("attention_bwd", attention_bwd(&c.a, &c.q, &c.k, &c.v, &ot, l, &dt, &tq, &tk, &tv, gb ? ptr(*gb) : nullptr,
                                       work.p(), work.bytes(), stream_of(q)));
  written(dq);
  written(dk);
  written(dv);
  return {gq, gk, gv, gb};
}

Tensor relative_bias_fwd_(const Tensor& table, int64_t queries, int64_t keys, int64_t max_distance, bool two_sided,
                          at::ScalarType dtype, const Opt& out) {
  check_gpu(table);
  CHECK_VALUE(table.dim() == 2 && queries >= 0 && keys >= 0,
              "table must have shape (buckets, heads), and the lengths must not be negative");
  const int64_t heads = table.size(1);
  const float* t = table_of(table, heads, table);
  const std::array<int64_t, 3> sizes{heads, queries, keys};
  const at::IntArrayRef shape(sizes);
  CHECK_VALUE(!out || (out->sizes() == shape && out->is_contiguous() && out->scalar_type() == dtype &&
                       out->device() == table.device()),
              "out must be contiguous of the given dtype and of shape ", shape, " on the table's device");
  const c10::DeviceGuard guard(table.device());
  Tensor r = out ? *out : at::empty(shape, table.options().dtype(dtype));
  const attention_buckets b = buckets_of(table.size(0), max_distance, two_sided);
  check("relative_bias_fwd",
        relative_bias_fwd(t, r.data_ptr(), heads, queries, keys, &b, dtype_code(r), stream_of(table)));
  written(out);
  return r;
}

Tensor relative_bias_bwd_(const Tensor& dbias, int64_t count, int64_t max_distance, bool two_sided, const Opt& dtable,
                          const Opt& ws) {
  check_gpu(dbias);
  const int64_t n = dbias.dim();
  CHECK_VALUE(n == 3 || n == 4, "dbias must have shape (heads, queries, keys), with or without a batch before it");
  const int64_t batch = n == 4 ? dbias.size(0) : 1, heads = dbias.size(n - 3), tq = dbias.size(n - 2),
                tk = dbias.size(n - 1);
  CHECK_VALUE(dbias.stride(n - 1) == 1 || tk <= 1 || dbias.numel() == 0, "the last axis of dbias must be contiguous");
  const int code = dtype_code(dbias);
  const attention_buckets b = buckets_of(count, max_distance, two_sided);
  if (dtable) f32("dtable", *dtable, {count, heads}, dbias);
  int64_t need = 0;
  check("relative_bias_workspace", relative_bias_workspace(batch, heads, tq, tk, &b, &need));
  const c10::DeviceGuard guard(dbias.device());
  const Workspace work(dbias, need, ws);
  Tensor r = dtable ? *dtable : new_f32({count, heads}, dbias);
  check("relative_bias_bwd",
        relative_bias_bwd(dbias.data_ptr(), n == 4 ? dbias.stride(0) : 0, dbias.stride(n - 3), dbias.stride(n - 2),
                          ptr(r), batch, heads, tq, tk, &b, work.p(), work.bytes(), code, stream_of(dbias)));
  written(dtable);
  return r;
}

// forward, or (backward) without a residual
Tensor dropout_(const Tensor& x, double p, uint64_t seed, uint64_t offset, const Opt& device_seed,
                const Opt& residual, const Opt& y, bool backward) {
  const RowsOf r = rows_of(backward ? "dy" : "x", x);
  const int code = dtype_code(x);
  const int64_t rs = residual ? same_rows("residual", *residual, x) : 0;
  const int64_t ys = y ? same_rows(backward ? "dx" : "y", *y, x) : r.d;
  CHECK_VALUE(!device_seed || (device_seed->scalar_type() == at::kLong && device_seed->numel() == 1 &&
                               device_seed->device() == x.device()),
              "a seed tensor must hold one int64 on the tensors' device");
  const c10::DeviceGuard guard(x.device());
  Tensor out = y ? *y : at::empty(x.sizes(), x.options());
  const attention_dropout how{p, seed, offset,
                              device_seed ? static_cast<const uint64_t*>(device_seed->data_ptr()) : nullptr};
  if (backward)
    check("dropout_bwd", dropout_bwd(x.data_ptr(), out.data_ptr(), r.rows, r.d, r.stride, ys, &how, code,
                                     stream_of(x)));
  else
    check("dropout_fwd", dropout_fwd(x.data_ptr(), residual ? residual->data_ptr() : nullptr, out.data_ptr(), r.rows,
                                     r.d, r.stride, rs, ys, &how, code, stream_of(x)));
  written(y);
  return out;
}

}  // namespace

void define_attention(py::module_& m) {
  m.def("attention_abi_version", &attention_abi_version);
  m.def("attention_fwd", &attention_fwd_);
  m.def("attention_bwd", &attention_bwd_);
  m.def("relative_bias_fwd", &relative_bias_fwd_);
  m.def("relative_bias_bwd", &relative_bias_bwd_);
  m.def("dropout", &dropout_);
}

}  // namespace finetune_host
