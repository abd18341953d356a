// host.hpp -- what the parts of the Python module _finetune_host share: checks of
// tensors, results and workspaces from torch's allocator, the current stream.
#pragma once

#include <torch/extension.h>

#include <ATen/hip/impl/HIPStreamMasqueradingAsCUDA.h>
#include <c10/core/DeviceGuard.h>

#include <initializer_list>
#include <optional>
#include <tuple>
#include <vector>

#include "finetune.h"

namespace finetune_host {

using at::Tensor;
using Opt = std::optional<Tensor>;

#define CHECK_VALUE(cond, ...) TORCH_CHECK_VALUE(cond, __VA_ARGS__)

// A nonzero status of the library: raised as the package's FinetuneError
struct StatusError : std::exception {
  const char* func;
  int status;
  StatusError(const char* f, int s) : func(f), status(s) {}
};

inline void check(const char* func, int status) {
  if (status != RDFFT_OK) throw StatusError(func, status);
}

inline int dtype_code(const Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat: return RDFFT_F32;
    case at::kBFloat16: return RDFFT_BF16;
    case at::kHalf: return RDFFT_F16;
    default:
      TORCH_CHECK_TYPE(false, "unsupported dtype ", t.scalar_type(), ": use float32, bfloat16 or float16");
  }
}

inline void check_gpu(const Tensor& t) { CHECK_VALUE(t.is_cuda(), "tensors must be on a GPU (there is no CPU path)"); }

inline void* stream_of(const Tensor& t) {
  return c10::hip::getCurrentHIPStreamMasqueradingAsCUDA(t.device().index()).stream();
}

// a contiguous float32 array of `shape` on like's device
inline float* f32(const char* name, const Tensor& t, at::IntArrayRef shape, const Tensor& like) {
  CHECK_VALUE(t.scalar_type() == at::kFloat && t.sizes() == shape, name, " must be float32 of shape ", shape);
  CHECK_VALUE(t.device() == like.device(), "tensors must be on one device");
  CHECK_VALUE(t.is_contiguous(), "tensors must be contiguous");
  return static_cast<float*>(t.data_ptr());
}
inline float* f32(const char* name, const Opt& t, at::IntArrayRef shape, const Tensor& like) {
  return t ? f32(name, *t, shape, like) : nullptr;
}

// Counts a write to a tensor of the caller's, which torch cannot see: autograd
// refuses a backward that needs the values from before.
inline void written(const Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}
inline void written(const Opt& t) {
  if (t) written(*t);
}

inline Tensor new_f32(at::IntArrayRef shape, const Tensor& like) { return at::empty(shape, like.options().dtype(at::kFloat)); }

// The float32 arrays that a call returns.  Each has its own memory, so that one
// that is kept holds no other; but those that fit it together share one block of
// 512 bytes, the smallest that torch's allocator hands out (an allocation costs
// the host 0.8 us, one of 13 us in a loss step of a few kilobytes).
struct Results {
  static constexpr int64_t kShared = 128;  // floats
  const Tensor& like;
  Tensor block;
  int64_t used = 0;
  // `sizes`: of the arrays, in the order in which next() makes them
  Results(const Tensor& l, std::initializer_list<int64_t> sizes) : like(l) {
    int64_t n = 0;
    for (int64_t s : sizes)
      if (n + s <= kShared) n += s;
    if (n > 0) block = new_f32({n}, like);
  }
  Tensor next(at::IntArrayRef shape) {
    const int64_t n = c10::multiply_integers(shape);
    if (!block.defined() || used + n > kShared) return new_f32(shape, like);
    auto impl = c10::make_intrusive<at::TensorImpl>(c10::Storage(block.storage()), block.key_set(), block.dtype());
    impl->set_storage_offset(block.storage_offset() + used);
    impl->set_sizes_contiguous(shape);
    used += n;
    return Tensor(std::move(impl));
  }
};

// the caller's workspace, or new memory of the current stream's: no tensor is
// made of it
struct Workspace {
  Opt given;
  c10::DataPtr made;
  int64_t size;
  Workspace(const Tensor& like, int64_t bytes, const Opt& ws) : given(ws), size(bytes) {
    if (given) {
      CHECK_VALUE(given->device() == like.device() && given->is_contiguous(),
                  "ws must be contiguous and on the tensors' device");
      size = given->numel() * given->element_size();
    } else {
      made = c10::GetAllocator(like.device().type())->allocate(static_cast<size_t>(bytes));
    }
  }
  void* p() const { return given ? given->data_ptr() : made.get(); }
  int64_t bytes() const { return size; }
};

// ---- rows ----------------------------------------------------------------

struct RowsOf {
  int64_t rows, d, stride;
};

// rows (last axis contiguous) that are evenly spaced
inline RowsOf rows_of(const char* name, const Tensor& t) {
  check_gpu(t);
  CHECK_VALUE(t.dim() > 0, name, " must have at least one axis");
  const int64_t d = t.size(-1), rows = d ? t.numel() / d : 0;
  if (t.is_contiguous()) return {rows, d, d};
  CHECK_VALUE(t.stride(-1) == 1 || d <= 1 || rows == 0, "the last axis of ", name, " must be contiguous");
  if (rows <= 1) return {rows, d, d};
  int64_t want = -1, step = 1;  // the stride that folds all leading axes into one
  for (int64_t a = t.dim() - 2; a >= 0; --a) {
    if (t.size(a) == 1) continue;
    if (want < 0) want = t.stride(a);
    CHECK_VALUE(t.stride(a) == want * step, "the rows of ", name, " must be evenly spaced");
    step *= t.size(a);
  }
  return {rows, d, want};
}

inline int64_t same_rows(const char* name, const Tensor& t, const Tensor& like) {
  CHECK_VALUE(t.scalar_type() == like.scalar_type() && t.sizes() == like.sizes() && t.device() == like.device(), name,
              " must have the dtype, shape and device of x");
  return rows_of(name, t).stride;
}

inline float* ptr(const Tensor& t) { return static_cast<float*>(t.data_ptr()); }

}  // namespace finetune_host
