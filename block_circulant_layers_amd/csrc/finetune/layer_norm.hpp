// layer_norm.hpp -- layer normalisation, forward and backward.
//
// Per row: mean = sum x / d, rstd = 1 / sqrt(sum (x - mean)^2 / d + eps),
// hat = (x - mean) rstd, y = hat w + b.  With g = dy w,
//   dx = rstd (g - mean(g) - hat mean(g hat)),  dw = sum_rows dy hat,
//   db = sum_rows dy.
#pragma once

#include "device.hpp"

namespace finetune {

constexpr int kNormThreads = 256;

// One workgroup per row.  The variance is the mean square of x - mean (a
// second read of the row), not E x^2 - mean^2, which cancels for rows whose
// mean is large against their spread.
template <class Io>
__global__ void __launch_bounds__(kNormThreads)
    layer_norm_fwd_kernel(const typename Io::T* x, const float* w, const float* b, typename Io::T* y, float* mean,
                          float* rstd, int64_t rows, int d, int64_t xs, int64_t ys, float eps) {
  __shared__ float s[2][kNormThreads / kWave];
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const typename Io::T* xr = x + r * xs;
    float a = 0.0f;
    for (int j = threadIdx.x; j < d; j += kNormThreads) a += Io::widen(xr[j]);
    const float mu = block_sum<kNormThreads>(a, s[0]) / static_cast<float>(d);
    a = 0.0f;
    for (int j = threadIdx.x; j < d; j += kNormThreads) {
      const float v = Io::widen(xr[j]) - mu;
      a += v * v;
    }
    const float var = block_sum<kNormThreads>(a, s[1]) / static_cast<float>(d);
    const float rs = 1.0f / sqrtf(var + eps);
    if (threadIdx.x == 0) {
      if (mean) mean[r] = mu;
      if (rstd) rstd[r] = rs;
    }
    for (int j = threadIdx.x; j < d; j += kNormThreads) {
      float v = (Io::widen(xr[j]) - mu) * rs;
      if (w) v *= w[j];
      if (b) v += b[j];
      y[r * ys + j] = Io::narrow(v);
    }
    __syncthreads();
  }
}

// dx, one workgroup per row.
template <class Io>
__global__ void __launch_bounds__(kNormThreads)
    layer_norm_dx_kernel(const typename Io::T* x, const float* w, const float* mean, const float* rstd,
                         const typename Io::T* dy, typename Io::T* dx, int64_t rows, int d, int64_t xs, int64_t dys,
                         int64_t dxs) {
  __shared__ float s[2][kNormThreads / kWave];
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const float mu = mean[r], rs = rstd[r];
    float a = 0.0f, c = 0.0f;
    for (int j = threadIdx.x; j < d; j += kNormThreads) {
      const float g = Io::widen(dy[r * dys + j]) * (w ? w[j] : 1.0f);
      a += g;
      c += g * ((Io::widen(x[r * xs + j]) - mu) * rs);
    }
    a = block_sum<kNormThreads>(a, s[0]) / static_cast<float>(d);
    c = block_sum<kNormThreads>(c, s[1]) / static_cast<float>(d);
    for (int j = threadIdx.x; j < d; j += kNormThreads) {
      const float g = Io::widen(dy[r * dys + j]) * (w ? w[j] : 1.0f);
      const float hat = (Io::widen(x[r * xs + j]) - mu) * rs;
      dx[r * dxs + j] = Io::narrow(rs * (g - a - hat * c));
    }
    __syncthreads();
  }
}

// dw and db of row range blockIdx.y: column j's sums over rows
// [y * per, (y + 1) * per) go to slice y of the workspace.
template <class Io>
__global__ void __launch_bounds__(kNormThreads)
    layer_norm_dw_kernel(const typename Io::T* x, const float* mean, const float* rstd, const typename Io::T* dy,
                         float* ws, int64_t rows, int d, int64_t xs, int64_t dys, int64_t per) {
  const int j = blockIdx.x * kNormThreads + threadIdx.x;
  if (j >= d) return;
  const int64_t r0 = blockIdx.y * per, r1 = r0 + per < rows ? r0 + per : rows;
  float a = 0.0f, c = 0.0f;
  for (int64_t r = r0; r < r1; ++r) {
    const float v = Io::widen(dy[r * dys + j]);
    a += v;
    c += v * ((Io::widen(x[r * xs + j]) - mean[r]) * rstd[r]);
  }
  float* slice = ws + static_cast<int64_t>(blockIdx.y) * 2 * d;
  slice[j] = c;
  slice[d + j] = a;
}

// The slices summed in order.
__global__ void __launch_bounds__(kNormThreads)
    layer_norm_dw_sum_kernel(const float* ws, float* dw, float* db, int d, int parts) {
  const int j = blockIdx.x * kNormThreads + threadIdx.x;
  if (j >= d) return;
  float a = 0.0f, c = 0.0f;
  for (int p = 0; p < parts; ++p) {
    c += ws[static_cast<int64_t>(p) * 2 * d + j];
    a += ws[static_cast<int64_t>(p) * 2 * d + d + j];
  }
  if (dw) dw[j] = c;
  if (db) db[j] = a;
}

}  // namespace finetune
