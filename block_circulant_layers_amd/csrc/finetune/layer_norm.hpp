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

// A row is held by T threads, E elements each, in 16-byte pieces: piece i of
// thread t holds columns (i T + t) V .. + V.  T = 8, 16, ... 1024 with 16
// elements a thread cover rows of up to 128, 256, ... 16384 elements; a workgroup
// of 256 threads (T, if that is more) holds 256 / T rows at once and walks over
// the rows, so that weight, bias and the sums over rows stay on the chip.  (With
// T = 8, 64, 256 and 1024 alone most threads of some rows hold nothing: the
// backward of 21390 rows of 1030 fp32 took 255 us, 83 us with the others.)
constexpr int kNormElems = 16;
constexpr int norm_wg(int t) { return t > kNormThreads ? t : kNormThreads; }

// RAGGED: the row's length is no multiple of a piece, so a piece may be cut.  A
// cut piece is loaded as the row's last whole one, and settle() moves its
// elements into place once they are wanted: with loads by element in a branch
// of the lane that holds the cut piece, its wave waited for all of its loads at
// once, the next row's among them (48547 rows of 1212 fp16: forward 87 us,
// backward 192 us; of 1208 47 and 77; with whole loads 1212 take 52 and 85 us).
// Its stores go by halves, quarters, ... of a piece.
template <class Io, int T, bool RAGGED, bool STREAM>
struct NormRow {
  static constexpr int V = Io::kVec;
  static constexpr int E = kNormElems;
  static constexpr int N = E / V;  // pieces a thread
  typename Io::Vec raw[N];

  static __device__ __forceinline__ int col(int i) { return (i * T + static_cast<int>(threadIdx.x) % T) * V; }
  // whether element e of piece i lies in the row
  static __device__ __forceinline__ bool has(int i, int e, int d) {
    return RAGGED ? col(i) + e < d : col(i) < d;
  }
  __device__ __forceinline__ void load(const typename Io::T* p, int d) {
    if (RAGGED && T == 8 && d < V) {  // no whole piece in the row
      raw[0] = {};
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (col(0) + e < d) raw[0][e] = p[col(0) + e];
#pragma unroll
      for (int i = 1; i < N; ++i) raw[i] = {};
      return;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = col(i);
      raw[i] = {};
      if (c < d) raw[i] = load_vec<Io, STREAM>(p + (RAGGED && c + V > d ? d - V : c));
    }
  }
  // the 32-bit words of a piece, its first `n` elements gone and zeros behind the others
  static constexpr int W = V / 4;  // elements a word
  typedef uint32_t Words __attribute__((ext_vector_type(4)));
  typedef uint32_t Two __attribute__((ext_vector_type(2), aligned(2), may_alias));
  typedef uint32_t One __attribute__((aligned(2), may_alias));
  static __device__ __forceinline__ Words shifted(Words q, int n) {
    if (n & (2 * W)) q = Words{q[2], q[3], 0, 0};
    if (n & W) q = Words{q[1], q[2], q[3], 0};
    if (W > 1 && (n & 1)) {
#pragma unroll
      for (int k = 0; k < 4; ++k) q[k] = q[k] >> 16 | (k < 3 ? q[(k + 1) % 4] << 16 : 0);
    }
    return q;
  }
  __device__ __forceinline__ void settle(int d) {
    if (!RAGGED || (T == 8 && d < V)) return;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = col(i);
      if (c < d && c + V > d)
        raw[i] = __builtin_bit_cast(typename Io::Vec, shifted(__builtin_bit_cast(Words, raw[i]), c + V - d));
    }
  }
  __device__ __forceinline__ float at(int k) const { return Io::widen(raw[k / V][k % V]); }
  static __device__ __forceinline__ void store(typename Io::T* p, int d, const float* v) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = col(i);
      typename Io::Vec o;
#pragma unroll
      for (int e = 0; e < V; ++e) o[e] = Io::narrow(v[i * V + e]);
      if (c + V <= d) {
        store_vec<Io, STREAM>(p + c, o);
      } else if (RAGGED && c < d) {
        Words q = __builtin_bit_cast(Words, o);
        typename Io::T* at = p + c;
        if ((d - c) & (2 * W)) {
          *reinterpret_cast<Two*>(at) = Two{q[0], q[1]};
          q = shifted(q, 2 * W);
          at += 2 * W;
        }
        if ((d - c) & W) {
          *reinterpret_cast<One*>(at) = q[0];
          q = shifted(q, W);
          at += W;
        }
        if (W > 1 && ((d - c) & 1)) *at = static_cast<typename Io::T>(q[0]);
      }
    }
  }
  // fp32 parameters of the thread's columns, `fill` where there are none
  static __device__ __forceinline__ void params(const float* p, int d, float fill, float* v) {
    typedef float Vec __attribute__((ext_vector_type(V), aligned(4)));
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = col(i);
      Vec q = fill;
      if (p && c + V <= d) {
        q = *reinterpret_cast<const Vec*>(p + c);
      } else if (RAGGED && p) {
#pragma unroll
        for (int e = 0; e < V; ++e)
          if (c + e < d) q[e] = p[c + e];
      }
#pragma unroll
      for (int e = 0; e < V; ++e) v[i * V + e] = q[e];
    }
  }
};

// y, mean and rstd.  The variance is the mean square of x - mean, taken from
// the registers, not E x^2 - mean^2, which cancels for rows whose mean is
// large against their spread.  The next row's loads are in flight while a row
// is summed.
template <class Io, int T, bool RAGGED, bool STREAM>
__global__ void __launch_bounds__(norm_wg(T))
    layer_norm_fwd_kernel(const typename Io::T* x, const float* w, const float* b, typename Io::T* y, float* mean,
                          float* rstd, int64_t rows, int d, int64_t xs, int64_t ys, float eps) {
  using Row = NormRow<Io, T, RAGGED, STREAM>;
  constexpr int WG = norm_wg(T), G = WG / T, E = Row::E;
  __shared__ float s[2][WG / kWave];
  const int64_t step = static_cast<int64_t>(gridDim.x) * G;
  float wr[E], br[E];
  Row::params(w, d, 1.0f, wr);
  Row::params(b, d, 0.0f, br);
  const float n = static_cast<float>(d);
  const int64_t first = static_cast<int64_t>(blockIdx.x) * G;
  Row next;
  int64_t r = first + threadIdx.x / T;
  if (r < rows) next.load(x + r * xs, d);
  // every thread of the workgroup makes the same number of rounds (barriers inside)
  for (int64_t r0 = first; r0 < rows; r0 += step, r += step) {
    Row cur = next;
    cur.settle(d);
    if (r + step < rows) next.load(x + (r + step) * xs, d);
    float v[E], a = 0.0f;
#pragma unroll
    for (int k = 0; k < E; ++k) a += v[k] = cur.at(k);
    const float mu = group_sum<T>(a, s[0]) / n;
    a = 0.0f;
#pragma unroll
    for (int k = 0; k < E; ++k) {
      v[k] = Row::has(k / Row::V, k % Row::V, d) ? v[k] - mu : 0.0f;
      a += v[k] * v[k];
    }
    const float rs = 1.0f / sqrtf(group_sum<T>(a, s[1]) / n + eps);
    if (r < rows) {
      if (threadIdx.x % T == 0) {
        if (mean) mean[r] = mu;
        if (rstd) rstd[r] = rs;
      }
#pragma unroll
      for (int k = 0; k < E; ++k) v[k] = v[k] * rs * wr[k] + br[k];
      Row::store(y + r * ys, d, v);
    }
  }
}

// dx, and the sums of dy hat and dy over the rows this workgroup walks over,
// stored as slice blockIdx.x of the workspace (null: not needed): x and dy are
// read once for all three gradients, the next row loaded ahead.  1024 threads have
// 128 registers each, which hold the rows and weights but not the sums too
// (they spilled): those rows keep their sums in LDS, 128 KB a workgroup, every
// thread its own slots, and in fp32 load no row ahead.
constexpr size_t norm_bwd_lds(int t) { return t == 1024 ? 2 * kNormElems * t * sizeof(float) : 0; }

template <class Io, int T, bool RAGGED, bool STREAM>
__global__ void __launch_bounds__(norm_wg(T))
    layer_norm_bwd_kernel(const typename Io::T* x, const float* w, const float* mean, const float* rstd,
                          const typename Io::T* dy, typename Io::T* dx, float* ws, int64_t rows, int d, int64_t xs,
                          int64_t dys, int64_t dxs) {
  using Row = NormRow<Io, T, RAGGED, STREAM>;
  constexpr int WG = norm_wg(T), G = WG / T, E = Row::E;
  __shared__ float s[2][2][WG / kWave];
  const int64_t step = static_cast<int64_t>(gridDim.x) * G;
  constexpr bool IN_LDS = T == 1024, AHEAD = !IN_LDS || sizeof(typename Io::T) == 2;
  FINETUNE_DYNAMIC_LDS(sums);  // IN_LDS: [2][E][T]
  float* const mine = sums + threadIdx.x;
  float wr[E], dw[IN_LDS ? 1 : E] = {}, db[IN_LDS ? 1 : E] = {};
  if constexpr (IN_LDS)
    for (int k = 0; k < 2 * E; ++k) mine[k * T] = 0.0f;
  Row::params(w, d, 1.0f, wr);
  const float n = static_cast<float>(d);
  const int64_t first = static_cast<int64_t>(blockIdx.x) * G;
  Row nx, ng;
  float nm = 0.0f, nr = 0.0f;
  int64_t r = first + threadIdx.x / T;
  auto fetch = [&](int64_t row) {
    nx.load(x + row * xs, d);
    ng.load(dy + row * dys, d);
    nm = mean[row];
    nr = rstd[row];
  };
  if (AHEAD && r < rows) fetch(r);
  int turn = 0;
  for (int64_t r0 = first; r0 < rows; r0 += step, r += step, turn ^= 1) {
    if (!AHEAD) fetch(r);  // one row a workgroup: r = r0
    Row cx = nx, cg = ng;
    cx.settle(d);
    cg.settle(d);
    const float mu = nm, rs = nr;
    if (AHEAD && r + step < rows) fetch(r + step);
    const bool live = r < rows;
    // With q = dy rstd and t = x - mean, hat enters as q t: A = sum q w and C =
    // rstd sum q w t give dx = q w - A / d - t rstd C / d.  (dy hat instead is as
    // many instructions, but where a row ends, at x = dy = 0, hat = -mean rstd may
    // be infinite, and 0 times it NaN.)
    float a = 0.0f, c = 0.0f;
#pragma unroll
    for (int k = 0; k < E; ++k) {
      const float g = cg.at(k), q = g * rs, t = cx.at(k) - mu;
      // columns past the row hold g = 0; a round without a row adds nothing
      a += q * wr[k];
      c += q * wr[k] * t;
      if constexpr (IN_LDS) {
        mine[k * T] += q * t;
        mine[(E + k) * T] += g;
      } else if (live) {
        dw[k] += q * t;
        db[k] += g;
      }
    }
    if (dx) {
      a = group_sum<T>(a, s[turn][0]) / n;
      c = rs * (group_sum<T>(c, s[turn][1]) / n);
      if (live) {
        float v[E];
#pragma unroll
        for (int k = 0; k < E; ++k) v[k] = cg.at(k) * rs * wr[k] - a - (cx.at(k) - mu) * rs * c;
        Row::store(dx + r * dxs, d, v);
      }
    }
  }
  if (!ws) return;
  float* slice = ws + static_cast<int64_t>(blockIdx.x) * 2 * d;
  if constexpr (G > 1) {
    // the groups' sums meet in LDS, in the order of the groups
    __shared__ float join[G][T * E];
    float* part[2] = {dw, db};
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      __syncthreads();
#pragma unroll
      for (int k = 0; k < E; ++k) join[threadIdx.x / T][Row::col(k / Row::V) + k % Row::V] = part[q][k];
      __syncthreads();
      for (int c = threadIdx.x; c < d; c += WG) {
        float t = join[0][c];
        for (int g = 1; g < G; ++g) t += join[g][c];
        slice[q * d + c] = t;
      }
    }
  } else {
    // 16 bytes at a time where the columns are there
    typedef float Quad __attribute__((ext_vector_type(4), aligned(4)));
#pragma unroll
    for (int k = 0; k < E; k += 4) {
      Quad q[2];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        q[0][e] = IN_LDS ? mine[(k + e) * T] : dw[IN_LDS ? 0 : k + e];
        q[1][e] = IN_LDS ? mine[(E + k + e) * T] : db[IN_LDS ? 0 : k + e];
      }
      const int c = Row::col(k / Row::V) + k % Row::V;
      if (c + 4 <= d) {
        *reinterpret_cast<Quad*>(slice + c) = q[0];
        *reinterpret_cast<Quad*>(slice + d + c) = q[1];
      } else if (RAGGED) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (c + e < d) {
            slice[c + e] = q[0][e];
            slice[d + c + e] = q[1][e];
          }
      }
    }
  }
}

// ---- rows of any length: one workgroup per row, the row read again for every
// ---- sum (2048 rows of 32768 bf16: forward 146 us, backward 183 us, 1.8 and 2.2
// ---- TB/s; element by element, bound by the loads each sum waits for)

// Three reads of x.  The variance is the mean square of x - mean, not
// E x^2 - mean^2, which cancels for rows whose mean is large against their
// spread.
template <class Io>
__global__ void __launch_bounds__(kNormThreads)
    layer_norm_wide_fwd_kernel(const typename Io::T* x, const float* w, const float* b, typename Io::T* y, float* mean,
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

// dx, one workgroup per row; two reads of x and dy.
template <class Io>
__global__ void __launch_bounds__(kNormThreads)
    layer_norm_wide_dx_kernel(const typename Io::T* x, const float* w, const float* mean, const float* rstd,
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
    layer_norm_wide_dw_kernel(const typename Io::T* x, const float* mean, const float* rstd, const typename Io::T* dy,
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

// ---- the sums over rows from the slices of the workspace, in order

// 32 columns (one 128-byte line of a slice) by 32 groups of slices a workgroup:
// 2 x 4096 columns fill the chip's 256 compute units, and a thread's few loads
// are all in flight at once.
constexpr int kSumCols = 32;
constexpr int kSumGroups = 32;  // groups of slices summed side by side, then in order

__global__ void __launch_bounds__(kSumCols* kSumGroups)
    layer_norm_dw_sum_kernel(const float* ws, float* dw, float* db, int d, int parts) {
  __shared__ float s[kSumGroups][kSumCols];
  const int t = threadIdx.x % kSumCols, g = threadIdx.x / kSumCols;
  const int c = blockIdx.x * kSumCols + t;  // dw's columns, then db's
  float a = 0.0f;
  if (c < 2 * d) {
#pragma unroll 8
    for (int p = g; p < parts; p += kSumGroups) a += ws[static_cast<int64_t>(p) * 2 * d + c];
  }
  s[g][t] = a;
  __syncthreads();
  if (g != 0 || c >= 2 * d) return;
  for (int i = 1; i < kSumGroups; ++i) a += s[i][t];
  float* o = c < d ? dw : db;
  if (o) o[c < d ? c : c - d] = a;
}

}  // namespace finetune
