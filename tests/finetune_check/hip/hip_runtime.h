// hip/hip_runtime.h stand-in for running the fine-tuning kernels on CPU threads.
//
// Test infrastructure only: finetune_lib.hip is built for the host against this
// header, so the C ABI, its launch arithmetic and the kernel templates run
// unchanged, with
//   * one host thread per GPU thread of a workgroup, workgroups one after
//     another; __syncthreads() a barrier of the workgroup's threads;
//   * the lane moves (DPP, permlane swaps, shuffles) as exchanges through a slot
//     per thread between two barriers of the wave's 64 threads;
//   * __shared__ arrays static, the launch's dynamic LDS a fresh NaN-filled
//     block a workgroup.
#pragma once

#include <pthread.h>

#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <functional>
#include <vector>

#define __global__
#define __device__
#define __host__
#define __forceinline__ inline
#define __launch_bounds__(...)
#define __shared__ static
#define __restrict__ __restrict

using std::exp;
using std::expm1;
using std::fabs;
using std::log;
using std::log1p;
using std::sqrt;

struct dim3 {
  unsigned x = 1, y = 1, z = 1;
  constexpr dim3() = default;
  constexpr dim3(unsigned a, unsigned b = 1, unsigned c = 1) : x(a), y(b), z(c) {}
};
struct float2 {
  float x, y;
};
struct double2 {
  double x, y;
};
inline float2 make_float2(float x, float y) { return {x, y}; }
inline double2 make_double2(double x, double y) { return {x, y}; }

typedef int hipError_t;
typedef void* hipStream_t;
constexpr hipError_t hipSuccess = 0;
inline hipError_t hipGetLastError() { return hipSuccess; }

namespace emu {

struct Ctx {
  dim3 tid, bid, bdim, gdim;
  pthread_barrier_t *group = nullptr, *wave = nullptr;
};
inline thread_local Ctx ctx;
inline float* dyn_lds = nullptr;
inline uint32_t slots[1024];
inline long launches = 0;

inline void fail(const char* what) {
  std::fprintf(stderr, "EMU ERROR: %s\n", what);
  std::abort();
}

struct WorkItem {
  std::function<void()>* body;
  std::vector<float>* dyn;
  Ctx c;
};
// one GPU thread's host thread: it runs every workgroup of the launch in turn
inline void* run_item(void* p) {
  auto* w = static_cast<WorkItem*>(p);
  ctx = w->c;
  for (unsigned by = 0; by < ctx.gdim.y; ++by)
    for (unsigned bx = 0; bx < ctx.gdim.x; ++bx) {
      pthread_barrier_wait(ctx.group);  // the workgroup before is done with the shared arrays
      if (ctx.tid.x == 0)
        for (auto& v : *w->dyn) v = std::nanf("");
      if (w->dyn->size() > 1) pthread_barrier_wait(ctx.group);
      ctx.bid = dim3(bx, by);
      (*w->body)();
    }
  return nullptr;
}

inline void launch(dim3 grid, dim3 block, size_t dyn_bytes, std::function<void()> body) {
  const unsigned nt = block.x;
  if (nt == 0 || nt > 1024 || nt % 64 != 0 || block.y != 1 || block.z != 1) fail("workgroup size");
  if (grid.x == 0 || grid.y == 0 || grid.y > 65535 || grid.z != 1) fail("grid size");
  if (dyn_bytes > 160 * 1024) fail("LDS size");
  std::vector<float> dyn(dyn_bytes / sizeof(float) + 1);  // one slot that no kernel uses, for an address
  dyn_lds = dyn.data();
  std::vector<pthread_t> th(nt);
  std::vector<WorkItem> items(nt);
  std::vector<pthread_barrier_t> bars(1 + nt / 64);
  pthread_barrier_init(&bars[0], nullptr, nt);
  for (unsigned w = 0; w < nt / 64; ++w) pthread_barrier_init(&bars[1 + w], nullptr, 64);
  pthread_attr_t attr;
  pthread_attr_init(&attr);
  pthread_attr_setstacksize(&attr, 1 << 20);
  ++launches;
  for (unsigned t = 0; t < nt; ++t) {
    items[t] = {&body, &dyn, Ctx{dim3(t), dim3(0, 0), block, grid, &bars[0], &bars[1 + t / 64]}};
    if (pthread_create(&th[t], &attr, run_item, &items[t]) != 0) fail("pthread_create");
  }
  for (unsigned t = 0; t < nt; ++t) pthread_join(th[t], nullptr);
  for (auto& b : bars) pthread_barrier_destroy(&b);
  pthread_attr_destroy(&attr);
}

// v of the wave's lane `from(lane)`; every lane of the wave takes part
template <class F>
inline uint32_t lane_read(uint32_t v, F from) {
  const unsigned t = ctx.tid.x, base = t / 64 * 64;
  slots[t] = v;
  pthread_barrier_wait(ctx.wave);
  const uint32_t r = slots[base + from(t - base)];
  pthread_barrier_wait(ctx.wave);
  return r;
}

inline uint32_t dpp(uint32_t v, int ctrl) {
  return lane_read(v, [ctrl](unsigned l) -> unsigned {
    if (ctrl < 0x100) return (l & ~3u) | ((ctrl >> (2 * (l & 3))) & 3);  // a permutation within four lanes
    if (ctrl == 0x141) return (l & ~7u) | (7 - (l & 7));                 // eight lanes mirrored
    if (ctrl == 0x140) return (l & ~15u) | (15 - (l & 15));              // sixteen lanes mirrored
    fail("lane move not modelled");
    return l;
  });
}

struct Pair {
  uint32_t v[2];
  uint32_t operator[](int i) const { return v[i]; }
};
// the odd runs of W lanes of the first operand change places with the even runs of the second
inline Pair swap_runs(uint32_t a, uint32_t b, unsigned W) {
  const unsigned l = ctx.tid.x % 64;
  const bool odd = l / W % 2 == 1;
  const uint32_t from_b = lane_read(b, [W](unsigned q) { return q - q / W % 2 * W; });
  const uint32_t from_a = lane_read(a, [W](unsigned q) { return q + (1 - q / W % 2) * W; });
  return {{odd ? from_b : a, odd ? b : from_a}};
}

}  // namespace emu

#define threadIdx (emu::ctx.tid)
#define blockIdx (emu::ctx.bid)
#define blockDim (emu::ctx.bdim)
#define gridDim (emu::ctx.gdim)
#define FINETUNE_DYNAMIC_LDS(name) float* name = emu::dyn_lds
#define FINETUNE_MAX3(out, a, b, c) out = std::fmax(std::fmax(a, b), c)
#define FINETUNE_OPAQUE(x) (void)(x)

inline void __syncthreads() { pthread_barrier_wait(emu::ctx.group); }

#define __builtin_amdgcn_update_dpp(old, v, ctrl, row, bank, bound) emu::dpp(v, ctrl)
#define __builtin_amdgcn_permlane16_swap(a, b, x, y) emu::swap_runs(a, b, 16)
#define __builtin_amdgcn_permlane32_swap(a, b, x, y) emu::swap_runs(a, b, 32)
#define __builtin_amdgcn_exp2f(x) std::exp2(x)

inline float __shfl_xor(float v, int mask, int) {
  return __builtin_bit_cast(float, emu::lane_read(__builtin_bit_cast(uint32_t, v), [mask](unsigned l) { return l ^ mask; }));
}
inline float __uint_as_float(uint32_t u) { return __builtin_bit_cast(float, u); }

#define hipLaunchKernelGGL(kernel, grid, block, lds, stream, ...) \
  emu::launch(grid, block, lds, [=]() { kernel(__VA_ARGS__); })
