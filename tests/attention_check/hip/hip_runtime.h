// hip/hip_runtime.h stand-in for running the sublayer kernels on CPU threads:
// the one of the fine-tuning kernels, and with it
//   * the matrix instructions and the LDS's transposed reads as exchanges
//     between the wave's 64 threads;
//   * a wave's LDS fence as a barrier of its threads.
// Test infrastructure only.
#pragma once

#include "../../finetune_check/hip/hip_runtime.h"

#include <climits>

using std::fabs;
using std::log2;

namespace emu {

typedef float Sixteen __attribute__((ext_vector_type(16)));
typedef short Four __attribute__((ext_vector_type(4)));

inline float a_slots[1024][8], b_slots[1024][8];
inline short t_slots[1024][4];

// D += A B of a 32 x (2 N) and a (2 N) x 32 block, N elements of each operand a lane
template <int N, class A, class B>
inline Sixteen mfma(const A& a, const B& b, Sixteen c) {
  const unsigned t = ctx.tid.x, base = t / 64 * 64, l = t % 64;
  for (int k = 0; k < N; ++k) a_slots[t][k] = static_cast<float>(a[k]), b_slots[t][k] = static_cast<float>(b[k]);
  pthread_barrier_wait(ctx.wave);
  for (unsigned r = 0; r < 16; ++r) {
    const unsigned row = 8 * (r / 4) + 4 * (l / 32) + r % 4;
    float s = c[r];
    for (int k = 0; k < 2 * N; ++k)
      s += a_slots[base + row + 32 * (k / N)][k % N] * b_slots[base + l % 32 + 32 * (k / N)][k % N];
    c[r] = s;
  }
  pthread_barrier_wait(ctx.wave);
  return c;
}
struct One {
  float v;
  float operator[](int) const { return v; }
};

inline Four read_transposed(const uint16_t* p) {
  const unsigned t = ctx.tid.x, base = t / 16 * 16, i = t % 16;
  for (int k = 0; k < 4; ++k) t_slots[t][k] = static_cast<short>(p[k]);
  pthread_barrier_wait(ctx.wave);
  Four r;
  for (int k = 0; k < 4; ++k) r[k] = t_slots[base + 4 * k + i / 4][i % 4];
  pthread_barrier_wait(ctx.wave);
  return r;
}

inline bool any(bool v) {
  const unsigned t = ctx.tid.x, base = t / 64 * 64;
  slots[t] = v;
  pthread_barrier_wait(ctx.wave);
  bool r = false;
  for (unsigned l = 0; l < 64; ++l) r = r || slots[base + l];
  pthread_barrier_wait(ctx.wave);
  return r;
}

}  // namespace emu

#define __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, x, y, z) emu::mfma<8>(a, b, c)
#define __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, x, y, z) emu::mfma<8>(a, b, c)
#define __builtin_amdgcn_mfma_f32_32x32x2f32(a, b, c, x, y, z) emu::mfma<1>(emu::One{a}, emu::One{b}, c)
#define __builtin_amdgcn_sched_barrier(mask) (void)0
#define __any(v) emu::any(v)
#define FINETUNE_READ_TRANSPOSED(p) emu::read_transposed(p)
#define FINETUNE_WAVE_FENCE() pthread_barrier_wait(emu::ctx.wave)
