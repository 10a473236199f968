// Weights straight from memory into matrix instructions: the products of at
// most a few blocks of 16 rows, bound by the weights' bytes.
//
// The wavefronts of a workgroup share K, 64 values of it at a time.  Each has
// two groups of such units in flight in registers: one is loaded while the
// other feeds the matrix instructions.
#pragma once

#include "common.h"

namespace moe {

__device__ __forceinline__ f32x4_t mfma_bf16(const uint4& a, const uint4& b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0,
                                                 0, 0);
}

// One wavefront's share of acc[s][p] += W_s x_p^T: kSets matrices of 16 rows
// by kX row blocks (or bf16 parts of one).  w and x: this lane's row of each, 8
// (lane >> 4) values in; units: 64-value units of K in all.  load(p): 16 bytes
// from p on.  kJoin: all x are parts of the same rows, summed into acc[s][0].
template <int kWaves, int kSets, int kX, bool kJoin, int kDepth, int kAcc, class Load>
__device__ __forceinline__ void stream(const uint16_t* const (&w)[kSets], const uint16_t* const (&x)[kX], int units,
                                       f32x4_t (&acc)[kSets][kAcc], Load&& load) {
  static_assert(kAcc == (kJoin ? 1 : kX), "one sum a row block");
  constexpr int U = kDepth / (kSets + kX) > 0 ? kDepth / (kSets + kX) : 1;  // units a group: 8 kDepth registers
  struct Group {
    uint4 a[U][kSets][2], b[U][kX][2];
  };
  const int wave = threadIdx.x >> 6;
  auto fetch = [&](int first, Group& g) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int unit = first + u * kWaves;
      if (unit < units) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int s = 0; s < kSets; ++s) g.a[u][s][i] = load(w[s] + unit * 64 + 32 * i);
#pragma unroll
          for (int p = 0; p < kX; ++p) g.b[u][p][i] = load(x[p] + unit * 64 + 32 * i);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int s = 0; s < kSets; ++s) g.a[u][s][i] = make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int p = 0; p < kX; ++p) g.b[u][p][i] = make_uint4(0, 0, 0, 0);
        }
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  auto sums = [&](const Group& g) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int p = kX - 1; p >= 0; --p)
#pragma unroll
          for (int s = 0; s < kSets; ++s) {
            f32x4_t& c = acc[s][kJoin ? 0 : p];
            c = mfma_bf16(g.a[u][s][i], g.b[u][p][i], c);
          }
    __builtin_amdgcn_sched_barrier(0);
  };
  constexpr int kStep = U * kWaves;
  Group g0, g1;
  int at = __builtin_amdgcn_readfirstlane(wave);
  if (at >= units) return;
  fetch(at, g0);
  for (; at < units; at += 2 * kStep) {
    fetch(at + kStep, g1);
    sums(g0);
    if (at + kStep >= units) return;
    fetch(at + 2 * kStep, g0);
    sums(g1);
  }
}

}  // namespace moe
