// Router selection: top-k by fl32(logit + bias) with ties to the lower expert
// index, and gates = softmax over the selected raw logits.
// One wavefront per token (select.h).
#include "common.h"
#include "kernels.h"
#include "select.h"

namespace moe {
namespace {

template <int NPER>  // experts per lane: E <= 64 * NPER
__global__ __launch_bounds__(256) void topk_gates_kernel(const float* __restrict__ logits,
                                                         const float* __restrict__ bias,
                                                         int64_t T, int E, int k,
                                                         int32_t* __restrict__ topk,
                                                         float* __restrict__ gates) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= T) return;
  int mine;
  float gate;
  const float* __restrict__ row = logits + t * E;
  select_topk_of<NPER>([&](int e) { return row[e]; }, bias, E, k, mine, gate);
  if (lane < k) {
    topk[t * k + lane] = mine;
    gates[t * k + lane] = gate;
  }
}

}  // namespace

hipError_t launch_topk_gates(const float* logits, const float* bias, int64_t T, int E, int k,
                             int32_t* topk_idx, float* gates, hipStream_t s) {
  if (T <= 0) return hipSuccess;
  const int64_t blocks = (T + 3) / 4;
  const dim3 grid((unsigned)blocks);
  const int nper = (E + 63) / 64;
  if (nper <= 1)
    topk_gates_kernel<1><<<grid, 256, 0, s>>>(logits, bias, T, E, k, topk_idx, gates);
  else if (nper <= 2)
    topk_gates_kernel<2><<<grid, 256, 0, s>>>(logits, bias, T, E, k, topk_idx, gates);
  else if (nper <= 4)
    topk_gates_kernel<4><<<grid, 256, 0, s>>>(logits, bias, T, E, k, topk_idx, gates);
  else if (nper <= 6)
    topk_gates_kernel<6><<<grid, 256, 0, s>>>(logits, bias, T, E, k, topk_idx, gates);
  else if (nper <= 8)
    topk_gates_kernel<8><<<grid, 256, 0, s>>>(logits, bias, T, E, k, topk_idx, gates);
  else
    topk_gates_kernel<16><<<grid, 256, 0, s>>>(logits, bias, T, E, k, topk_idx, gates);
  return hipGetLastError();
}

}  // namespace moe
