// Routing by scores: s = sigmoid(l) or softmax(l); keys s + bias choose the
// experts (within the best groups, where there are groups), the raw scores
// make the gates, renormalised over the selected and scaled on request.
//
// Selected ids are whole numbers, so the keys must be ordered as the formula
// orders them: keys are computed in fp64.  One wavefront per token; lane l
// holds experts l, l + 64, ...
#include "common.h"
#include "kernels.h"

namespace moe {
namespace {

constexpr double kNone = -__builtin_huge_val();

__device__ __forceinline__ double shfl_xor_f64(double v, int m) {
  const uint64_t b = __double_as_longlong(v);
  const uint32_t lo = __shfl_xor(static_cast<uint32_t>(b), m), hi = __shfl_xor(static_cast<uint32_t>(b >> 32), m);
  return __longlong_as_double((static_cast<uint64_t>(hi) << 32) | lo);
}

// The (key, index) pair that comes first: larger key, then lower index.
__device__ __forceinline__ void take_first(double& key, int& idx, double k2, int i2) {
  if (k2 > key || (k2 == key && i2 < idx)) {
    key = k2;
    idx = i2;
  }
}
__device__ __forceinline__ void wave_first(double& key, int& idx) {
  for (int m = 1; m < 64; m <<= 1) take_first(key, idx, shfl_xor_f64(key, m), __shfl_xor(idx, m));
}

// Score of one logit; softmax scores from the row's maximum and sum.
__device__ __forceinline__ double score64(const ScoreArgs& a, float l, double m, double sum) {
  return a.sigmoid ? 1.0 / (1.0 + exp(-(double)l)) : exp((double)l - m) / sum;
}

// One wavefront: the token's selected ids and gates from fp64 keys.  keys: E
// doubles of LDS of this wavefront (read where there are groups).
template <int NPER>
__device__ __forceinline__ void select_token(const ScoreArgs& a, const float* __restrict__ row,
                                             const float* __restrict__ bias, double* keys, int32_t* topk,
                                             float* gates) {
  const int lane = threadIdx.x & 63;
  const int E = a.E;
  float v[NPER];
#pragma unroll
  for (int i = 0; i < NPER; ++i) v[i] = row[min(i * 64 + lane, E - 1)];
  double m = 0.0, sum = 1.0;
  if (!a.sigmoid) {
    float mx = -3.402823466e38f;  // a row of -inf alone keeps this: every exponential is then 0
#pragma unroll
    for (int i = 0; i < NPER; ++i) mx = fmaxf(mx, v[i]);
    for (int d = 1; d < 64; d <<= 1) mx = fmaxf(mx, __shfl_xor(mx, d));
    m = mx;
    sum = 0.0;
#pragma unroll
    for (int i = 0; i < NPER; ++i)
      if (i * 64 + lane < E) sum += exp((double)v[i] - m);
    for (int d = 1; d < 64; d <<= 1) sum += shfl_xor_f64(sum, d);
    sum = fmax(sum, 1e-300);
  }
  double key[NPER];
  uint32_t open = 0;  // bit i: this lane's expert i can still be taken
#pragma unroll
  for (int i = 0; i < NPER; ++i) {
    const int e = i * 64 + lane;
    key[i] = kNone;
    if (e < E) {
      const double x = score64(a, v[i], m, sum) + (bias ? (double)bias[e] : 0.0);
      key[i] = x == x ? x : kNone;
      open |= 1u << i;
    }
  }
  if (a.groups > 1) {
    const int gs = E / a.groups;
#pragma unroll
    for (int i = 0; i < NPER; ++i)
      if (i * 64 + lane < E) keys[i * 64 + lane] = key[i];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    double gsc = kNone;
    if (lane < a.groups) {
      double t1 = kNone, t2 = kNone;
      for (int j = 0; j < gs; ++j) {
        const double x = keys[lane * gs + j];
        t2 = x > t1 ? t1 : fmax(t2, x);
        t1 = fmax(t1, x);
      }
      gsc = a.group_top == 2 && gs > 1 ? t1 + t2 : t1;
    }
    uint64_t kept = 0;
    bool mine = lane < a.groups;
    for (int j = 0; j < a.top_groups; ++j) {
      double best = mine ? gsc : kNone;
      int g = mine ? lane : 1 << 20;
      wave_first(best, g);
      kept |= 1ull << (g & 63);
      if (lane == g) mine = false;
    }
#pragma unroll
    for (int i = 0; i < NPER; ++i) {
      const int e = i * 64 + lane;
      if (e < E && !((kept >> (e / gs)) & 1)) open &= ~(1u << i);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
  int sel = 0;  // lane j < k ends with the j-th selected expert
  for (int j = 0; j < a.k; ++j) {
    double best = kNone;
    int e = 1 << 20;
#pragma unroll
    for (int i = 0; i < NPER; ++i)
      if ((open >> i) & 1) take_first(best, e, key[i], i * 64 + lane);
    wave_first(best, e);
    if ((e & 63) == lane) open &= ~(1u << (e >> 6));
    if (lane == j) sel = e;
  }
  const bool on = lane < a.k;
  const double s = on ? score64(a, row[sel], m, sum) : 0.0;
  double S = 1.0;
  if (a.renorm) {
    S = s;
    for (int d = 1; d < 64; d <<= 1) S += shfl_xor_f64(S, d);
    S += 1e-20;
  }
  if (on) {
    topk[lane] = sel;
    gates[lane] = (float)(s / S * (double)a.scale);
  }
}

template <int NPER>
__global__ __launch_bounds__(256) void route_scored_kernel(ScoreArgs a, const float* __restrict__ logits,
                                                           const float* __restrict__ bias, int32_t* topk,
                                                           float* gates) {
  __shared__ double keys[4][NPER * 64];
  const int w = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * 4 + w;
  if (t >= a.T) return;
  select_token<NPER>(a, logits + t * a.E, bias, keys[w], topk + t * a.k, gates + t * a.k);
}

// Gradient: ds_j of the selected scores (lane j), then the row.
template <int NPER>
__global__ __launch_bounds__(256) void route_scored_bwd_kernel(ScoreArgs a, const float* __restrict__ logits,
                                                               const int32_t* __restrict__ topk,
                                                               const float* __restrict__ d_gates, float* d_logits) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= a.T) return;
  const int E = a.E;
  const float* row = logits + t * E;
  int idx = -1;
  float dg = 0.0f;
  if (lane < a.k) {
    idx = topk[t * a.k + lane];
    dg = d_gates[t * a.k + lane] * a.scale;
  }
  const bool on = idx >= 0 && idx < E;
  const float l = row[on ? idx : 0];
  float p[NPER];
  float s, rest = 0.0f;  // rest: 1 - sigmoid, from its own formula (1 - s loses bits near 1)
  if (a.sigmoid) {
    const float x = expf(-fabsf(l)), r = 1.0f / (1.0f + x);
    s = on ? (l >= 0.0f ? r : x * r) : 0.0f;
    rest = l >= 0.0f ? x * r : r;
  } else {
    float mx = -3.402823466e38f, sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NPER; ++i) p[i] = row[min(i * 64 + lane, E - 1)];
#pragma unroll
    for (int i = 0; i < NPER; ++i) mx = fmaxf(mx, p[i]);
    for (int d = 1; d < 64; d <<= 1) mx = fmaxf(mx, __shfl_xor(mx, d));
#pragma unroll
    for (int i = 0; i < NPER; ++i) {
      p[i] = i * 64 + lane < E ? expf(p[i] - mx) : 0.0f;
      sum += p[i];
    }
    for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
    sum = fmaxf(sum, 1e-37f);
#pragma unroll
    for (int i = 0; i < NPER; ++i) p[i] = p[i] / sum;
    s = on ? expf(l - mx) / sum : 0.0f;
  }
  if (!on) dg = 0.0f;
  float ds = dg;
  if (a.renorm) {
    float S = s, dot = dg * s;
    for (int d = 1; d < 64; d <<= 1) {
      S += __shfl_xor(S, d);
      dot += __shfl_xor(dot, d);
    }
    S += 1e-20f;
    ds = on ? (dg - dot / S) / S : 0.0f;
  }
  float base = 0.0f;
  float val;
  if (a.sigmoid) {
    val = ds * s * rest;
  } else {
    val = ds;
    base = ds * s;
    for (int d = 1; d < 64; d <<= 1) base += __shfl_xor(base, d);
  }
  float out[NPER];
#pragma unroll
  for (int i = 0; i < NPER; ++i) out[i] = -base;
  for (int j = 0; j < a.k; ++j) {
    const int e = __shfl(on ? idx : -1, j);
    const float x = __shfl(val, j);
#pragma unroll
    for (int i = 0; i < NPER; ++i)
      if (e == i * 64 + lane) out[i] += x;
  }
#pragma unroll
  for (int i = 0; i < NPER; ++i)
    if (i * 64 + lane < E) d_logits[t * E + i * 64 + lane] = a.sigmoid ? out[i] : out[i] * p[i];
}

}  // namespace

// f(NPER) with the smallest instantiated NPER >= ceil(E / 64)
#define MOE_BY_EXPERTS(E, CALL)  \
  do {                           \
    const int nper = ((E) + 63) / 64; \
    if (nper <= 1) { CALL(1); }  \
    else if (nper <= 2) { CALL(2); } \
    else if (nper <= 4) { CALL(4); } \
    else if (nper <= 6) { CALL(6); } \
    else if (nper <= 8) { CALL(8); } \
    else { CALL(16); }           \
  } while (0)

hipError_t launch_route_scored(const ScoreArgs& a, const float* logits, const float* bias, int32_t* topk,
                               float* gates, hipStream_t s) {
  if (a.T <= 0) return hipSuccess;
  const dim3 grid((unsigned)((a.T + 3) / 4));
#define CALL(N) route_scored_kernel<N><<<grid, 256, 0, s>>>(a, logits, bias, topk, gates)
  MOE_BY_EXPERTS(a.E, CALL);
#undef CALL
  return hipGetLastError();
}

hipError_t launch_route_scored_bwd(const ScoreArgs& a, const float* logits, const int32_t* topk,
                                   const float* d_gates, float* d_logits, hipStream_t s) {
  if (a.T <= 0) return hipSuccess;
  const dim3 grid((unsigned)((a.T + 3) / 4));
#define CALL(N) route_scored_bwd_kernel<N><<<grid, 256, 0, s>>>(a, logits, topk, d_gates, d_logits)
  MOE_BY_EXPERTS(a.E, CALL);
#undef CALL
  return hipGetLastError();
}

}  // namespace moe
