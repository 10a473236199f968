// Routing by scores: s = sigmoid(l) or softmax(l); keys s + bias choose the
// experts (within the best groups, where there are groups), the raw scores
// make the gates, renormalised over the selected and scaled on request.
//
// Selected ids are whole numbers, so the keys must be ordered as the formula
// orders them, whatever an fp32 exponential rounds to.  For k <= 8 a token is
// first selected from fp32 keys by 16 lanes, four tokens to a wavefront.  Where
// keys that matter lie closer than their error bound (one token in 500 to 1000
// for random logits of deviation 1.5, by the bound itself; one in 10^4 for
// sharp softmax scores), the few near the edge are compared by fp64 keys, one
// per lane; where they are more than 16, and for every other shape, one
// wavefront selects the token from fp64 keys.  Sigmoids of many logits far
// above 10 and no bias are such a batch: fp32 scores all round to 1.
//
// Measured, 16384 tokens of 384 experts, top-8, in us: the best 4 of 8 groups,
// with a bias, sigmoid 12.5, softmax 17.1 (its error bound's logarithms, the
// sum and the largest bias); no groups 11.2 and 15.2, no bias either 7.3 and
// 7.7.  The sorting networks' issue, not the bytes' 5, bounds them.  Saturated
// sigmoids (logits of deviation 8 and above without a bias): 60 to 90.  k > 8:
// top-12 of 384 54, top-10 and top-16 of 512 55 and 79.  Gradients: sigmoid 7.1,
// softmax 10.6.  One token 4.2, a launch and its chain of exchanges.
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
      key[i] = x == x ? fmin(x, 1e300) : kNone;  // so that no sum of two is a NaN
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

// ------------------------------------------------------- 16 lanes a token
// Keys as doubles with the expert in the low mantissa bits (an fp32 key
// leaves 29 free), so that one fp64 maximum carries key and index, the lower
// index first among equal keys.  A lane reduces its experts to the 8 largest,
// sorted, by merging sorted lists of 8; four exchanges within the 16 lanes
// merge those, after which every lane holds the token's 8 largest in order.
//
// How far an fp32 key can be from the formula's, u = 2^-24 the rounding unit:
//   sigmoid: the exponential of l is off by 4 u l + 2 u relatively, which
//     moves s by s (1 - s) of that (<= 0.23 * 4 u + 0.25 * 2 u); 1 + e and the
//     reciprocal add 3 u s: within 4.5 u
//   softmax p = e^-d / S, d = max - l: e^-d is off by 4 u d + 4 u relatively,
//     the product with 1 / S by u, and p d = p ln(1/(p S)): within u (5 p +
//     4 m / S), m the largest t ln(1/t) of any t <= p S.  This shrinks with
//     the score, which a key x bounds by |x| and the largest bias: far from
//     the largest logit, where most of a sharp softmax lies, keys are told
//     apart as well as near it.  S itself (NPER + 4 additions, the
//     exponentials' own errors) is a factor common to all p, within (NPER +
//     24) u, and turns two keys around only by that factor of their p's
//     difference, which at a near tie is the difference of two biases
//   adding the bias: u |key|.  Scores below 2^-126 are flushed to 0.
// Two keys closer than both errors are not told apart here, nor two groups
// whose scores, each with its keys' errors (those of the keys, which a sum of
// opposite ones does not show) and its own rounding, overlap.  Without a bias
// and without groups the logits themselves are the keys: exact, as long as
// fp64 scores still separate what fp32 logits separate.
constexpr int kTop = 8;

__device__ __forceinline__ double pack_key(float key, int e) {
  // The sum turns -0.0 into the 0.0 it equals (its sign bit would also ask for
  // the other form of the index) and quiets a NaN, of which the median makes
  // the least value; an infinity has no mantissa to carry an index.
  const float f = __builtin_amdgcn_fmed3f(key + 0.0f, -3.402823466e38f, 3.402823466e38f);
  const uint64_t b = (uint64_t)__double_as_longlong((double)f);
  return __longlong_as_double((long long)(b | (uint32_t)(f < 0.0f ? e : 1023 - e)));
}
__device__ __forceinline__ int packed_expert(uint32_t lo, uint32_t hi) {
  const int i = (int)(lo & 1023);
  return (hi >> 31) ? i : 1023 - i;
}
__device__ __forceinline__ float packed_key(double d) {
  const uint64_t b = (uint64_t)__double_as_longlong(d) & ~(uint64_t)1023;
  return (float)__longlong_as_double((long long)b);
}

// Maximum and minimum as single instructions: packed keys are never NaN, and
// fmax / fmin would quiet each operand first.
__device__ __forceinline__ double max64(double a, double b) {
  double r;
  asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}
__device__ __forceinline__ double min64(double a, double b) {
  double r;
  asm("v_min_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}

__device__ __forceinline__ void order(double& a, double& b) {  // larger first
  const double x = max64(a, b), y = min64(a, b);
  a = x;
  b = y;
}

// Descending sort of 8 (odd-even merge sort, 19 exchanges).
__device__ __forceinline__ void sort8(double* v) {
  order(v[0], v[1]); order(v[2], v[3]); order(v[4], v[5]); order(v[6], v[7]);
  order(v[0], v[2]); order(v[1], v[3]); order(v[4], v[6]); order(v[5], v[7]);
  order(v[1], v[2]); order(v[5], v[6]);
  order(v[0], v[4]); order(v[1], v[5]); order(v[2], v[6]); order(v[3], v[7]);
  order(v[2], v[4]); order(v[3], v[5]);
  order(v[1], v[2]); order(v[3], v[4]); order(v[5], v[6]);
}

// v = the 8 largest of two descending lists: their element-wise maximum with
// one reversed is bitonic.
__device__ __forceinline__ void merge8(double* v, const double* o) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = max64(v[i], o[7 - i]);
#pragma unroll
  for (int d = 4; d > 0; d >>= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if ((i & d) == 0) order(v[i], v[i + d]);
}

// Partner's value in the n-th exchange of 16 lanes: lane ^ 1, lane ^ 2, the
// mirror within 8, the mirror within 16 (each pairs lanes whose values still
// differ).
template <int kStep>
__device__ __forceinline__ uint32_t partner(uint32_t v) {
  constexpr int ctrl = kStep == 0 ? 0xB1 : kStep == 1 ? 0x4E : kStep == 2 ? 0x141 : 0x140;
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, 0xF, 0xF, false);
}
template <int kStep>
__device__ __forceinline__ double partner(double v) {
  const uint64_t b = (uint64_t)__double_as_longlong(v);
  const uint64_t lo = partner<kStep>((uint32_t)b), hi = partner<kStep>((uint32_t)(b >> 32));
  return __longlong_as_double((long long)(lo | (hi << 32)));
}
template <int kStep>
__device__ __forceinline__ float partner(float v) {
  return __uint_as_float(partner<kStep>(__float_as_uint(v)));
}
__device__ __forceinline__ float min16(float v) {
  v = fminf(v, partner<0>(v));
  v = fminf(v, partner<1>(v));
  v = fminf(v, partner<2>(v));
  return fminf(v, partner<3>(v));
}
__device__ __forceinline__ float max16(float v) {
  v = fmaxf(v, partner<0>(v));
  v = fmaxf(v, partner<1>(v));
  v = fmaxf(v, partner<2>(v));
  return fmaxf(v, partner<3>(v));
}
__device__ __forceinline__ float sum16(float v) {
  v += partner<0>(v);
  v += partner<1>(v);
  v += partner<2>(v);
  return v + partner<3>(v);
}
template <int kStep>
__device__ __forceinline__ void merge_partner(double* v) {
  double o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = partner<kStep>(v[i]);
  merge8(v, o);
}

// Where lane c's i-th value lies: expert (i / V) * step + c * lane_step + i %
// V (V values per load), i below `per`.  full: every lane's NPER values exist.
struct LaneMap {
  int step, lane_step, per;
  bool full;
};
template <int V>
__device__ __forceinline__ int mapped(const LaneMap& m, int c, int i) {
  return (i / V) * m.step + c * m.lane_step + i % V;
}

template <int NPER, int V>
__device__ __forceinline__ void load_row(const float* __restrict__ row, int E, const LaneMap& m, int c, float* v) {
#pragma unroll
  for (int i = 0; i < NPER; i += V) {
    const int e = min(mapped<V>(m, c, i), E - V);  // past the end: not used
    if constexpr (V == 4) {
      const f32x4_t x = *reinterpret_cast<const f32x4_t*>(row + e);
#pragma unroll
      for (int q = 0; q < 4; ++q) v[i + q] = x[q];
    } else {
      v[i] = row[e];
    }
  }
}
template <int NPER, int V>
__device__ __forceinline__ void mask_row(int E, const LaneMap& m, int c, float* v) {
  if (m.full) return;
#pragma unroll
  for (int i = 0; i < NPER; ++i) v[i] = (i < m.per) & (mapped<V>(m, c, i) < E) ? v[i] : -__builtin_huge_valf();
}

// Tokens whose selection hangs on keys too close for fp32 (`again`, equal in
// the 16 lanes of a token): the experts whose keys reach `edge`, at most 16,
// are compared by fp64 keys, one per lane.  cand: 64 ints of LDS of this
// wavefront.
template <int NPER, int V, bool kSigmoid>
__device__ __forceinline__ void select_close(const ScoreArgs& a, const LaneMap& map, const float* __restrict__ row,
                                             const float* __restrict__ bias, const float* key, float edge, float mx,
                                             bool again, int* cand, int32_t* topk, float* gates) {
  const int lane = threadIdx.x & 63, c = lane & 15;
  int* mine = cand + (lane & 48);
  int n = 0;
#pragma unroll
  for (int i = 0; i < NPER; ++i) {
    const bool take = again && key[i] >= edge;
    const uint32_t m = (uint32_t)(ballot64(take) >> (lane & 48)) & 0xFFFF;
    const int at = n + __popc(m & ((1u << c) - 1));
    if (take && at < 16) mine[at] = mapped<V>(map, c, i);
    n += __popc(m);
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  const bool on = again && c < min(n, 16);
  const int e = on ? mine[c] : 0;
  const float l = row[e];
  double s;
  if constexpr (kSigmoid) {
    s = score64(a, l, 0.0, 1.0);
  } else {
    double sum = 0.0;
    for (int j = c; j < a.E; j += 16) sum += exp((double)row[j] - (double)mx);
    for (int d = 1; d < 16; d <<= 1) sum += shfl_xor_f64(sum, d);
    s = score64(a, l, mx, fmax(sum, 1e-300));
  }
  const double x = s + (bias ? (double)bias[e] : 0.0);
  int rank = 0;
  for (int j = 0; j < 16; ++j) {
    const int from = (lane & 48) + j;
    const uint64_t b = (uint64_t)__double_as_longlong(x);
    const uint64_t lo = __shfl((uint32_t)b, from), hi = __shfl((uint32_t)(b >> 32), from);
    const double o = __longlong_as_double((long long)(lo | (hi << 32)));
    const int oe = __shfl(e, from);
    rank += (j < n && (o > x || (o == x && oe < e))) ? 1 : 0;
  }
  const bool sel = on && rank < a.k;
  double S = 1.0;
  if (a.renorm) {
    S = sel ? s : 0.0;
    for (int d = 1; d < 16; d <<= 1) S += shfl_xor_f64(S, d);
    S += 1e-20;
  }
  if (sel) {
    topk[rank] = e;
    gates[rank] = (float)(s / S * (double)a.scale);
  }
}

// Whether this lane's group stays, by fp64 keys: those of the lane's 4 largest
// fp32 keys hold its two largest, unless the fifth is too close to the second
// (`margin`: how far those two can be off together) or the lane has no two
// (`unsettled`).
template <bool kSigmoid>
__device__ __forceinline__ bool groups64(const ScoreArgs& a, const float* __restrict__ row,
                                         const float* __restrict__ bias, float mx, const double* top, float margin,
                                         int g, int span, bool& unsettled) {
  const int lane = threadIdx.x & 63, c = lane & 15;
  double sum = 1.0;
  if constexpr (!kSigmoid) {
    sum = 0.0;
    for (int j = c; j < a.E; j += 16) sum += exp((double)row[j] - (double)mx);
    for (int d = 1; d < 16; d <<= 1) sum += shfl_xor_f64(sum, d);
    sum = fmax(sum, 1e-300);
  }
  unsettled = !(packed_key(top[1]) - packed_key(top[4]) > margin && packed_key(top[1]) > -3.0e38f);
  double t1 = kNone, t2 = kNone;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint64_t b = (uint64_t)__double_as_longlong(top[j]);
    const int e = min(packed_expert((uint32_t)b, (uint32_t)(b >> 32)), a.E - 1);
    double x = score64(a, row[e], mx, sum) + (bias ? (double)bias[e] : 0.0);
    if (!(packed_key(top[j]) > -3.0e38f)) x = kNone;
    t2 = fmax(t2, fmin(t1, x));
    t1 = fmax(t1, x);
  }
  for (int d = 1; d < span; d <<= 1) {
    const double o1 = shfl_xor_f64(t1, d), o2 = shfl_xor_f64(t2, d);
    t2 = fmax(fmin(t1, o1), fmax(t2, o2));
    t1 = fmax(t1, o1);
  }
  const double s = a.group_top == 2 && a.E > a.groups ? t1 + t2 : t1;
  int before = 0;
  for (int o = 0; o < a.groups; ++o) {
    const int from = (lane & 48) + o * span;
    const uint64_t b = (uint64_t)__double_as_longlong(s);
    const uint64_t lo = __shfl((uint32_t)b, from), hi = __shfl((uint32_t)(b >> 32), from);
    const double x = __longlong_as_double((long long)(lo | (hi << 32)));
    before += (x > s || (x == s && o < g)) ? 1 : 0;
  }
  return before < a.top_groups;
}

// kLogit: the logits are the keys (no bias, no groups).
template <int NPER, int V, bool kSigmoid, bool kLogit>
__global__ __launch_bounds__(256) void route_top8_kernel(ScoreArgs a, LaneMap map, const float* __restrict__ logits,
                                                         const float* __restrict__ bias, int32_t* __restrict__ topk,
                                                         float* __restrict__ gates) {
  constexpr int NPER64 = (NPER + 3) / 4;  // experts per lane of a whole wavefront
  __shared__ double keys64[4][NPER64 * 64];
  __shared__ int cand[4][64];
  const int lane = threadIdx.x & 63, c = lane & 15, wave = threadIdx.x >> 6;
  const int64_t t0 = ((int64_t)blockIdx.x * 4 + wave) * 4;
  if (t0 >= a.T) return;
  const bool exists = t0 + (lane >> 4) < a.T;
  const int64_t t = exists ? t0 + (lane >> 4) : a.T - 1;
  const int E = a.E;
  const float* row = logits + t * E;
  float key[NPER];
  load_row<NPER, V>(row, E, map, c, key);
  mask_row<NPER, V>(E, map, c, key);
  // `hard`: left to the whole wavefront's fp64 selection
  bool hard = false;
  float mx = 0.0f, sum = 1.0f, bmax = 0.0f;
  if (!kSigmoid || kLogit) {
    mx = -3.402823466e38f;
#pragma unroll
    for (int i = 0; i < NPER; ++i) mx = fmaxf(mx, key[i]);
    mx = max16(mx);
  }
  if constexpr (!kSigmoid) {
    float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NPER; ++i) {
      const float p = __expf(key[i] - mx);
      if constexpr (!kLogit) key[i] = p;
      part[i & 3] += p;
    }
    sum = fmaxf(sum16((part[0] + part[1]) + (part[2] + part[3])), 1e-37f);
  }
  if constexpr (kLogit) {
    // fp64 sigmoids of neighbouring fp32 logits coincide above about 20
    if (kSigmoid) hard = !(mx <= 20.0f);
  } else {
    const float r = 1.0f / sum;
#pragma unroll
    for (int i = 0; i < NPER; ++i) key[i] = kSigmoid ? sigmoid(key[i]) : key[i] * r;
    if (bias) {
      float b[NPER];
      load_row<NPER, V>(bias, E, map, c, b);
#pragma unroll
      for (int i = 0; i < NPER; ++i) key[i] += b[i];
      if constexpr (!kSigmoid) {
#pragma unroll
        for (int i = 0; i < NPER; ++i) bmax = fmaxf(bmax, fabsf(b[i]));
        bmax = max16(bmax);
      }
    }
    mask_row<NPER, V>(E, map, c, key);
  }
  double top[kTop];
#pragma unroll
  for (int i = 0; i < NPER; i += kTop) {
    double l[kTop];
#pragma unroll
    for (int j = 0; j < kTop; ++j)
      l[j] = i + j < NPER ? pack_key(key[i + j], mapped<V>(map, c, i + j)) : -__builtin_huge_val();
    sort8(l);
    if (i == 0) {
#pragma unroll
      for (int j = 0; j < kTop; ++j) top[j] = l[j];
    } else {
      merge8(top, l);
    }
  }
  // how far an fp32 key x can be off, and the difference below which two keys
  // of magnitude up to x are not told apart
  constexpr float u = 5.9604645e-8f;
  auto off = [&](float x) {
    x = fminf(fabsf(x), 3.402823466e38f);
    if constexpr (kSigmoid) return 8.0f * u + 2.0f * u * x;
    const float p = fminf(x + bmax, 1.0f / sum);  // at least the score
    const float t = __builtin_amdgcn_fmed3f(p * sum, 1e-36f, 0.36787944f);
    return u * (6.0f * p - 5.0f * t * __logf(t) / sum + 1.25f * x) + 1e-36f +
           0.5f * (NPER + 24) * u * fminf(1.0f, 2.0f * bmax);
  };
  auto tol = [&](float x) {
    if constexpr (kLogit) return 0x1p-30f * (1.0f + fabsf(x));  // fp64 scores still differ by it
    return 2.0f * off(x);
  };
  float shut = 0.0f;  // -inf where this lane's experts cannot be taken
  if constexpr (!kLogit) {
    if (a.groups > 1) {
      // a lane's experts are of one group, groups are 16 / G neighbouring lanes
      const int span = 16 / a.groups;
      double t1 = top[0], t2 = top[1];
      auto join = [&](double o1, double o2) {
        t2 = max64(min64(t1, o1), max64(t2, o2));
        t1 = max64(t1, o1);
      };
      if (span > 1) join(partner<0>(t1), partner<0>(t2));
      if (span > 2) join(partner<1>(t1), partner<1>(t2));
      if (span > 4) join(partner<2>(t1), partner<2>(t2));
      const bool two = a.group_top == 2 && t2 > -1e300;
      const float k1 = packed_key(t1), k2 = packed_key(t2), gsc = two ? k1 + k2 : k1;
      const float gerr = off(k1) + (two ? off(k2) + u * fabsf(gsc) : 0.0f);
      const int g = c / span;
      int before = 0;
      for (int o = 0; o < a.groups; ++o) {
        const float s = __shfl(gsc, (lane & 48) + o * span);
        before += (s > gsc || (s == gsc && o < g)) ? 1 : 0;
      }
      bool in = before < a.top_groups;
      const float low = min16(in ? gsc - gerr : 3.402823466e38f), high = max16(in ? -3.402823466e38f : gsc + gerr);
      const bool close_groups = !(low > high);
      if (ballot64(close_groups) != 0) {
        bool unsettled;
        const float margin = off(packed_key(top[1])) + off(packed_key(top[4]));
        const bool in64 = groups64<kSigmoid>(a, row, bias, mx, top, margin, g, span, unsettled);
        in = close_groups ? in64 : in;
        hard = hard || (close_groups && unsettled);
      }
      if (!in) {
        shut = -__builtin_huge_valf();
#pragma unroll
        for (int j = 0; j < kTop; ++j) top[j] = -__builtin_huge_val();
      }
    }
  }
  merge_partner<0>(top);
  merge_partner<1>(top);
  merge_partner<2>(top);
  merge_partner<3>(top);
  // `close`: neighbours in order, or the last one taken and one that is not,
  // within the tolerance; lane c holds the c-th key
  uint32_t lo = 0, hi = 0;
#pragma unroll
  for (int j = 0; j < kTop; ++j) {
    const uint64_t b = (uint64_t)__double_as_longlong(top[j]);
    lo = (c & 7) == j ? (uint32_t)b : lo;
    hi = (c & 7) == j ? (uint32_t)(b >> 32) : hi;
  }
  const float own = packed_key(__longlong_as_double((long long)(((uint64_t)hi << 32) | lo)));
  const float next = __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(own), 0x101, 0xF, 0xF,
                                                                           false));  // lane c + 1
  const float last = __shfl(own, (lane & 48) + a.k - 1);
  const float gap = own - next;
  bool close = c + 1 < a.k && gap <= tol(fmaxf(fabsf(own), fabsf(next))) && !(kLogit && gap == 0.0f);
  const float edge = last - tol(last);
  int near = 0, equal = 0;
#pragma unroll
  for (int i = 0; i < NPER; ++i) {
    near += key[i] + shut >= edge ? 1 : 0;
    if constexpr (kLogit) equal += key[i] >= last ? 1 : 0;
  }
  const float n16 = sum16((float)near);
  if constexpr (kLogit) {
    close = close || n16 != sum16((float)equal);  // equal logits are exact ties: the index decided
    // fp64 scores of distant logits underflow and coincide
    hard = hard || !(last >= (kSigmoid ? -700.0f : mx - 700.0f));
  } else {
    close = close || n16 != (float)a.k;
  }
  hard = hard || !(fabsf(last) < 3.0e38f);

  // lane c < k: the c-th selected expert and its gate
  const bool on = c < a.k;
  const int e = min(packed_expert(lo, hi), E - 1);
  const float l = on ? row[e] : 0.0f;
  float s;
  if constexpr (kSigmoid) {
    const float x = expf(-fabsf(l)), r = 1.0f / (1.0f + x);
    s = l >= 0.0f ? r : x * r;
  } else {
    s = expf(l - mx) / sum;
  }
  s = on ? s : 0.0f;
  const float S = a.renorm ? sum16(s) + 1e-20f : 1.0f;
  const uint64_t closes = ballot64(close);
  const bool token_close = ((closes >> (lane & 48)) & 0xFFFF) != 0;
  const uint64_t hards = ballot64(hard || (token_close && n16 > 16.0f));
  const bool token_hard = ((hards >> (lane & 48)) & 0xFFFF) != 0;
  if (on && exists && !token_hard && !token_close) {
    topk[t * a.k + c] = e;
    gates[t * a.k + c] = s / S * a.scale;
  }
  if ((closes | hards) == 0) return;
  const bool again = exists && token_close && !token_hard;
  if (ballot64(again) != 0) {
#pragma unroll
    for (int i = 0; i < NPER; ++i) key[i] += shut;
    select_close<NPER, V, kSigmoid>(a, map, row, bias, key, edge, mx, again, cand[wave], topk + t * a.k,
                                    gates + t * a.k);
  }
  for (int i = 0; i < 4; ++i) {
    if (t0 + i >= a.T || ((hards >> (16 * i)) & 0xFFFF) == 0) continue;
    select_token<NPER64>(a, logits + (t0 + i) * E, bias, keys64[wave], topk + (t0 + i) * a.k, gates + (t0 + i) * a.k);
  }
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

// The gradient for k <= 16 and whole 16-byte rows: 16 lanes a token, four
// tokens to a wavefront, lane c holding the c-th selected expert and columns
// 64 i + 4 c .. + 3 of the row.
template <int NPER, bool kSigmoid>
__global__ __launch_bounds__(256) void route_bwd16_kernel(ScoreArgs a, const float* __restrict__ logits,
                                                          const int32_t* __restrict__ topk,
                                                          const float* __restrict__ d_gates,
                                                          float* __restrict__ d_logits) {
  __shared__ __attribute__((aligned(16))) float terms[16][NPER * 16];
  const int lane = threadIdx.x & 63, c = lane & 15;
  float* mine = terms[threadIdx.x >> 4];
  const int64_t t0 = ((int64_t)blockIdx.x * 4 + (threadIdx.x >> 6)) * 4;
  if (t0 >= a.T) return;
  const bool exists = t0 + (lane >> 4) < a.T;
  const int64_t t = exists ? t0 + (lane >> 4) : a.T - 1;
  const int E = a.E;
  const float* row = logits + t * E;
  const int idx = c < a.k ? topk[t * a.k + c] : -1;
  float dg = c < a.k ? d_gates[t * a.k + c] * a.scale : 0.0f;
  const LaneMap map{64, 4, 1 << 20, false};
  float p[kSigmoid ? 1 : NPER];
  if constexpr (!kSigmoid) {
    load_row<NPER, 4>(row, E, map, c, p);
    mask_row<NPER, 4>(E, map, c, p);
  }
  const bool on = idx >= 0 && idx < E;
  const float l = row[on ? idx : 0];
  float s, rest = 0.0f, r = 1.0f;
  if constexpr (kSigmoid) {
    const float x = expf(-fabsf(l));
    r = 1.0f / (1.0f + x);
    s = on ? (l >= 0.0f ? r : x * r) : 0.0f;
    rest = l >= 0.0f ? x * r : r;
  } else {
    float mx = -3.402823466e38f, sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NPER; ++i) mx = fmaxf(mx, p[i]);
    mx = max16(mx);
#pragma unroll
    for (int i = 0; i < NPER; ++i) {
      p[i] = expf(p[i] - mx);
      sum += p[i];
    }
    r = 1.0f / fmaxf(sum16(sum), 1e-37f);
    s = on ? expf(l - mx) * r : 0.0f;
  }
  if (!on) dg = 0.0f;
  float ds = dg;
  if (a.renorm) {
    const float S = sum16(s) + 1e-20f, dot = sum16(dg * s);  // over all 16 lanes: not inside the selection
    ds = on ? (dg - dot / S) / S : 0.0f;
  }
  const float val = kSigmoid ? ds * s * rest : ds;
  const float base = kSigmoid ? 0.0f : sum16(ds * s);
  // the selected experts' terms go to their columns through LDS (comparing
  // every column with every id costs NPER k selections a lane: 9.5 us); an id that
  // appears twice is written once, by its first lane, with the sum of all
  const int from = lane & 48;
  float total = 0.0f;
  bool first = on;
  for (int j = 0; j < a.k; ++j) {
    const int e = __shfl(on ? idx : -1, from + j);
    const float x = __shfl(val, from + j);
    total += e == idx ? x : 0.0f;
    first = first && !(e == idx && j < c);
  }
#pragma unroll
  for (int i = 0; i < NPER; i += 4) *reinterpret_cast<f32x4_t*>(mine + mapped<4>(map, c, i)) = f32x4_t{0.f, 0.f, 0.f, 0.f};
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  if (first) mine[idx] = total;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  if (!exists) return;
#pragma unroll
  for (int i = 0; i < NPER; i += 4) {
    const int e = mapped<4>(map, c, i);
    f32x4_t v = *reinterpret_cast<const f32x4_t*>(mine + e) - base;
    if constexpr (!kSigmoid) v *= f32x4_t{p[i], p[i + 1], p[i + 2], p[i + 3]} * r;
    if (e < E) *reinterpret_cast<f32x4_t*>(d_logits + t * E + e) = v;
  }
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

template <int NPER, int V>
void launch_top8(const ScoreArgs& a, const LaneMap& m, const float* logits, const float* bias, int32_t* topk,
                 float* gates, hipStream_t s) {
  const dim3 grid((unsigned)((a.T + 15) / 16));
  const bool by_logit = !bias && a.groups == 1;
  if (a.sigmoid) {
    if (by_logit)
      route_top8_kernel<NPER, V, true, true><<<grid, 256, 0, s>>>(a, m, logits, bias, topk, gates);
    else
      route_top8_kernel<NPER, V, true, false><<<grid, 256, 0, s>>>(a, m, logits, bias, topk, gates);
  } else {
    if (by_logit)
      route_top8_kernel<NPER, V, false, true><<<grid, 256, 0, s>>>(a, m, logits, bias, topk, gates);
    else
      route_top8_kernel<NPER, V, false, false><<<grid, 256, 0, s>>>(a, m, logits, bias, topk, gates);
  }
}

hipError_t launch_route_scored(const ScoreArgs& a, const float* logits, const float* bias, int32_t* topk,
                               float* gates, hipStream_t s) {
  if (a.T <= 0) return hipSuccess;
  const int64_t align = reinterpret_cast<int64_t>(logits) | reinterpret_cast<int64_t>(bias);
  const int per = (a.E + 15) / 16;
  // neighbouring experts in a lane, so that a lane's are of one group
  const bool by_lane = a.groups > 1 && 16 % a.groups == 0 && a.E % 16 == 0;
  if (a.k <= kTop && (a.groups == 1 || by_lane)) {
    const bool by4 = a.E % 4 == 0 && (align & 15) == 0 && (!by_lane || per % 4 == 0);
    LaneMap m = by_lane ? LaneMap{by4 ? 4 : 1, per, per, false} : LaneMap{by4 ? 64 : 16, by4 ? 4 : 1, 1 << 20, false};
#define CALL(N, V)                                           \
  do {                                                       \
    m.full = a.E == 16 * (N);                                \
    launch_top8<N, V>(a, m, logits, bias, topk, gates, s);   \
  } while (0)
    // values per lane: whole loads of 4
    const int need = by4 && !by_lane ? (per + 3) / 4 * 4 : per;
    if (by4) {
      if (need <= 4) CALL(4, 4);
      else if (need <= 8) CALL(8, 4);
      else if (need <= 16) CALL(16, 4);
      else if (need <= 24) CALL(24, 4);
      else if (need <= 32) CALL(32, 4);
      else CALL(64, 4);
    } else {
      if (need <= 8) CALL(8, 1);
      else if (need <= 24) CALL(24, 1);
      else CALL(64, 1);
    }
#undef CALL
    return hipGetLastError();
  }
  const dim3 grid((unsigned)((a.T + 3) / 4));
#define CALL(N) route_scored_kernel<N><<<grid, 256, 0, s>>>(a, logits, bias, topk, gates)
  MOE_BY_EXPERTS(a.E, CALL);
#undef CALL
  return hipGetLastError();
}

hipError_t launch_route_scored_bwd(const ScoreArgs& a, const float* logits, const int32_t* topk,
                                   const float* d_gates, float* d_logits, hipStream_t s) {
  if (a.T <= 0) return hipSuccess;
  const int64_t align = reinterpret_cast<int64_t>(logits) | reinterpret_cast<int64_t>(d_logits);
  if (a.k <= 16 && a.E % 4 == 0 && (align & 15) == 0) {
    const dim3 grid((unsigned)((a.T + 15) / 16));
#define CALL(N)                                                                               \
  do {                                                                                        \
    if (a.sigmoid)                                                                            \
      route_bwd16_kernel<N, true><<<grid, 256, 0, s>>>(a, logits, topk, d_gates, d_logits);   \
    else                                                                                      \
      route_bwd16_kernel<N, false><<<grid, 256, 0, s>>>(a, logits, topk, d_gates, d_logits);  \
  } while (0)
    if (a.E <= 64) CALL(4);
    else if (a.E <= 128) CALL(8);
    else if (a.E <= 256) CALL(16);
    else if (a.E <= 384) CALL(24);
    else if (a.E <= 512) CALL(32);
    else CALL(64);
#undef CALL
    return hipGetLastError();
  }
  const dim3 grid((unsigned)((a.T + 3) / 4));
#define CALL(N) route_scored_bwd_kernel<N><<<grid, 256, 0, s>>>(a, logits, topk, d_gates, d_logits)
  MOE_BY_EXPERTS(a.E, CALL);
#undef CALL
  return hipGetLastError();
}

}  // namespace moe
