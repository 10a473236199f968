// The dropless branch for at most 16 tokens (moe_forward_few): every weight of
// the latent projection, the router, the selected experts, the up-projection
// and the shared experts is read once, straight from memory into matrix
// instructions.
//
// The weights are the first matrix operand (16 rows of one K range a
// wavefront, the wavefronts of a workgroup sharing K) and the tokens the
// second: a token picks an expert once, so 16 tokens are at most 16 rows of any
// expert and one instruction takes them all.  Since the weights' bytes bound
// the time, the matrix instructions have time to spare, and activations between
// two products are not rounded to bf16: they are held as the sum of two bf16
// numbers (16 bits; the router sees three, all of fp32's), each multiplied
// separately.
#include "common.h"
#include "kernels.h"
#include "select.h"
#include "stream.h"

namespace moe {
namespace {

// Wavefronts of a workgroup, which share K (8 instead of 4: 16 tokens 125 us
// instead of 115, 4 tokens of a 6144-wide layer 382 instead of 386).  The
// router's also select, one token each at most.
constexpr int kWaves = 4, kThreads = 64 * kWaves, kRouteWaves = 16;

int64_t cdiv64(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Sum over the wavefronts; complete in wavefront 0, whose lane holds weight
// rows 4 (lane >> 4) .. + 3 of token lane & 15.
template <int W, int kSets>
__device__ __forceinline__ void join(f32x4_t (&acc)[kSets][1], f32x4_t* part) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (wave > 0) {
#pragma unroll
    for (int s = 0; s < kSets; ++s) part[((wave - 1) * kSets + s) * 64 + lane] = acc[s][0];
  }
  __syncthreads();
  if (wave == 0) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
#pragma unroll
      for (int s = 0; s < kSets; ++s) acc[s][0] += part[(j * kSets + s) * 64 + lane];
  }
}

// Values that another workgroup of the same kernel reads.  The 8 XCDs' L2s are
// not coherent with one another inside a kernel, so they are written through to
// memory and read from there (agent scope), a few kilobytes beside the weights.
template <class T>
__device__ __forceinline__ void put(T* p, T v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <class T>
__device__ __forceinline__ T get(const T* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ f32x4_t get4(const float* p) {
  const uint64_t* q = reinterpret_cast<const uint64_t*>(p);
  const uint64_t a = get(q), b = get(q + 1);
  return f32x4_t{__uint_as_float((uint32_t)a), __uint_as_float((uint32_t)(a >> 32)), __uint_as_float((uint32_t)b),
                 __uint_as_float((uint32_t)(b >> 32))};
}
__device__ __forceinline__ void put4(float* p, f32x4_t v) {
  uint64_t* q = reinterpret_cast<uint64_t*>(p);
  put(q, (uint64_t)__float_as_uint(v[0]) | (uint64_t)__float_as_uint(v[1]) << 32);
  put(q + 1, (uint64_t)__float_as_uint(v[2]) | (uint64_t)__float_as_uint(v[3]) << 32);
}

// kSets matrices by tokens held in kPlanes bf16 parts, over K values.
template <int W, int kSets, int kPlanes>
__device__ __forceinline__ void product(const uint16_t* const (&w)[kSets], const uint16_t* const (&x)[kPlanes], int K,
                                        f32x4_t (&acc)[kSets][1]) {
  stream<W, kSets, kPlanes, true, 4>(w, x, K / 64, acc, [](const uint16_t* p) { return ld16(p); });
}

// 4 neighbouring values as kPlanes bf16 parts, planes `plane` values apart.
template <int kPlanes>
__device__ __forceinline__ void store_parts(uint16_t* p, int64_t plane, f32x4_t v) {
#pragma unroll
  for (int i = 0; i < kPlanes; ++i) {
    const uint2 q = make_uint2(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]));
    *reinterpret_cast<uint2*>(p + i * plane) = q;
    v -= f32x4_t{__uint_as_float(q.x << 16), __uint_as_float(q.x & 0xFFFF0000u), __uint_as_float(q.y << 16),
                 __uint_as_float(q.y & 0xFFFF0000u)};
  }
}

__device__ __forceinline__ f32x4_t zero4() { return f32x4_t{0.f, 0.f, 0.f, 0.f}; }

// z = x W_lat^T: 16 columns.
__device__ __forceinline__ void latent_item(const Few& f, int item, f32x4_t* part) {
  const int lane = threadIdx.x & 63, at = (lane >> 4) * 8, t = min(lane & 15, f.T - 1);
  const uint16_t* w[1] = {f.w_latent + (int64_t)(item * 16 + (lane & 15)) * f.D + at};
  const uint16_t* x[1] = {f.x + (int64_t)t * f.D + at};
  f32x4_t acc[1][1] = {{zero4()}};
  product<kWaves, 1, 1>(w, x, f.D, acc);
  join<kWaves, 1>(acc, part);
  if (threadIdx.x < 64 && (lane & 15) < f.T)
    store_parts<3>(f.z + (int64_t)t * f.L + item * 16 + (lane >> 4) * 4, (int64_t)f.T * f.L, acc[0][0]);
}

// Hidden values of the shared experts, side by side: 16 of them.
__device__ __forceinline__ void shared_item(const Few& f, int item, f32x4_t* part) {
  const int lane = threadIdx.x & 63, at = (lane >> 4) * 8, t = min(lane & 15, f.T - 1);
  const int64_t row = (int64_t)(item * 16 + (lane & 15)) * f.D + at;
  const uint16_t* w[2] = {f.ws_gate + row, f.ws_up + row};
  const uint16_t* x[1] = {f.x + (int64_t)t * f.D + at};
  f32x4_t acc[2][1] = {{zero4()}, {zero4()}};
  product<kWaves, 2, 1>(w, x, f.D, acc);
  join<kWaves, 2>(acc, part);
  if (threadIdx.x < 64 && (lane & 15) < f.T) {
    f32x4_t h;
#pragma unroll
    for (int r = 0; r < 4; ++r) h[r] = silu(acc[0][0][r]) * acc[1][0][r];
    const int W = f.S * f.Fs;
    store_parts<2>(f.hs + (int64_t)t * W + item * 16 + (lane >> 4) * 4, (int64_t)f.T * W, h);
  }
}

// Router logits of 16 experts.
__device__ __forceinline__ void router_item(const Few& f, int item, f32x4_t* part) {
  const int lane = threadIdx.x & 63, at = (lane >> 4) * 8, t = min(lane & 15, f.T - 1);
  const uint16_t* w[1] = {f.w_router + (int64_t)min(item * 16 + (lane & 15), f.E - 1) * f.L + at};
  const uint16_t* z = f.z + (int64_t)t * f.L + at;
  const int64_t plane = (int64_t)f.T * f.L;
  const uint16_t* x[3] = {z, z + plane, z + 2 * plane};
  f32x4_t acc[1][1] = {{zero4()}};
  product<kRouteWaves, 1, 3>(w, x, f.L, acc);
  join<kRouteWaves, 1>(acc, part);
  if (threadIdx.x < 64 && (lane & 15) < f.T) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int e = item * 16 + (lane >> 4) * 4 + r;
      if (e < f.E) put(&f.logits[(int64_t)t * f.E + e], acc[0][0][r]);
    }
  }
}

// 16 hidden values of the n rows of the a-th selected expert, e.
__device__ __forceinline__ void hidden_item(const Few& f, int a, int e, int n, int item, f32x4_t* part) {
  const int lane = threadIdx.x & 63, at = (lane >> 4) * 8;
  const int r = f.rows[a * 16 + (lane & 15)];  // t k + j
  const int64_t row = ((int64_t)e * f.F + item * 16 + (lane & 15)) * f.L + at;
  const uint16_t* w[2] = {f.w_gate + row, f.w_up + row};
  const uint16_t* z = f.z + (int64_t)(r / f.k) * f.L + at;
  const uint16_t* x[2] = {z, z + (int64_t)f.T * f.L};
  f32x4_t acc[2][1] = {{zero4()}, {zero4()}};
  product<kWaves, 2, 2>(w, x, f.L, acc);
  join<kWaves, 2>(acc, part);
  if (threadIdx.x < 64 && (lane & 15) < n) {
    f32x4_t h;
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = silu(acc[0][0][i]) * acc[1][0][i];
    store_parts<2>(f.h + (int64_t)r * f.F + item * 16 + (lane >> 4) * 4, (int64_t)f.T * f.k * f.F, h);
  }
}

// 16 kC columns of its outputs.
template <int kC>
__device__ __forceinline__ void down_item(const Few& f, int a, int e, int n, int item, f32x4_t* part) {
  const int lane = threadIdx.x & 63, at = (lane >> 4) * 8;
  const int r = f.rows[a * 16 + (lane & 15)];
  const uint16_t* w[kC];
  f32x4_t acc[kC][1];
#pragma unroll
  for (int c = 0; c < kC; ++c) {
    w[c] = f.w_down + ((int64_t)e * f.L + (item * kC + c) * 16 + (lane & 15)) * f.F + at;
    acc[c][0] = zero4();
  }
  const uint16_t* h = f.h + (int64_t)r * f.F + at;
  const uint16_t* x[2] = {h, h + (int64_t)f.T * f.k * f.F};
  product<kWaves, kC, 2>(w, x, f.F, acc);
  join<kWaves, kC>(acc, part);
  if (threadIdx.x < 64 && (lane & 15) < n) {
#pragma unroll
    for (int c = 0; c < kC; ++c)
      put4(f.o + (int64_t)r * f.L + (item * kC + c) * 16 + (lane >> 4) * 4, acc[c][0]);
  }
}

// y_lat = sum over a token's experts, in order: 4 columns a thread.
__device__ __forceinline__ void combine_at(const Few& f, int t, int col) {
  f32x4_t s = zero4();
  for (int j = 0; j < f.k; ++j)
    s += f.gates[t * f.k + j] * get4(f.o + (int64_t)(t * f.k + j) * f.L + col);
  store_parts<2>(f.ylat + (int64_t)t * f.L + col, (int64_t)f.T * f.L, s);
}

// 16 columns of the shared experts' part of y, in fp32.
__device__ __forceinline__ void shared_out_item(const Few& f, int item, f32x4_t* part) {
  const int lane = threadIdx.x & 63, at = (lane >> 4) * 8, t = min(lane & 15, f.T - 1);
  const int64_t n = item * 16 + (lane & 15);
  const int W = f.S * f.Fs;
  f32x4_t acc[1][1] = {{zero4()}};
  for (int s = 0; s < f.S; ++s) {
    const uint16_t* w[1] = {f.ws_down + ((int64_t)s * f.D + n) * f.Fs + at};
    const uint16_t* h = f.hs + (int64_t)t * W + s * f.Fs + at;
    const uint16_t* x[2] = {h, h + (int64_t)f.T * W};
    product<kRouteWaves, 1, 2>(w, x, f.Fs, acc);
  }
  join<kRouteWaves, 1>(acc, part);
  if (threadIdx.x < 64 && (lane & 15) < f.T)
    *reinterpret_cast<f32x4_t*>(f.ypart + (int64_t)t * f.D + item * 16 + (lane >> 4) * 4) = acc[0][0];
}

// 16 columns of y: the up-projection, the shared experts' part and the residual.
__device__ __forceinline__ void output_item(const Few& f, int item, f32x4_t* part) {
  const int lane = threadIdx.x & 63, at = (lane >> 4) * 8, t = min(lane & 15, f.T - 1);
  const int64_t o = (int64_t)t * f.D + item * 16 + (lane >> 4) * 4;
  f32x4_t add = zero4();
  if (threadIdx.x < 64) {
    if (f.S > 0) add = *reinterpret_cast<const f32x4_t*>(f.ypart + o);
    if (f.res) {
      const uint2 r = *reinterpret_cast<const uint2*>(f.res + o);
      add += f32x4_t{__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xFFFF0000u), __uint_as_float(r.y << 16),
                     __uint_as_float(r.y & 0xFFFF0000u)};
    }
  }
  f32x4_t acc[1][1] = {{zero4()}};
  const uint16_t* w[1] = {f.w_up_proj + (int64_t)(item * 16 + (lane & 15)) * f.L + at};
  const uint16_t* y = f.ylat + (int64_t)t * f.L + at;
  const uint16_t* x[2] = {y, y + (int64_t)f.T * f.L};
  product<kWaves, 1, 2>(w, x, f.L, acc);
  join<kWaves, 1>(acc, part);
  if (threadIdx.x < 64 && (lane & 15) < f.T) {
    const f32x4_t v = acc[0][0] + add;
    *reinterpret_cast<uint2*>(f.y + o) = make_uint2(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]));
  }
}

// Selection for every token, then the selected experts in ascending order,
// each with its rows t k + j in token order.  One workgroup.
struct RouteLds {
  uint32_t mask[1024];  // of an expert: the tokens that take it (T <= 16), then its rank above them
  uint16_t ids[1024];   // [T][k], T k <= 1024
  int scan[kRouteWaves];
  int total;            // selected experts
};
constexpr int kRouteThreads = 64 * kRouteWaves;
__device__ void route_all(const Few& f, RouteLds& s) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  for (int e = threadIdx.x; e < f.E; e += kRouteThreads) s.mask[e] = 0;
  __syncthreads();
  for (int t = wave; t < f.T; t += kRouteWaves) {
    int mine;
    float g;
    const float* row = f.logits + (int64_t)t * f.E;
    select_topk([&](int e) { return get(row + e); }, f.bias, f.E, f.k, mine, g);
    if (lane < f.k) {
      f.topk[t * f.k + lane] = mine;
      f.gates[t * f.k + lane] = g;
      s.ids[t * f.k + lane] = (uint16_t)mine;
      atomicOr(&s.mask[mine], 1u << t);
    }
  }
  __syncthreads();
  // rank of every selected expert among the selected: an expert a thread
  const int e = threadIdx.x;
  const int n = e < f.E && s.mask[e] != 0;
  int x = n;
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(x, d);
    if (lane >= d) x += o;
  }
  if (lane == 63) s.scan[wave] = x;
  __syncthreads();
  const int a = x - n + [&] {
    int before = 0;
    for (int w = 0; w < wave; ++w) before += s.scan[w];
    return before;
  }();
  if (threadIdx.x == kRouteThreads - 1) {
    *f.n_act = a + n;
    s.total = a + n;
  }
  if (n) {
    f.act[a] = e | __popc(s.mask[e]) << 16;
    s.mask[e] |= (uint32_t)a << 16;
  }
  __syncthreads();
  // the rest of act is empty; an expert's rows are repeated up to 16
  for (int i = s.total + threadIdx.x; i < f.most; i += kRouteThreads) f.act[i] = -1;
  for (int i = threadIdx.x; i < f.T * f.k; i += kRouteThreads) {
    const int t = i / f.k;
    const uint32_t m = s.mask[s.ids[i]], taken = m & 0xFFFFu;
    const int n = __popc(taken);
    for (int r = __popc(taken & ((1u << t) - 1u)); r < 16; r += n) f.rows[(m >> 16) * 16 + r] = i;
  }
}
static_assert(kRouteThreads >= 1024, "the scan covers every expert");

// ------------------------------------------------------------- launches
// Five kernels, each waiting for the whole of the one before:
//   1  z and the shared experts' hidden values (what needs x alone)
//   2  the router; its last workgroup to finish selects for all tokens; meanwhile
//      the shared experts' part of y
//   3  the selected experts' hidden rows
//   4  their outputs; a column block's last workgroup to finish sums them to y_lat
//   5  y
// A step by the last of some workgroups costs two trips to memory, less than a
// launch; a wait of all workgroups for all others costs more than one: with 2 to
// 5 as one kernel of workgroups that take items by tickets and wait on
// counters, a token of a small layer took 90 us instead of 26 and 4 tokens of a
// 6144-wide one 800 instead of 385, most of it the tickets' atomics (device-wide
// ones on one address take about 37 ns each, one after the other).
constexpr int part_size(int waves, int sets) { return (waves - 1) * sets * 64; }

// The workgroup's results have reached memory, then *p is raised: whether all
// n have.
__device__ __forceinline__ bool last_of(int* p, int n) {
  __shared__ int before;
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
  wait_vm_all();
  __syncthreads();
  if (threadIdx.x == 0) before = __hip_atomic_fetch_add(p, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  return before == n - 1;
}

__global__ __launch_bounds__(kThreads) void few_first_kernel(Few f) {
  __shared__ f32x4_t part[part_size(kWaves, 2)];
  // counters of the later kernels: one for the router, one for each 16 (or 32) columns of y_lat
  const int i = blockIdx.x * kThreads + threadIdx.x;
  if (i < 1 + f.L / 16) f.counters[i] = 0;
  const int n = f.L / 16;
  if ((int)blockIdx.x < n)
    latent_item(f, blockIdx.x, part);
  else
    shared_item(f, blockIdx.x - n, part);
}
__global__ __launch_bounds__(kRouteThreads) void few_route_kernel(Few f) {
  __shared__ f32x4_t part[part_size(kRouteWaves, 1)];
  __shared__ RouteLds route;
  const int n = (f.E + 15) / 16;
  if ((int)blockIdx.x < n) {
    router_item(f, blockIdx.x, part);
    if (last_of(f.counters, n)) route_all(f, route);
  } else {
    shared_out_item(f, blockIdx.x - n, part);
  }
}
__global__ __launch_bounds__(kThreads) void few_hidden_kernel(Few f) {
  __shared__ f32x4_t part[part_size(kWaves, 2)];
  const int en = f.act[blockIdx.y];
  if (en >= 0) hidden_item(f, blockIdx.y, en & 0xFFFF, en >> 16, blockIdx.x, part);
}
template <int kC>
__global__ __launch_bounds__(kThreads) void few_down_kernel(Few f) {
  __shared__ f32x4_t part[part_size(kWaves, kC)];
  const int en = f.act[blockIdx.y], n_act = *f.n_act, item = blockIdx.x;
  if (en < 0) return;
  down_item<kC>(f, blockIdx.y, en & 0xFFFF, en >> 16, item, part);
  if (last_of(&f.counters[1 + item], n_act))
    for (int i = threadIdx.x; i < f.T * 4 * kC; i += kThreads)
      combine_at(f, i / (4 * kC), (item * 4 * kC + i % (4 * kC)) * 4);
}
__global__ __launch_bounds__(kThreads) void few_output_kernel(Few f) {
  __shared__ f32x4_t part[part_size(kWaves, 1)];
  output_item(f, blockIdx.x, part);
}

}  // namespace

int few_counter_ints(int L) { return 1 + L / 16; }

hipError_t launch_few(const Few& f, hipStream_t s) {
  if (f.T <= 0) return hipSuccess;
  few_first_kernel<<<(unsigned)(f.L / 16 + f.S * f.Fs / 16), kThreads, 0, s>>>(f);
  few_route_kernel<<<(unsigned)(cdiv64(f.E, 16) + (f.S > 0 ? f.D / 16 : 0)), kRouteThreads, 0, s>>>(f);
  few_hidden_kernel<<<dim3(f.F / 16, f.most), kThreads, 0, s>>>(f);
  // 32 columns a workgroup where that leaves two for every CU: the hidden rows, in
  // two parts and for any number of rows as much as 32 rows of weights, are read
  // half as often (16 tokens by 960 columns, 60 experts 108 us, 115 with 16
  // columns; 64 columns: the same, and 267 instead of 258 where 16 tokens pick
  // from 128 experts.  The hidden kernel with 32 values a workgroup: 262).
  if ((int64_t)f.L / 32 * f.most >= 512)  // L is a multiple of 64
    few_down_kernel<2><<<dim3(f.L / 32, f.most), kThreads, 0, s>>>(f);
  else
    few_down_kernel<1><<<dim3(f.L / 16, f.most), kThreads, 0, s>>>(f);
  few_output_kernel<<<(unsigned)(f.D / 16), kThreads, 0, s>>>(f);
  return hipGetLastError();
}

}  // namespace moe
