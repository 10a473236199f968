// Quantiser to e4m3 with one fp32 scale for 1 x 128 or 128 x 128 blocks of
// the (possibly transposed) source:  s = max|x| / 448, q = e4m3(448 x / max|x|).
//
// Bound by memory: each source value is read once (2 or 4 bytes), each result
// written once (1 byte).  A thread takes 16 consecutive values of a row (32
// or 64 bytes of loads, one 16-byte store), so 8 lanes hold a 1 x 128 block
// and its maximum is three lane exchanges; several blocks per thread keep
// that many loads in flight before the first is used.
#include <type_traits>

#include "kernels.h"
#include "quant.h"

namespace moe {
namespace {

constexpr int kRun = 16;             // values per thread and block
constexpr int kLanes = kQB / kRun;   // lanes per row of a block
constexpr int kGroups = 256 / kLanes;  // rows a workgroup takes at once

// 16 values of the source, as loaded.
template <typename T>
struct Run {
  static constexpr int kChunks = kRun * (int)sizeof(T) / 16;
  uint4 v[kChunks];

  // inside: 16-byte aligned and every value exists
  __device__ __forceinline__ void load(const char* p) {
#pragma unroll
    for (int i = 0; i < kChunks; ++i) v[i] = ld16_stream(p + i * 16);
  }
  // n values exist (0 .. 16, any alignment of T); the rest are zeros
  __device__ __forceinline__ void load_edge(const char* p, int n) {
    uint32_t w[kChunks * 4] = {};
#pragma unroll
    for (int i = 0; i < kRun; ++i)
      if (i < n) {
        if constexpr (sizeof(T) == 4)
          w[i] = reinterpret_cast<const uint32_t*>(p)[i];
        else
          w[i / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[i] << (16 * (i & 1));
      }
#pragma unroll
    for (int i = 0; i < kChunks; ++i) v[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  }
  __device__ __forceinline__ void values(float* f) const {
#pragma unroll
    for (int i = 0; i < kChunks; ++i) unpack(v[i], f + i * Chunk<T>::kElems, T{});
  }
  __device__ __forceinline__ float amax() const {
    float f[kRun], m = 0.0f;
    values(f);
#pragma unroll
    for (int i = 0; i < kRun; ++i) m = fmaxf(m, fabsf(f[i]));
    return m;
  }
};

// Source geometry of one launch.
struct Source {
  const char* x;
  int64_t rows, cols, ld;  // elements
  bool aligned;            // base and rows 16-byte aligned
};

// Largest over the 8 lanes of a block's row (lanes 8 g .. 8 g + 7).
__device__ __forceinline__ float max8(float m) {
  m = fmaxf(m, __shfl_xor(m, 1));
  m = fmaxf(m, __shfl_xor(m, 2));
  return fmaxf(m, __shfl_xor(m, 4));
}

__device__ __forceinline__ uint4 quantize16(const float* f, const BlockQuant& bq) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = e4m3_quad(bq(f[4 * i]), bq(f[4 * i + 1]), bq(f[4 * i + 2]), bq(f[4 * i + 3]));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// 1 x 128 blocks, not transposed: 32 rows x NB blocks per workgroup.  The
// scales ([K block][row]) meet in LDS, so that 32 rows of a block are written
// together.
template <typename T, int NB>
__global__ __launch_bounds__(256) void quantize_rows_kernel(Source s, char* __restrict__ q, int64_t ldq,
                                                            float* __restrict__ scale, int64_t scale_ld, int tiles_k) {
  __shared__ float sc[NB][kGroups + 1];
  const int tr = blockIdx.x / tiles_k, tk = blockIdx.x - tr * tiles_k;
  const int g = threadIdx.x / kLanes, c = threadIdx.x % kLanes;
  const int64_t r0 = (int64_t)tr * kGroups, k0 = (int64_t)tk * (NB * kQB);
  const int64_t row = r0 + g, col = k0 + c * kRun;
  const char* p = s.x + (row * s.ld + col) * (int64_t)sizeof(T);
  Run<T> v[NB];
  if (s.aligned && r0 + kGroups <= s.rows && k0 + NB * kQB <= s.cols) {
#pragma unroll
    for (int i = 0; i < NB; ++i) v[i].load(p + i * (kQB * (int)sizeof(T)));
  } else {
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int64_t left = row < s.rows ? s.cols - (col + i * kQB) : 0;
      v[i].load_edge(p + i * (kQB * (int)sizeof(T)), (int)max(min(left, (int64_t)kRun), (int64_t)0));
    }
  }
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const float amax = fmaxf(max8(v[i].amax()), kQuantTiny);
    const BlockQuant bq(amax);
    float f[kRun];
    v[i].values(f);
    const uint4 w = quantize16(f, bq);
    if (row < s.rows && k0 + i * kQB < s.cols) st16(q + row * ldq + col + i * kQB, w);
    if (c == 0) sc[i][g] = block_scale(amax);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < NB * kGroups; i += 256) {
    const int b = i / kGroups, r = i % kGroups;
    if (r0 + r < s.rows && k0 + b * kQB < s.cols) scale[(k0 / kQB + b) * scale_ld + r0 + r] = sc[b][r];
  }
}

// 128 x 128 tile per workgroup: square blocks, and every transposed result.
// A thread holds 16 columns of 4 neighbouring rows; a transposed tile passes
// through LDS as bytes, four rows of a column in one 32-bit word.
constexpr int kTLd = kQB / 4 + 1;  // words per transposed row: odd, so that columns spread over the banks

template <typename T, bool kSquare, bool kTranspose>
__global__ __launch_bounds__(256) void quantize_tile_kernel(Source s, char* __restrict__ q, int64_t ldq,
                                                            float* __restrict__ scale, int64_t scale_ld, int tiles_k) {
  static_assert(kSquare || kTranspose, "1 x 128 blocks that are not transposed have a kernel of their own");
  __shared__ uint32_t tile[kTranspose ? kQB * kTLd : 1];
  __shared__ float part[4][kSquare ? 1 : kQB];
  const int tr = blockIdx.x / tiles_k, tk = blockIdx.x - tr * tiles_k;
  const int g = threadIdx.x / kLanes, c = threadIdx.x % kLanes, wave = threadIdx.x >> 6;
  const int64_t r0 = (int64_t)tr * kQB, k0 = (int64_t)tk * kQB;
  const int64_t col = k0 + c * kRun;
  const char* p = s.x + ((r0 + g * 4) * s.ld + col) * (int64_t)sizeof(T);
  Run<T> v[4];
  if (s.aligned && r0 + kQB <= s.rows && k0 + kQB <= s.cols) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i].load(p + i * s.ld * (int64_t)sizeof(T));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t left = r0 + g * 4 + i < s.rows ? s.cols - col : 0;
      v[i].load_edge(p + i * s.ld * (int64_t)sizeof(T), (int)max(min(left, (int64_t)kRun), (int64_t)0));
    }
  }
  uint4 w[4];  // bytes of row i
  if constexpr (kSquare) {
    float m = fmaxf(fmaxf(v[0].amax(), v[1].amax()), fmaxf(v[2].amax(), v[3].amax()));
    for (int d = 1; d < 64; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
    if ((threadIdx.x & 63) == 0) part[wave][0] = m;
    __syncthreads();
    m = fmaxf(fmaxf(fmaxf(part[0][0], part[1][0]), fmaxf(part[2][0], part[3][0])), kQuantTiny);
    const BlockQuant bq(m);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float f[kRun];
      v[i].values(f);
      w[i] = quantize16(f, bq);
    }
    if (threadIdx.x == 0) scale[kTranspose ? (k0 / kQB) * scale_ld + r0 / kQB : (r0 / kQB) * scale_ld + k0 / kQB] = block_scale(m);
  } else {
    // a block is a column of the tile: its largest over the thread's rows,
    // the wavefront's 8 row groups, then the 4 wavefronts
    float m[kRun];
#pragma unroll
    for (int j = 0; j < kRun; ++j) m[j] = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float f[kRun];
      v[i].values(f);
#pragma unroll
      for (int j = 0; j < kRun; ++j) m[j] = fmaxf(m[j], fabsf(f[j]));
    }
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
      for (int d = kLanes; d < 64; d <<= 1) m[j] = fmaxf(m[j], __shfl_xor(m[j], d));
      if ((threadIdx.x & 63) < kLanes) part[wave][c * kRun + j] = m[j];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
      const int n = c * kRun + j;
      const float amax = fmaxf(fmaxf(fmaxf(part[0][n], part[1][n]), fmaxf(part[2][n], part[3][n])), kQuantTiny);
      const BlockQuant bq(amax);
      float x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float f[kRun];
        v[i].values(f);
        x[i] = bq(f[j]);
      }
      tile[n * kTLd + g] = e4m3_quad(x[0], x[1], x[2], x[3]);
      if (g == 0 && k0 + n < s.cols) scale[(r0 / kQB) * scale_ld + k0 + n] = block_scale(amax);
    }
  }
  if constexpr (!kTranspose) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (r0 + g * 4 + i < s.rows) st16(q + (r0 + g * 4 + i) * ldq + col, w[i]);
    return;
  }
  if constexpr (kSquare) {
    // 4 x 4 byte transposes: word j of the four rows -> columns 4 j .. 4 j + 3
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t a[4] = {j == 0 ? w[0].x : j == 1 ? w[0].y : j == 2 ? w[0].z : w[0].w,
                             j == 0 ? w[1].x : j == 1 ? w[1].y : j == 2 ? w[1].z : w[1].w,
                             j == 0 ? w[2].x : j == 1 ? w[2].y : j == 2 ? w[2].z : w[2].w,
                             j == 0 ? w[3].x : j == 1 ? w[3].y : j == 2 ? w[3].z : w[3].w};
#pragma unroll
      for (int n = 0; n < 4; ++n)
        tile[(c * kRun + j * 4 + n) * kTLd + g] = ((a[0] >> (8 * n)) & 0xFF) | (((a[1] >> (8 * n)) & 0xFF) << 8) |
                                                  (((a[2] >> (8 * n)) & 0xFF) << 16) | ((a[3] >> (8 * n)) << 24);
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = g + i * kGroups;
    if (k0 + n < s.cols) {
      const uint32_t* t = tile + n * kTLd + c * 4;
      st16(q + (k0 + n) * ldq + r0 + c * kRun, make_uint4(t[0], t[1], t[2], t[3]));
    }
  }
}

template <typename T>
hipError_t launch_typed(const QuantizeArgs& a, hipStream_t st) {
  Source s{static_cast<const char*>(a.x), a.rows, a.cols, a.ld, false};
  s.aligned = (reinterpret_cast<uintptr_t>(a.x) & 15) == 0 && (a.ld * (int64_t)sizeof(T)) % 16 == 0;
  const int64_t tk = (a.cols + kQB - 1) / kQB;
  if (a.block_rows == 1 && !a.transpose) {
    // blocks per thread: as many as leave every CU a few workgroups; 64
    // registers of loads at the most
    constexpr int kMost = sizeof(T) == 2 ? 8 : 4;
    const int64_t tr = (a.rows + kGroups - 1) / kGroups;
    auto go = [&](auto nb) {
      constexpr int NB = decltype(nb)::value;
      const int64_t t = (tk + NB - 1) / NB;
      quantize_rows_kernel<T, NB><<<dim3((unsigned)(tr * t)), 256, 0, st>>>(s, a.q, a.ldq, a.scale, a.scale_ld, (int)t);
    };
    if (tr * tk >= 1024 * kMost && tk >= kMost)
      go(std::integral_constant<int, kMost>{});
    else if (tr * tk >= 1024)
      go(std::integral_constant<int, 2>{});
    else
      go(std::integral_constant<int, 1>{});
    return hipGetLastError();
  }
  const dim3 grid((unsigned)((a.rows + kQB - 1) / kQB * tk));
  if (a.block_rows == 1)
    quantize_tile_kernel<T, false, true><<<grid, 256, 0, st>>>(s, a.q, a.ldq, a.scale, a.scale_ld, (int)tk);
  else if (a.transpose)
    quantize_tile_kernel<T, true, true><<<grid, 256, 0, st>>>(s, a.q, a.ldq, a.scale, a.scale_ld, (int)tk);
  else
    quantize_tile_kernel<T, true, false><<<grid, 256, 0, st>>>(s, a.q, a.ldq, a.scale, a.scale_ld, (int)tk);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize(const QuantizeArgs& a, hipStream_t s) {
  if (a.rows <= 0 || a.cols <= 0) return hipSuccess;
  return a.dt == DT_F32 ? launch_typed<float>(a, s) : launch_typed<bf16_t>(a, s);
}

}  // namespace moe
