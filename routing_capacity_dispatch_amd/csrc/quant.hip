// Quantiser to e4m3 with one fp32 scale for 1 x 128 or 128 x 128 blocks of
// the (possibly transposed) source:  s = max|x| / 448, q = e4m3(448 x / max|x|).
//
// Bound by memory: each source value is read once (2 or 4 bytes), each result
// written once (1 byte).  A thread takes 16 consecutive values of a row (32
// or 64 bytes of loads, one 16-byte store), so 8 lanes hold a 1 x 128 block
// and its maximum is three lane exchanges; several blocks per thread keep
// that many loads in flight before the first is used.
// Measured: 16384 x 6144 in 1 x 128 blocks, plain and transposed, bf16 50 and 53
// us (6.1 TB/s), fp32 92 and 107; in 128 x 128 blocks 48 and 53, 95 and 106; 2056
// x 4100 fp32, transposed, 128 x 128 10.1 us (4.2 TB/s: two workgroups a CU, so
// the first loads' latency shows).
#include <type_traits>

#include "kernels.h"
#include "quant.h"

namespace moe {
namespace {

constexpr int kRun = 16;             // values per thread and block
constexpr int kLanes = kQB / kRun;   // lanes per row of a block
constexpr int kGroups = 256 / kLanes;  // rows a workgroup takes at once

// 16 bytes at an address that is a multiple of kAlign (2 or 4).  No
// nontemporal hint, though each byte is read once: neighbouring loads share
// lines, and with the hint each fetches its own (8192 x 4096 fp32: 42 us with
// it, 26 without).
typedef u32x4_t u32x4_by2_t __attribute__((aligned(2)));
typedef u32x4_t u32x4_by4_t __attribute__((aligned(4)));
template <int kAlign>
__device__ __forceinline__ uint4 ld16_any(const char* p) {
  using any_t = std::conditional_t<kAlign == 2, u32x4_by2_t, u32x4_by4_t>;
  const u32x4_t v = *reinterpret_cast<const any_t*>(p);
  return make_uint4(v.x, v.y, v.z, v.w);
}

// 16 values of the source, as loaded: 16-byte loads whatever the rows'
// alignment (global memory takes any; a row that starts off a 16-byte
// boundary costs little beside loads of single values).
template <typename T>
struct Run {
  static constexpr int kChunks = kRun * (int)sizeof(T) / 16;
  uint4 v[kChunks];

  __device__ __forceinline__ void load(const char* p) {
#pragma unroll
    for (int i = 0; i < kChunks; ++i) v[i] = ld16_any<(int)sizeof(T)>(p + i * 16);
  }
  // n values exist (0 .. 16); the rest are zeros.  The 16 bytes are loaded
  // whole wherever they lie inside [any, end), the source's first byte and
  // end (past a row's last value lie the next row's, which are cleared): only
  // the source's last bytes are loaded one by one, and none of those loads
  // stands behind a branch of its own (past the end the last value again, or
  // where there is none, the source's first).
  __device__ __forceinline__ void load_edge(const char* p, int n, const char* any, const char* end_) {
    const char* w = n > 0 ? p : any;
    if (w + kRun * (int)sizeof(T) <= end_) {
      load(w);
      constexpr int kPer = 4 / (int)sizeof(T);  // values per word
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int first = (4 * i + j) * kPer;
          x[j] = n >= first + kPer ? x[j] : n <= first ? 0u : x[j] & 0xFFFFu;
        }
        v[i] = make_uint4(x[0], x[1], x[2], x[3]);
      }
      return;
    }
    const char* q = n > 0 ? p : any;
    const int end = n > 0 ? n - 1 : 0;
    uint32_t x[kRun];
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      if constexpr (sizeof(T) == 4)
        x[i] = reinterpret_cast<const uint32_t*>(q)[min(i, end)];
      else
        x[i] = reinterpret_cast<const uint16_t*>(q)[min(i, end)];
    }
#pragma unroll
    for (int i = 0; i < kRun; ++i) x[i] = i < n ? x[i] : 0u;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < kChunks; ++i) v[i] = make_uint4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < kChunks; ++i)
        v[i] = make_uint4(x[8 * i] | x[8 * i + 1] << 16, x[8 * i + 2] | x[8 * i + 3] << 16,
                          x[8 * i + 4] | x[8 * i + 5] << 16, x[8 * i + 6] | x[8 * i + 7] << 16);
    }
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
  const char* end;         // behind the last value
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
  if (r0 + kGroups <= s.rows && k0 + NB * kQB <= s.cols) {
#pragma unroll
    for (int i = 0; i < NB; ++i) v[i].load(p + i * (kQB * (int)sizeof(T)));
  } else {
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int64_t left = row < s.rows ? s.cols - (col + i * kQB) : 0;
      v[i].load_edge(p + i * (kQB * (int)sizeof(T)), (int)max(min(left, (int64_t)kRun), (int64_t)0), s.x, s.end);
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

// Rows in 1 x 128 blocks, each copied to the rows row_of names (at most 64; a
// negative one names none): dispatched rows are quantised once and moved as
// bytes, where copying them first would move twice as many and quantise each
// copy (the Marin-shaped layer, 131072 dispatched rows: 410 us as scatter and
// quantiser, 114 so: 0.5 GB).  One wavefront per row, 8 blocks a pass.
__global__ __launch_bounds__(256) void quantize_scatter_kernel(const char* __restrict__ x, int64_t T, int cols,
                                                               const int32_t* __restrict__ row_of, int k,
                                                               char* __restrict__ q, float* __restrict__ scale,
                                                               int64_t scale_ld) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= T) return;
  const int to = lane < k ? row_of[t * k + lane] : -1;
  const char* row = x + t * cols * 2;
  for (int col = lane * kRun; col < cols; col += 64 * kRun) {  // cols: a multiple of 128, so 8 lanes stay together
    Run<bf16_t> v;
    v.load(row + col * 2);
    const float amax = fmaxf(max8(v.amax()), kQuantTiny);
    const BlockQuant bq(amax);
    float f[kRun];
    v.values(f);
    const uint4 w = quantize16(f, bq);
    const float s = block_scale(amax);
    for (int j = 0; j < k; ++j) {
      const int64_t r = __builtin_amdgcn_readlane(to, j);
      if (r < 0) continue;
      st16(q + r * cols + col, w);
      if (lane % kLanes == 0) scale[(col / kQB) * scale_ld + r] = s;
    }
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
  // kSquare: maxima of the wavefronts; else column maxima of the 16 groups of
  // 8 rows, then (row 0) of the tile
  __shared__ __attribute__((aligned(16))) float part[kSquare ? 4 : 16][kSquare ? 1 : kQB];
  const int tr = blockIdx.x / tiles_k, tk = blockIdx.x - tr * tiles_k;
  const int g = threadIdx.x / kLanes, c = threadIdx.x % kLanes, wave = threadIdx.x >> 6;
  const int64_t r0 = (int64_t)tr * kQB, k0 = (int64_t)tk * kQB;
  const int64_t col = k0 + c * kRun;
  const char* p = s.x + ((r0 + g * 4) * s.ld + col) * (int64_t)sizeof(T);
  Run<T> v[4];
  if (r0 + kQB <= s.rows && k0 + kQB <= s.cols) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i].load(p + i * s.ld * (int64_t)sizeof(T));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t left = r0 + g * 4 + i < s.rows ? s.cols - col : 0;
      v[i].load_edge(p + i * s.ld * (int64_t)sizeof(T), (int)max(min(left, (int64_t)kRun), (int64_t)0), s.x, s.end);
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
    // its neighbour 8 lanes on, then over LDS
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
    for (int j = 0; j < kRun; ++j)  // rotation by 8 within 16 lanes
      m[j] = fmaxf(m[j], __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(m[j]), 0x128, 0xF, 0xF, false)));
    if ((threadIdx.x & 15) < kLanes) {
      f32x4_t* to = reinterpret_cast<f32x4_t*>(&part[threadIdx.x >> 4][c * kRun]);
#pragma unroll
      for (int j = 0; j < 4; ++j) to[j] = f32x4_t{m[4 * j], m[4 * j + 1], m[4 * j + 2], m[4 * j + 3]};
    }
    __syncthreads();
    if (threadIdx.x < kQB) {
      float x = kQuantTiny;
#pragma unroll
      for (int i = 0; i < 16; ++i) x = fmaxf(x, part[i][threadIdx.x]);
      part[0][threadIdx.x] = x;
      if (k0 + threadIdx.x < s.cols) scale[(r0 / kQB) * scale_ld + k0 + threadIdx.x] = block_scale(x);
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
      const int n = c * kRun + j;
      const BlockQuant bq(part[0][n]);
      float x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float f[kRun];
        v[i].values(f);
        x[i] = bq(f[j]);
      }
      tile[n * kTLd + g] = e4m3_quad(x[0], x[1], x[2], x[3]);
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
  const char* x = static_cast<const char*>(a.x);
  const Source s{x, a.rows, a.cols, a.ld, x + ((a.rows - 1) * a.ld + a.cols) * (int64_t)sizeof(T)};
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

hipError_t launch_quantize_scatter(const void* x, int64_t T, int cols, const int32_t* row_of, int k, char* q,
                                   float* scale, int64_t scale_ld, hipStream_t s) {
  if (T <= 0) return hipSuccess;
  quantize_scatter_kernel<<<(unsigned)((T + 3) / 4), 256, 0, s>>>(static_cast<const char*>(x), T, cols, row_of, k, q,
                                                                  scale, scale_ld);
  return hipGetLastError();
}

}  // namespace moe
