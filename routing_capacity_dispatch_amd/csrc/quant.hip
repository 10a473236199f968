// Quantiser to e4m3 with one fp32 scale for 1 x 128 or 128 x 128 blocks of
// the (possibly transposed) source:  s = max|x| / 448, q = e4m3(448 x / max|x|).
//
// One workgroup per 128 x 128 tile of the source, staged in LDS as fp32, so
// that the transposed result is written in whole 128-byte rows as well.
#include "kernels.h"
#include "quant.h"

namespace moe {
namespace {

constexpr int kTileLd = kQB + 1;  // floats per staged row: odd, so that columns spread over the banks

template <typename T>
__device__ __forceinline__ float load_elem(const void* p, int64_t i);
template <>
__device__ __forceinline__ float load_elem<float>(const void* p, int64_t i) {
  return static_cast<const float*>(p)[i];
}
template <>
__device__ __forceinline__ float load_elem<bf16_t>(const void* p, int64_t i) {
  return bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
}

template <typename T>
__global__ __launch_bounds__(256) void quantize_tile_kernel(QuantizeArgs a, int tiles_c) {
  __shared__ float tile[kQB * kTileLd];
  __shared__ float part[4];
  const int tr = blockIdx.x / tiles_c, tc = blockIdx.x - tr * tiles_c;
  const int64_t r0 = (int64_t)tr * kQB, c0 = (int64_t)tc * kQB;
  for (int i = threadIdx.x; i < kQB * kQB; i += 256) {
    const int r = i >> 7, c = i & 127;
    float v = 0.0f;
    if (r0 + r < a.rows && c0 + c < a.cols) v = load_elem<T>(a.x, (r0 + r) * a.ld + c0 + c);
    // logical row first: the row of the result
    tile[a.transpose ? c * kTileLd + r : r * kTileLd + c] = v;
  }
  __syncthreads();
  const int64_t R0 = a.transpose ? c0 : r0, K0 = a.transpose ? r0 : c0;
  const int64_t R = a.transpose ? a.cols : a.rows;
  // two threads a row, 64 values each
  const int row = threadIdx.x >> 1, half = threadIdx.x & 1;
  const float* src = tile + row * kTileLd + half * 64;
  float amax = 0.0f;
  for (int i = 0; i < 64; ++i) amax = fmaxf(amax, fabsf(src[i]));
  amax = fmaxf(amax, __shfl_xor(amax, 1));
  if (a.block_rows == kQB) {
    for (int d = 2; d < 64; d <<= 1) amax = fmaxf(amax, __shfl_xor(amax, d));
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = amax;
    __syncthreads();
    amax = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
  }
  amax = fmaxf(amax, kQuantTiny);
  const BlockQuant bq(amax);
  if (R0 + row < R) {
    char* dst = a.q + (R0 + row) * a.ldq + K0 + half * 64;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float* s = src + i * 16 + j * 4;
        w[j] = e4m3_quad(bq(s[0]), bq(s[1]), bq(s[2]), bq(s[3]));
      }
      st16(dst + i * 16, make_uint4(w[0], w[1], w[2], w[3]));
    }
    if (a.block_rows == 1) {
      if (half == 0) a.scale[(K0 / kQB) * a.scale_ld + R0 + row] = block_scale(amax);
    } else if (threadIdx.x == 0) {
      a.scale[(R0 / kQB) * a.scale_ld + K0 / kQB] = block_scale(amax);
    }
  }
}

}  // namespace

hipError_t launch_quantize(const QuantizeArgs& a, hipStream_t s) {
  if (a.rows <= 0 || a.cols <= 0) return hipSuccess;
  const int64_t tr = (a.rows + kQB - 1) / kQB, tc = (a.cols + kQB - 1) / kQB;
  const dim3 grid((unsigned)(tr * tc));
  if (a.dt == DT_F32)
    quantize_tile_kernel<float><<<grid, 256, 0, s>>>(a, (int)tc);
  else
    quantize_tile_kernel<bf16_t><<<grid, 256, 0, s>>>(a, (int)tc);
  return hipGetLastError();
}

}  // namespace moe
