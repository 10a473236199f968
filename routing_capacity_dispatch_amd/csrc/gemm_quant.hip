// Products of e4m3 operands with one fp32 scale for each block of 128 along
// K (weights: 128 x 128 blocks), on v_mfma_f32_16x16x128_f8f6f4: one
// instruction covers exactly one block, so
//   C[m][n] = sum over blocks b of sa[m][b] sb[n][b] P_b[m][n],
// P_b the matrix-core product of block b (started from zero) and the scales
// applied in fp32 as it is added.
//
// Both operands hold 32 bytes of K per lane; A and B are loaded alike, so
// the order of K inside a block does not matter as long as it is the same:
// lane l takes bytes 16 (l >> 4) .. + 15 and 64 + 16 (l >> 4) .. + 15 of row
// l & 15, which makes each load instruction read 64 contiguous bytes a row.
#include "kernels.h"
#include "quant.h"

namespace moe {
namespace {

typedef int i32x8_t __attribute__((ext_vector_type(8)));

struct Frag8 {
  uint4 lo, hi;
};

__device__ __forceinline__ Frag8 load_frag(const char* row, int lane) {
  const char* p = row + ((lane >> 4) << 4);
  return Frag8{ld16(p), ld16(p + 64)};
}

// P = A B^T over one block of 128; no scale operands, so none is applied.
__device__ __forceinline__ f32x4_t mfma_block(const Frag8& a, const Frag8& b) {
  const i32x8_t x = {(int)a.lo.x, (int)a.lo.y, (int)a.lo.z, (int)a.lo.w, (int)a.hi.x, (int)a.hi.y, (int)a.hi.z, (int)a.hi.w};
  const i32x8_t y = {(int)b.lo.x, (int)b.lo.y, (int)b.lo.z, (int)b.lo.w, (int)b.hi.x, (int)b.hi.y, (int)b.hi.z, (int)b.hi.w};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, f32x4_t{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}

__device__ __forceinline__ void store_out(int out_dt, void* C, int64_t i, float v) {
  if (out_dt == DT_BF16)
    static_cast<uint16_t*>(C)[i] = f32_to_bf16(v);
  else
    static_cast<float*>(C)[i] = v;
}

// Expert e's rows, kept inside the M rows that exist whatever the offsets say.
__device__ __forceinline__ void expert_range(const int32_t* offsets, int e, int64_t M, int64_t& row0, int64_t& rows) {
  row0 = min(max((int64_t)offsets[e], (int64_t)0), M);
  rows = min((int64_t)offsets[e + 1], M) - row0;
}

// -------------------------------------------------------------- few rows
// One wavefront: 16 rows x 16 columns, operands straight from memory.  KS
// wavefronts of the workgroup share a column tile and take every KS-th block
// of K; their sums meet in LDS in a fixed order.
constexpr int kSkinnyWaves = 4;

template <int KS>
__global__ __launch_bounds__(64 * kSkinnyWaves) void skinny_kernel(QuantGemm g) {
  __shared__ f32x4_t part[kSkinnyWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int ks = wave % KS;
  const int64_t n0 = ((int64_t)blockIdx.x * (kSkinnyWaves / KS) + wave / KS) * 16;
  const int64_t n = min(n0 + (lane & 15), g.N - 1);
  int64_t row0 = 0, rows = g.M, first = (int64_t)blockIdx.y * 16, step = (int64_t)gridDim.y * 16;
  const char* B = g.B;
  const float* sb = g.b_scale;
  if (g.offsets) {
    const int e = blockIdx.y;
    expert_range(g.offsets, e, g.M, row0, rows);
    first = 0;
    step = 16;
    B += (int64_t)e * g.b_stride;
    sb += (int64_t)e * g.b_scale_stride;
  }
  const char* brow = B + n * g.ldb;
  const float* sbp = g.b_rows == 1 ? sb + n : sb + (n >> 7) * g.b_scale_ld;
  const int64_t sb_step = g.b_rows == 1 ? g.b_scale_ld : 1;
  const int nb = g.K / kQB;
  for (int64_t m0 = first; m0 < rows; m0 += step) {
    const char* arow = g.A + (row0 + min(m0 + (lane & 15), rows - 1)) * g.lda;
    const int64_t mr = m0 + (lane >> 4) * 4;
    const float* sap[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) sap[r] = g.a_scale + row0 + min(mr + r, rows - 1);
    f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
    for (int b = ks; b < nb; b += KS) {
      const Frag8 fa = load_frag(arow + (int64_t)b * kQB, lane), fb = load_frag(brow + (int64_t)b * kQB, lane);
      const float s = sbp[b * sb_step];
      const f32x4_t p = mfma_block(fa, fb);
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[r] = fmaf(p[r], s * sap[r][b * g.a_scale_ld], acc[r]);
    }
    if constexpr (KS > 1) {
      __syncthreads();
      part[wave][lane] = acc;
      __syncthreads();
      if (ks == 0) {
#pragma unroll
        for (int j = 1; j < KS; ++j)
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[r] += part[wave + j][lane][r];
      }
    }
    if (ks == 0 && n0 + (lane & 15) < g.N) {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (mr + r < rows) store_out(g.out_dt, g.C, (row0 + mr + r) * g.ldc + n, acc[r]);
    }
  }
}

// One workgroup: an expert's 128 features (16 per wavefront, gate and up),
// 16 rows at a time, so the hidden rows' scale of those features is the
// maximum over the workgroup.
__global__ __launch_bounds__(512) void skinny_gate_up_kernel(QuantGateUp g) {
  __shared__ float part[8][16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int e = blockIdx.y;
  int64_t row0 = 0, rows = g.M;
  if (g.offsets) {
    expert_range(g.offsets, e, g.M, row0, rows);
  }
  const int nb = g.K / kQB;
  const int fb = blockIdx.x;
  const int f = fb * kQB + wave * 16 + (lane & 15);
  const char* wg = g.Wg + ((int64_t)e * g.F + f) * g.K;
  const char* wu = g.Wu + ((int64_t)e * g.F + f) * g.K;
  const float* sg = g.sg + ((int64_t)e * (g.F / kQB) + fb) * nb;
  const float* su = g.su + ((int64_t)e * (g.F / kQB) + fb) * nb;
  const int64_t col = (g.offsets ? 0 : (int64_t)e * g.F) + fb * kQB;
  for (int64_t m0 = 0; m0 < rows; m0 += 16) {
    const char* arow = g.A + (row0 + min(m0 + (lane & 15), rows - 1)) * g.lda;
    const int64_t mr = m0 + (lane >> 4) * 4;
    const float* sap[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) sap[r] = g.a_scale + row0 + min(mr + r, rows - 1);
    f32x4_t ga = {0.f, 0.f, 0.f, 0.f}, ua = {0.f, 0.f, 0.f, 0.f};
    for (int b = 0; b < nb; ++b) {
      const int64_t k = (int64_t)b * kQB;
      const Frag8 fa = load_frag(arow + k, lane), f0 = load_frag(wg + k, lane), f1 = load_frag(wu + k, lane);
      const f32x4_t p = mfma_block(fa, f0), q = mfma_block(fa, f1);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float s = sap[r][b * g.a_scale_ld];
        ga[r] = fmaf(p[r], s * sg[b], ga[r]);
        ua[r] = fmaf(q[r], s * su[b], ua[r]);
      }
    }
    float h[4], mx[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      h[r] = silu(ga[r]) * ua[r];
      mx[r] = fabsf(h[r]);
      for (int d = 1; d < 16; d <<= 1) mx[r] = fmaxf(mx[r], __shfl_xor(mx[r], d));
    }
    __syncthreads();
    if ((lane & 15) == 0)
#pragma unroll
      for (int r = 0; r < 4; ++r) part[wave][(lane >> 4) * 4 + r] = mx[r];
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float amax = kQuantTiny;
#pragma unroll
      for (int w = 0; w < 8; ++w) amax = fmaxf(amax, part[w][(lane >> 4) * 4 + r]);
      if (mr + r < rows) {
        const BlockQuant bq(amax);
        g.H[(row0 + mr + r) * g.ldh + col + wave * 16 + (lane & 15)] = (char)(e4m3_quad(bq(h[r]), 0.f, 0.f, 0.f) & 0xFF);
        if (wave == 0 && (lane & 15) == 0) g.h_scale[(col / kQB) * g.h_scale_ld + row0 + mr + r] = block_scale(amax);
      }
    }
  }
}

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

int64_t quant_gemm_ws_bytes(const QuantGemm& g) { return 0; }

hipError_t launch_quant_gemm(const QuantGemm& g, void* ws, hipStream_t s) {
  if (g.M <= 0 || g.N <= 0) return hipSuccess;
  const int64_t rows = g.offsets ? g.E : (cdiv(g.M, 16) < 65535 ? cdiv(g.M, 16) : 65535);
  skinny_kernel<1><<<dim3((unsigned)cdiv(g.N, 16 * kSkinnyWaves), (unsigned)rows), 64 * kSkinnyWaves, 0, s>>>(g);
  return hipGetLastError();
}

hipError_t launch_quant_gate_up(const QuantGateUp& g, hipStream_t s) {
  if (g.M <= 0 || g.E <= 0) return hipSuccess;
  skinny_gate_up_kernel<<<dim3((unsigned)(g.F / kQB), (unsigned)g.E), 512, 0, s>>>(g);
  return hipGetLastError();
}

}  // namespace moe
