// Linear layers with their epilogue: y = act(x W^T + b) + r, and the gradients
// dx = d W, dW = d^T x, db = sum of d over rows, d = dy act'(pre).  bf16
// operands, fp32 accumulation, each result rounded once.
//
// Few rows, and small products, go straight from memory into matrix
// instructions, the wavefronts of a workgroup sharing K.  The rest takes the
// tiles of gemm_buf.h, in four kinds (below), the K of tiles that are few or
// long shared by several workgroups.  Both products of a backward run in one
// launch, so that one fills the compute units that the other leaves idle.
#include "common.h"
#include "gemm_buf.h"
#include "kernels.h"
#include "stream.h"

namespace moe {
namespace {

using core::Acc;
using core::dense_tile;
using core::xcd_order;

// All 160 KB of LDS, one workgroup a CU: the fastest where there are several
// rounds of them (16384 x 6144 x 2048: 360 us, 128 x 128 tiles 400)
using BigTile = core::Tile<256, 256, 4, 2, 64, 2, 3>;
// Two workgroups of 8 wavefronts a CU, one's epilogue under the other's loop (6144 x
// 4096 x 2048 with everything: 120 us, big tiles 145; with 4 wavefronts 4608 x 4096
// x 2048 takes 107 instead of 89)
using SmallTile = core::Tile<128, 128, 4, 2, 64, 2, 2>;
// For at most one a CU, five K tiles in flight (2048 x 2048 x 2048: 24.5 us,
// 28 with two; with 4 wavefronts 28)
using MidTile = core::Tile<128, 128, 4, 2, 64, 5>;
// Two workgroups a CU, five K tiles in flight each: for few tiles, whose time
// is the loads' (512 x 2048 x 2048: 15 us, 128 x 128 30, or 26 with K shared;
// nine K tiles in flight: the same)
using DeepTile = core::Tile<64, 64, 2, 2, 64, 5>;

int64_t cdiv64(int64_t a, int64_t b) { return (a + b - 1) / b; }

// ------------------------------------------------------------- epilogue
// Phi(u), the normal distribution's integral up to u, and e = exp(-u^2 / 2):
// Phi(-|u|) = erfc(z) / 2, z = |u| / sqrt 2, and erfc(z) exp(z^2) is smooth in
// t = 1 / (1 + 0.32 z): a polynomial of degree 8 fitted to it (weighted least
// squares towards the least relative error over 0 <= z <= 10) is off by 6e-8 of
// it.  A quarter of erff's instructions, and no cancellation for negative u.
__device__ __forceinline__ float normal_cdf(float u, float& e) {
  const float z = fabsf(u) * 0.70710678118654752f;
  const float t = __builtin_amdgcn_rcpf(fmaf(0.32f, z, 1.0f));
  float q = -1.768869357629155e-01f;
  q = fmaf(q, t, 7.061705589258108e-01f);
  q = fmaf(q, t, -7.767581516428086e-01f);
  q = fmaf(q, t, 8.161300437402584e-01f);
  q = fmaf(q, t, -1.918512878265418e-01f);
  q = fmaf(q, t, 2.817898999523091e-01f);
  q = fmaf(q, t, 1.584962424419372e-01f);
  q = fmaf(q, t, 1.830312881592669e-01f);
  q = fmaf(q, t, -1.216013331140874e-04f);
  e = __expf(-0.5f * u * u);
  const float tail = 0.5f * q * e;
  return u < 0.0f ? tail : 1.0f - tail;
}

__device__ __forceinline__ float act_of(float u, int act) {
  switch (act) {
    case ACT_RELU: return u < 0.0f ? 0.0f : u;  // a NaN stays one
    case ACT_SILU: return silu(u);
    case ACT_GELU: {
      float e;
      return u * normal_cdf(u, e);
    }
    default: return u;
  }
}
__device__ __forceinline__ float act_slope(float u, int act) {
  switch (act) {
    case ACT_RELU: return u > 0.0f ? 1.0f : 0.0f;
    case ACT_SILU: {
      const float p = sigmoid(u);
      return p * (1.0f + u * (1.0f - p));
    }
    case ACT_GELU: {  // Phi(u) + u phi(u)
      float e;
      const float p = normal_cdf(u, e);
      return fmaf(u * 0.39894228040143268f, e, p);
    }
    default: return 1.0f;
  }
}

__device__ __forceinline__ float ld_elem(const void* p, int64_t i, int dt) {
  return dt == DT_F32 ? static_cast<const float*>(p)[i] : bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
}
__device__ __forceinline__ void st_elem(void* p, int64_t i, int dt, float v) {
  if (dt == DT_F32)
    static_cast<float*>(p)[i] = v;
  else
    static_cast<uint16_t*>(p)[i] = f32_to_bf16(v);
}

// C neighbouring values of a row, C 4 or 8, at any alignment of an element
// (the hardware takes wide accesses at any address)
typedef u32x4_t u32x4_any_t __attribute__((aligned(2)));
typedef unsigned int u32x2_any_t __attribute__((ext_vector_type(2), aligned(2)));
template <int C>
__device__ __forceinline__ void ld_vec(const void* p, int64_t i, int dt, float* v) {
  if (dt == DT_F32) {
    const uint16_t* q = reinterpret_cast<const uint16_t*>(static_cast<const float*>(p) + i);
#pragma unroll
    for (int c = 0; c < C; c += 4) unpack(buf::ld16_any(q + 2 * c), v + c, float{});
  } else {
    const uint16_t* q = static_cast<const uint16_t*>(p) + i;
    if constexpr (C == 8) {
      unpack(buf::ld16_any(q), v, bf16_t{});
    } else {
      const u32x2_any_t w = *reinterpret_cast<const u32x2_any_t*>(q);
      v[0] = __uint_as_float(w.x << 16);
      v[1] = __uint_as_float(w.x & 0xFFFF0000u);
      v[2] = __uint_as_float(w.y << 16);
      v[3] = __uint_as_float(w.y & 0xFFFF0000u);
    }
  }
}
// kStream: with the nontemporal hint
template <bool kStream>
__device__ __forceinline__ void st16_any(void* p, const uint4& v) {
  const u32x4_t w = {v.x, v.y, v.z, v.w};
  if constexpr (kStream)
    __builtin_nontemporal_store(w, static_cast<u32x4_any_t*>(p));
  else
    *static_cast<u32x4_any_t*>(p) = w;
}
template <int C, bool kStream = false>
__device__ __forceinline__ void st_vec(void* p, int64_t i, int dt, const float* v) {
  if (dt == DT_F32) {
    float* q = static_cast<float*>(p) + i;
#pragma unroll
    for (int c = 0; c < C; c += 4) st16_any<kStream>(q + c, pack(v + c, float{}));
  } else {
    uint16_t* q = static_cast<uint16_t*>(p) + i;
    if constexpr (C == 8) {
      st16_any<kStream>(q, pack(v, bf16_t{}));
    } else {
      u32x2_any_t w;
      w.x = bf16_pair(v[0], v[1]);
      w.y = bf16_pair(v[2], v[3]);
      *reinterpret_cast<u32x2_any_t*>(q) = w;
    }
  }
}

// The residual of C neighbouring columns as it lies in memory, fetched before
// it is needed (where all of them are inside the row).
template <int C>
struct Residual {
  uint4 w[C / 4];  // C fp32, or C bf16 in the first
};
template <int C>
__device__ __forceinline__ Residual<C> fetch(const Linear& g, int64_t m, int n) {
  Residual<C> r;
  if (g.res && n + C <= g.N) {
    const int64_t at = m * g.ldr + n;
    if (g.out_dt == DT_F32) {
#pragma unroll
      for (int i = 0; i < C / 4; ++i)
        r.w[i] = buf::ld16_any(reinterpret_cast<const uint16_t*>(static_cast<const float*>(g.res) + at + 4 * i));
    } else if constexpr (C == 8) {
      r.w[0] = buf::ld16_any(static_cast<const uint16_t*>(g.res) + at);
    } else {
      const u32x2_any_t q = *reinterpret_cast<const u32x2_any_t*>(static_cast<const uint16_t*>(g.res) + at);
      r.w[0] = make_uint4(q.x, q.y, 0, 0);
    }
  }
  return r;
}

template <int C>
struct Bias {
  float v[C];
};
template <int C>
__device__ __forceinline__ Bias<C> bias_at(const Linear& g, int n) {
  Bias<C> b;
#pragma unroll
  for (int c = 0; c < C; ++c) b.v[c] = g.bias ? ld_elem(g.bias, min(n + c, g.N - 1), g.bias_dt) : 0.0f;
  return b;
}

// C neighbouring sums of row m from column n on: bias, pre-activation out,
// activation, residual, result.
// kStream: results of many large tiles, written past the caches, which the
// operands then keep (16384 x 6144 x 2048 with everything: 506 -> 479 us).
template <int C, bool kStream = false>
__device__ __forceinline__ void finish(const Linear& g, int64_t m, int n, float* v, const Bias<C>& bias,
                                       const Residual<C>& ahead) {
  if (n >= g.N) return;
  const bool whole = n + C <= g.N;
  const int cnt = min(C, g.N - n);
#pragma unroll
  for (int c = 0; c < C; ++c) v[c] += bias.v[c];
  if (g.pre) {
    if (whole) {
      st_vec<C, kStream>(g.pre, m * g.ldp + n, DT_BF16, v);
    } else {
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (c < cnt) st_elem(g.pre, m * g.ldp + n + c, DT_BF16, v[c]);
    }
  }
  if (g.act != ACT_NONE) {
#pragma unroll
    for (int c = 0; c < C; ++c) v[c] = act_of(v[c], g.act);
  }
  if (g.res && whole) {
    float r[8];
    if (g.out_dt == DT_F32) {
#pragma unroll
      for (int i = 0; i < C / 4; ++i) unpack(ahead.w[i], r + 4 * i, float{});
    } else {
      unpack(ahead.w[0], r, bf16_t{});
    }
#pragma unroll
    for (int c = 0; c < C; ++c) v[c] += r[c];
  } else if (g.res) {
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (c < cnt) v[c] += ld_elem(g.res, m * g.ldr + n + c, g.out_dt);
  }
  if (whole) {
    st_vec<C, kStream>(g.y, m * g.ldy + n, g.out_dt, v);
  } else {
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (c < cnt) st_elem(g.y, m * g.ldy + n + c, g.out_dt, v[c]);
  }
}

// ---------------------------------------------------------------- tiles
// One tile of C over one share of K; with several shares the fp32 sums go to
// g.part [shares][M][ldpart] and linear_finish_kernel adds them.  t: tile and share.
// kRegs: operands of any alignment, by way of registers.
template <class TL, bool kRegs, bool AK, bool BK>
__device__ __forceinline__ void linear_tile(const Linear& g, int t, char* lds) {
  const int tiles = g.tiles_m * g.tiles_n;
  const int share = t / tiles;
  int mt, nt;
  dense_tile(t - share * tiles, g.tiles_m, g.tiles_n, mt, nt);
  const int m0 = mt * TL::BM, n0 = nt * TL::BN;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int k0 = share * g.share_k, kn = min(g.share_k, g.K - k0), ktiles = (kn + TL::BK - 1) / TL::BK;
  const uint16_t* x = static_cast<const uint16_t*>(g.x) + (AK ? k0 * g.ldx : k0);
  const uint16_t* w = static_cast<const uint16_t*>(g.w) + (BK ? k0 * g.ldw : k0);
  // a lane's columns are the same in every row; their bias is on its way while
  // the product runs (the big tile has no registers left for it)
  Bias<8> bias;
  const int c0 = n0 + buf::Epilogue<TL>::column();
  if constexpr (TL::BM < 256) bias = bias_at<8>(g, c0);
  Acc<TL> acc;
  acc.zero();
  if constexpr (kRegs) {
    buf::ARegs<TL, AK> a;
    buf::BRegs<TL, BK> b;
    a.init(x, m0, (int)g.M, g.ldx, kn, wave, lane);
    b.init(w, n0, g.N, g.ldw, kn, wave, lane);
    buf::mainloop_regs<TL, AK, BK, false>(a, b, ktiles, lds, acc);
  } else {
    buf::ARows<TL, AK> a;
    buf::BRows<TL, BK> b;
    a.init(x, m0, (int)g.M, g.ldx, kn, wave, lane);
    b.init(w, n0, g.N, g.ldw, kn, wave, lane);
    if constexpr (TL::NS == 2)
      buf::mainloop<TL, AK, BK, false>(a, b, ktiles, lds, acc);
    else
      buf::mainloop_pipe<TL, AK, BK, false>(a, b, ktiles, lds, acc);
  }
  const int rows = min((int)g.M - m0, TL::BM);
  if (g.shares > 1) {
    float* part = g.part + (int64_t)share * g.M * g.ldpart;
    buf::Epilogue<TL>::run(acc, lds, rows, [&](int r, int c, float* v) {
      if (n0 + c < g.N) st_vec<8>(part, (int64_t)(m0 + r) * g.ldpart + n0 + c, DT_F32, v);
    });
  } else {
    if constexpr (TL::BM == 256) bias = bias_at<8>(g, c0);
    buf::Epilogue<TL>::template run<Residual<8>>(
        acc, lds, rows, [&](int r, int c) { return fetch<8>(g, m0 + r, n0 + c); },
        [&](int r, int c, float* v, const Residual<8>& x) { finish<8, TL::BM == 256>(g, m0 + r, n0 + c, v, bias, x); });
  }
}

template <class TL>
constexpr int tile_lds() {
  return TL::MAIN_LDS > buf::Epilogue<TL>::kBytes ? TL::MAIN_LDS : buf::Epilogue<TL>::kBytes;
}

template <class TL, bool kRegs>
__global__ __launch_bounds__(TL::THREADS) void linear_tile_kernel(Linear g) {
  __shared__ __attribute__((aligned(1024))) char lds[tile_lds<TL>()];
  const int t = xcd_order(blockIdx.x, gridDim.x);
  if (t < g.tiles_m * g.tiles_n * g.shares) linear_tile<TL, kRegs, false, false>(g, t, lds);
}

// db[n] = sum of part[.][n], in order within each of the workgroup's row lanes
__device__ __forceinline__ void bias_sums(const LinearGrads& p, int block, float* red) {
  const int c = threadIdx.x & 63, r = threadIdx.x >> 6, lanes = blockDim.x >> 6;
  const int n = block * 64 + c;
  float s = 0.0f;
  if (n < p.N) {
#pragma unroll 4
    for (int64_t b = r; b < p.sum_blocks; b += lanes) s += p.sums[b * p.N + n];
  }
  red[r * 64 + c] = s;
  __syncthreads();
  if (r != 0 || n >= p.N) return;
  for (int i = 1; i < lanes; ++i) s += red[i * 64 + c];
  p.db[n] = s;
}

// dw (both operands K-major, the longer K mostly: first), dx (W K-major), db.
template <class TL, bool kRegs>
__global__ __launch_bounds__(TL::THREADS) void linear_grads_kernel(LinearGrads p) {
  __shared__ __attribute__((aligned(1024))) char lds[tile_lds<TL>()];
  int b = blockIdx.x;
  if (b < p.grid_dw) {
    const int t = xcd_order(b, p.grid_dw);
    if (t < p.dw.tiles_m * p.dw.tiles_n * p.dw.shares) linear_tile<TL, kRegs, true, true>(p.dw, t, lds);
    return;
  }
  b -= p.grid_dw;
  if (b < p.grid_dx) {
    const int t = xcd_order(b, p.grid_dx);
    if (t < p.dx.tiles_m * p.dx.tiles_n * p.dx.shares) linear_tile<TL, kRegs, false, true>(p.dx, t, lds);
    return;
  }
  bias_sums(p, b - p.grid_dx, reinterpret_cast<float*>(lds));
}

// Sums of the shares, in their order, then the epilogue: 8 columns a thread.
__device__ __forceinline__ void finish_at(const Linear& g, int64_t i) {
  const int64_t chunks = g.ldpart / 8;
  if (g.shares < 2 || i >= g.M * chunks) return;
  const int64_t m = i / chunks;
  const int n = (int)(i - m * chunks) * 8;
  const Residual<8> ahead = fetch<8>(g, m, n);
  const Bias<8> bias = bias_at<8>(g, n);
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < g.shares; ++s) {
    float u[8];
    ld_vec<8>(g.part, ((int64_t)s * g.M + m) * g.ldpart + n, DT_F32, u);
#pragma unroll
    for (int c = 0; c < 8; ++c) v[c] += u[c];
  }
  finish<8>(g, m, n, v, bias, ahead);
}
__global__ __launch_bounds__(256) void linear_finish_kernel(Linear g) {
  finish_at(g, (int64_t)blockIdx.x * 256 + threadIdx.x);
}
__global__ __launch_bounds__(256) void linear_grads_finish_kernel(LinearGrads p, int first) {
  if ((int)blockIdx.x < first)
    finish_at(p.dw, (int64_t)blockIdx.x * 256 + threadIdx.x);
  else
    finish_at(p.dx, (int64_t)(blockIdx.x - first) * 256 + threadIdx.x);
}

// ----------------------------------------------- straight from memory
constexpr int kStreamWaves = 4;
using buf::ld16_any;
using buf::ld8_until;

// 16 MB rows of x by 16 SB rows of W, operands of any alignment, the wavefronts
// of the workgroup sharing K: nothing passes through LDS but their sums, and no
// wavefront waits for another until the end.  The weights are the first operand,
// so a lane ends with 4 neighbouring columns of row lane & 15 of each block.
// Its loads take 64 bytes of a row at a time, which streams few rows' weights as
// well as tiles do, and many rows' worse: 1 x 6144 x 2048 7.7 us (DeepTile 10.1),
// 64 x 1024 x 1024 4.8 (9.0), 333 x 1001 x 1250 10 (12), but 64 x 6144 x 2048 20
// (13.5) and 512 x 2048 x 2048 26 (15).
template <int SB, int MB>
__global__ __launch_bounds__(64 * kStreamWaves) void linear_stream_kernel(Linear g) {
  constexpr int kBlocks = SB * MB, kOwn = (kBlocks + kStreamWaves - 1) / kStreamWaves;
  __shared__ f32x4_t part[kStreamWaves][kBlocks][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int m0 = blockIdx.y * 16 * MB, n0 = blockIdx.x * 16 * SB, at = (lane >> 4) * 8;
  const uint16_t* w[SB];
  const uint16_t* x[MB];
#pragma unroll
  for (int s = 0; s < SB; ++s)
    w[s] = static_cast<const uint16_t*>(g.w) + (int64_t)min(n0 + s * 16 + (lane & 15), g.N - 1) * g.ldw + at;
#pragma unroll
  for (int b = 0; b < MB; ++b)
    x[b] = static_cast<const uint16_t*>(g.x) + (int64_t)min(m0 + b * 16 + (lane & 15), (int)g.M - 1) * g.ldx + at;
  // block q = (q / MB, q % MB) is finished by wavefront q % kStreamWaves: what it
  // reads is on its way before the product starts
  Bias<4> bias[kOwn];
  Residual<4> ahead[kOwn];
  auto row = [&](int q) { return m0 + q % MB * 16 + (lane & 15); };
  auto col = [&](int q) { return n0 + q / MB * 16 + (lane >> 4) * 4; };
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    const int q = i * kStreamWaves + wave;
    if (q < kBlocks) bias[i] = bias_at<4>(g, col(q));
    if (q < kBlocks && row(q) < g.M) ahead[i] = fetch<4>(g, row(q), col(q));
  }
  f32x4_t acc[SB][MB];
#pragma unroll
  for (int s = 0; s < SB; ++s)
#pragma unroll
    for (int b = 0; b < MB; ++b) acc[s][b] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  stream<kStreamWaves, SB, MB, false, 8>(w, x, g.K / 64, acc, [](const uint16_t* p) { return ld16_any(p); });
  // fewer than 64 values of K are left: 32 for each of the last two wavefronts
  {
    const int k = (g.K & ~63) + (kStreamWaves - 1 - wave) * 32;
    if (k < g.K) {
      uint4 v[MB];
#pragma unroll
      for (int b = 0; b < MB; ++b) v[b] = ld8_until(x[b] - at, k + at, g.K);
#pragma unroll
      for (int s = 0; s < SB; ++s) {
        const uint4 a = ld8_until(w[s] - at, k + at, g.K);
#pragma unroll
        for (int b = 0; b < MB; ++b) acc[s][b] = mfma_bf16(a, v[b], acc[s][b]);
      }
    }
  }
#pragma unroll
  for (int s = 0; s < SB; ++s)
#pragma unroll
    for (int b = 0; b < MB; ++b) part[wave][s * MB + b][lane] = acc[s][b];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    const int q = i * kStreamWaves + wave;
    if (q >= kBlocks) break;
    f32x4_t sum = part[0][q][lane];
#pragma unroll
    for (int j = 1; j < kStreamWaves; ++j) sum += part[j][q][lane];
    float v[4] = {sum[0], sum[1], sum[2], sum[3]};
    if (row(q) < g.M) finish<4>(g, row(q), col(q), v, bias[i], ahead[i]);
  }
}
static_assert(kStreamWaves >= 2, "the rest of K goes to two wavefronts");

// -------------------------------------------------------- copies, slopes
// Rows [rows][cols] into rows of ldd (a multiple of 8), zeros past cols.
__device__ __forceinline__ void pack_at(const PackRows& p, int64_t i) {
  const int64_t chunks = p.ldd / 8;
  if (i >= p.rows * chunks) return;
  const int64_t r = i / chunks;
  const int c = (int)(i - r * chunks) * 8;
  st16(static_cast<uint16_t*>(p.dst) + r * p.ldd + c, ld8_until(static_cast<const uint16_t*>(p.src) + r * p.ld, c, p.cols));
}
__global__ __launch_bounds__(256) void pack_rows_kernel(PackRows a, PackRows b, unsigned first) {
  if (blockIdx.x < first)
    pack_at(a, (int64_t)blockIdx.x * 256 + threadIdx.x);
  else
    pack_at(b, (int64_t)(blockIdx.x - first) * 256 + threadIdx.x);
}

// d = dy act'(pre) as bf16 rows of ldd (zeros past N), and sums of d (before
// its rounding) over the rows of each block of kSlopeRows: part [blocks][N].
// bf16 is what the matrix instructions take beside x and W: the rounding is as
// large as that of the results (together 0.0024 of their norm, 0.0017 without it);
// d in two bf16 numbers would be without it for twice the matrix instructions.
constexpr int kSlopeRows = 32;
struct Slope {
  const void* dy;
  int64_t ldy;
  int dy_dt;
  const uint16_t* pre;
  int64_t ldp;
  int act;
  int64_t M;
  int N;
  uint16_t* d;     // null: only the sums
  int64_t ldd;
  float* part;     // null: no sums
};
// 256 threads: 16 chunks of 8 columns x 16 row lanes
__global__ __launch_bounds__(256) void slope_kernel(Slope p) {
  __shared__ float red[16][16 * 8 + 4];
  const int cx = threadIdx.x & 15, ry = threadIdx.x >> 4;
  const int n = (blockIdx.x * 16 + cx) * 8;
  const int64_t r0 = (int64_t)blockIdx.y * kSlopeRows;
  float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  const bool whole = n + 8 <= p.N;
#pragma unroll
  for (int i = 0; i < kSlopeRows / 16; ++i) {
    const int64_t m = r0 + i * 16 + ry;
    if (m >= p.M || n >= p.N) continue;
    float d[8], u[8];
    if (whole) {
      ld_vec<8>(p.dy, m * p.ldy + n, p.dy_dt, d);
      if (p.act != ACT_NONE) ld_vec<8>(p.pre, m * p.ldp + n, DT_BF16, u);
    } else {
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const bool in = n + c < p.N;
        d[c] = in ? ld_elem(p.dy, m * p.ldy + n + c, p.dy_dt) : 0.0f;
        u[c] = in && p.act != ACT_NONE ? bf16_to_f32(p.pre[m * p.ldp + n + c]) : 0.0f;
      }
    }
    if (p.act != ACT_NONE) {
#pragma unroll
      for (int c = 0; c < 8; ++c) d[c] = n + c < p.N ? d[c] * act_slope(u[c], p.act) : 0.0f;
    }
    if (p.d) st_vec<8>(p.d, m * p.ldd + n, DT_BF16, d);
#pragma unroll
    for (int c = 0; c < 8; ++c) sum[c] += d[c];
  }
  if (!p.part) return;
#pragma unroll
  for (int c = 0; c < 8; ++c) red[ry][cx * 8 + c] = sum[c];
  __syncthreads();
  if (threadIdx.x < 128) {
    float s = 0.0f;
#pragma unroll
    for (int r = 0; r < 16; ++r) s += red[r][threadIdx.x];
    const int col = blockIdx.x * 128 + threadIdx.x;
    if (col < p.N) p.part[(int64_t)blockIdx.y * p.N + col] = s;
  }
}

unsigned grid8(int64_t n) { return (unsigned)((n + 7) & ~int64_t(7)); }

int tile_side(int cls) { return cls == TILE_BIG ? 256 : cls == TILE_DEEP ? 64 : 128; }

int slots_of(int cls) { return cls == TILE_BIG || cls == TILE_MID ? 256 : 512; }

// Microseconds of one K tile of a workgroup, as measured with every slot taken.
double k_tile_us(int cls) { return cls == TILE_BIG ? 1.6 : cls == TILE_SMALL ? 0.9 : cls == TILE_MID ? 0.7 : 0.35; }

void set_tiles(Linear& g, const LinearPlan& p) {
  const int side = tile_side(p.cls);
  g.tiles_m = (int)cdiv64(g.M, side);
  g.tiles_n = (int)cdiv64(g.N, side);
  g.shares = p.shares;
  g.share_k = p.share_k;
  g.ldpart = (g.N + 7) & ~7;
}

unsigned finish_grid(const Linear& g) { return g.shares > 1 ? (unsigned)cdiv64(g.M * (g.ldpart / 8), 256) : 0; }

}  // namespace

namespace {
// Length in K tiles of n0 tiles of K k0 and n1 of k1 <= k0 on 256 CUs, the longer
// ones first, the shorter ones beside those of the last round.
int64_t rounds(int64_t n0, int64_t k0, int64_t n1, int64_t k1) {
  const int64_t last = n0 % 256;
  int64_t t = cdiv64(n0, 256) * k0;
  if (last && k1 > 0) n1 -= (256 - last) * (k0 / k1);
  return t + (n1 > 0 ? cdiv64(n1, 256) * k1 : 0);
}
// 256 tiles of 128 a side, a CU's first or second, take 0.28 of the time of 256
// of 256 a side (0.26 to 0.31 over 300 to 16384 rows).
bool big_is_faster(int64_t big, int64_t small) { return 25 * big <= 7 * small; }
int class_of(int64_t big, int64_t small, bool faster) {
  return big >= 192 && faster ? TILE_BIG : small > 256 ? TILE_SMALL : small > 128 ? TILE_MID : TILE_DEEP;
}
}  // namespace

// Big tiles where there are enough of them and their rounds of the chip come out
// shorter: a last round that is nearly empty, and tiles that lie in large part
// outside the product, count (gradients of 4096 x 2048 x 2048, 192 big tiles: 111
// us, 72 with 768 of 128 a side; of 8192 x 2048 x 4096: 256 and 282).  Up to 256
// of 128 a side have a CU each; down to 129 that is faster than twice as many
// rounds of 64 a side (1536 x 2048 x 2048 24 and 30 us, 1024 x 2048 x 2048 24 and 20).
int tile_class(int64_t big, int64_t small) {
  return class_of(big, small, big_is_faster(rounds(big, 1, 0, 0), rounds(small, 1, 0, 0)));
}
int linear_class(int64_t M0, int64_t N0, int64_t K0, int64_t M1, int64_t N1, int64_t K1) {
  if (K0 < K1) return linear_class(M1, N1, K1, M0, N0, K0);
  auto tiles = [](int64_t M, int64_t N, int64_t side) { return cdiv64(M, side) * cdiv64(N, side); };
  const int64_t b0 = tiles(M0, N0, 256), b1 = tiles(M1, N1, 256), s0 = tiles(M0, N0, 128), s1 = tiles(M1, N1, 128);
  const int64_t k0 = cdiv64(K0, 64), k1 = cdiv64(K1, 64);
  return class_of(b0 + b1, s0 + s1, big_is_faster(rounds(b0, k0, b1, k1), rounds(s0, k0, s1, k1)));
}

double linear_units(int cls, int64_t M, int64_t N, int64_t K) {
  return (double)cdiv64(M, tile_side(cls)) * (double)cdiv64(N, tile_side(cls)) * (double)cdiv64(K, 64);
}

// Shares of K: the number with which the product's own rounds of the chip, and
// the launch that joins the shares (about 4 us and their sums' way through
// memory), take the least time.  Only K longer than an even part of all the K
// tiles of the launch (`units`) is looked at.
LinearPlan linear_plan(int cls, int64_t M, int64_t N, int64_t K, double units) {
  LinearPlan p{};
  p.cls = cls;
  const int64_t kt = cdiv64(K, 64), slots = slots_of(cls);
  const int64_t tiles = cdiv64(M, tile_side(cls)) * cdiv64(N, tile_side(cls));
  const double sums = (double)M * (double)N * 8.0 / 5.0e6;  // us to write and read one share's sums
  p.shares = 1;
  if (kt > 8 && (double)kt > units / (double)slots) {
    double best = (double)(cdiv64(tiles, slots) * kt) * k_tile_us(cls);
    for (int64_t s = 2; s <= kt / 4 && s <= 64; ++s) {
      const double t = (double)(cdiv64(tiles * s, slots) * cdiv64(kt, s)) * k_tile_us(cls) + 4.0 + sums * (double)s;
      if (t < 0.95 * best) {
        best = t;
        p.shares = (int)s;
      }
    }
  }
  const int64_t each = kt > 0 ? cdiv64(kt, p.shares) : 1;
  p.share_k = (int)(each * 64);
  p.shares = kt > 0 ? (int)cdiv64(kt, each) : 1;
  p.part_bytes = p.shares > 1 ? (int64_t)p.shares * M * ((N + 7) & ~int64_t(7)) * 4 : 0;
  return p;
}

hipError_t launch_linear_tiles(const Linear& in, const LinearPlan& p, bool regs, hipStream_t s) {
  if (in.M <= 0 || in.N <= 0) return hipSuccess;
  Linear g = in;
  set_tiles(g, p);
  const unsigned grid = grid8((int64_t)g.tiles_m * g.tiles_n * g.shares);
  if (p.cls == TILE_BIG)
    linear_tile_kernel<BigTile, false><<<grid, BigTile::THREADS, 0, s>>>(g);
  else if (p.cls == TILE_SMALL)
    linear_tile_kernel<SmallTile, false><<<grid, SmallTile::THREADS, 0, s>>>(g);
  else if (p.cls == TILE_MID)
    linear_tile_kernel<MidTile, false><<<grid, MidTile::THREADS, 0, s>>>(g);
  else if (!regs)
    linear_tile_kernel<DeepTile, false><<<grid, DeepTile::THREADS, 0, s>>>(g);
  else
    linear_tile_kernel<DeepTile, true><<<grid, DeepTile::THREADS, 0, s>>>(g);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || g.shares == 1) return e;
  linear_finish_kernel<<<finish_grid(g), 256, 0, s>>>(g);
  return hipGetLastError();
}

// Few rows, or operands that the L2s hold and a few hundred workgroups take.
// blocks: 16 x 16 blocks a workgroup, 0: tiles are better.
static int stream_blocks(int64_t M, int64_t N, int64_t K) {
  if (M <= 16) return 1;
  if ((M + N) * K > int64_t(3) << 20) return 0;
  const int64_t m = cdiv64(M, 16), n = cdiv64(N, 16);
  if (m * n <= 400) return 1;
  if (cdiv64(m, 2) * cdiv64(n, 2) <= 400) return 4;
  return cdiv64(m, 4) * cdiv64(n, 2) <= 400 ? 8 : 0;
}
bool linear_streams(int64_t M, int64_t N, int64_t K) { return stream_blocks(M, N, K) > 0; }

hipError_t launch_linear_stream(const Linear& g, hipStream_t s) {
  if (g.M <= 0 || g.N <= 0) return hipSuccess;
  const unsigned m = (unsigned)cdiv64(g.M, 16), n = (unsigned)cdiv64(g.N, 16);
  const int blocks = stream_blocks(g.M, g.N, g.K);
  if (blocks == 1)
    linear_stream_kernel<1, 1><<<dim3(n, m), 64 * kStreamWaves, 0, s>>>(g);
  else if (blocks == 4)
    linear_stream_kernel<2, 2><<<dim3((n + 1) / 2, (m + 1) / 2), 64 * kStreamWaves, 0, s>>>(g);
  else
    linear_stream_kernel<2, 4><<<dim3((n + 1) / 2, (m + 3) / 4), 64 * kStreamWaves, 0, s>>>(g);
  return hipGetLastError();
}

hipError_t launch_linear_grads(const LinearGrads& in, const LinearPlan& pw, const LinearPlan& px, bool regs,
                               hipStream_t s) {
  LinearGrads p = in;
  auto range = [](Linear& g, const LinearPlan& q) {
    if (g.M <= 0 || g.N <= 0 || !g.y) {
      g.shares = 1;
      return 0;
    }
    set_tiles(g, q);
    return (int)grid8((int64_t)g.tiles_m * g.tiles_n * g.shares);
  };
  p.grid_dw = range(p.dw, pw);
  p.grid_dx = range(p.dx, px);
  const unsigned grid = (unsigned)(p.grid_dw + p.grid_dx + (p.db ? cdiv64(p.N, 64) : 0));
  if (grid == 0) return hipSuccess;
  if (pw.cls == TILE_BIG)
    linear_grads_kernel<BigTile, false><<<grid, BigTile::THREADS, 0, s>>>(p);
  else if (pw.cls == TILE_SMALL)
    linear_grads_kernel<SmallTile, false><<<grid, SmallTile::THREADS, 0, s>>>(p);
  else if (pw.cls == TILE_MID)
    linear_grads_kernel<MidTile, false><<<grid, MidTile::THREADS, 0, s>>>(p);
  else if (!regs)
    linear_grads_kernel<DeepTile, false><<<grid, DeepTile::THREADS, 0, s>>>(p);
  else
    linear_grads_kernel<DeepTile, true><<<grid, DeepTile::THREADS, 0, s>>>(p);
  const hipError_t e = hipGetLastError();
  const unsigned fw = p.grid_dw ? finish_grid(p.dw) : 0, fx = p.grid_dx ? finish_grid(p.dx) : 0;
  if (e != hipSuccess || fw + fx == 0) return e;
  linear_grads_finish_kernel<<<fw + fx, 256, 0, s>>>(p, (int)fw);
  return hipGetLastError();
}

hipError_t launch_pack_rows(const PackRows& a, const PackRows& b, hipStream_t s) {
  auto blocks = [](const PackRows& p) { return p.dst ? (unsigned)cdiv64(p.rows * (p.ldd / 8), 256) : 0u; };
  const unsigned first = blocks(a), second = blocks(b);
  if (first + second == 0) return hipSuccess;
  pack_rows_kernel<<<first + second, 256, 0, s>>>(a, b, first);
  return hipGetLastError();
}

int64_t slope_blocks(int64_t M) { return cdiv64(M, kSlopeRows); }

hipError_t launch_slope(const void* dy, int64_t ldy, int dy_dt, const void* pre, int64_t ldp, int act, int64_t M,
                        int N, void* d, int64_t ldd, float* part, hipStream_t s) {
  if (N <= 0 || M <= 0) return hipSuccess;
  Slope p{};
  p.dy = dy;
  p.ldy = ldy;
  p.dy_dt = dy_dt;
  p.pre = static_cast<const uint16_t*>(pre);
  p.ldp = ldp;
  p.act = act;
  p.M = M;
  p.N = N;
  p.d = static_cast<uint16_t*>(d);
  p.ldd = ldd;
  p.part = part;
  slope_kernel<<<dim3((unsigned)cdiv64(N, 128), (unsigned)slope_blocks(M)), 256, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace moe
