// Linear layers with their epilogue: y = act(x W^T + b) + r, and the gradients
// dx = d W, dW = d^T x, db = sum of d over rows, d = dy act'(pre).  bf16
// operands, fp32 accumulation, each result rounded once.
//
// Up to kSkinnyRows rows the product is bound by the weights' bytes: they go
// straight from memory into matrix instructions, the wavefronts of a workgroup
// sharing K.  More rows take the tiles of gemm_buf.h, K shared by several
// workgroups where the tiles alone would leave compute units idle.  Operands
// whose rows do not start on 16 bytes, or end inside 16, are copied into such
// rows first (tiles only).
#include "common.h"
#include "gemm_buf.h"
#include "kernels.h"

namespace moe {
namespace {

using core::Acc;
using core::dense_tile;
using core::xcd_order;

// All 160 KB of LDS, one workgroup a CU; or two of them a CU
using BigTile = core::Tile<256, 256, 4, 2, 64, 2, 3>;
using SmallTile = core::Tile<128, 128, 2, 2, 64, 2, 2>;

int64_t cdiv64(int64_t a, int64_t b) { return (a + b - 1) / b; }

// ------------------------------------------------------------- epilogue
__device__ __forceinline__ float act_of(float u, int act) {
  switch (act) {
    case ACT_RELU: return u < 0.0f ? 0.0f : u;  // a NaN stays one
    case ACT_SILU: return silu(u);
    case ACT_GELU: return 0.5f * u * (1.0f + erff(u * 0.70710678118654752f));
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
    case ACT_GELU:  // Phi(u) + u phi(u)
      return 0.5f * (1.0f + erff(u * 0.70710678118654752f)) + u * __expf(-0.5f * u * u) * 0.39894228040143268f;
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

// C neighbouring values of a row, C 4 or 8, on C * size bytes' alignment
template <int C>
__device__ __forceinline__ void ld_vec(const void* p, int64_t i, int dt, float* v) {
  if (dt == DT_F32) {
    const float* q = static_cast<const float*>(p) + i;
#pragma unroll
    for (int c = 0; c < C; c += 4) unpack(ld16(q + c), v + c, float{});
  } else {
    const uint16_t* q = static_cast<const uint16_t*>(p) + i;
    if constexpr (C == 8) {
      unpack(ld16(q), v, bf16_t{});
    } else {
      const uint2 w = *reinterpret_cast<const uint2*>(q);
      v[0] = __uint_as_float(w.x << 16);
      v[1] = __uint_as_float(w.x & 0xFFFF0000u);
      v[2] = __uint_as_float(w.y << 16);
      v[3] = __uint_as_float(w.y & 0xFFFF0000u);
    }
  }
}
template <int C>
__device__ __forceinline__ void st_vec(void* p, int64_t i, int dt, const float* v) {
  if (dt == DT_F32) {
    float* q = static_cast<float*>(p) + i;
#pragma unroll
    for (int c = 0; c < C; c += 4) st16(q + c, pack(v + c, float{}));
  } else {
    uint16_t* q = static_cast<uint16_t*>(p) + i;
    if constexpr (C == 8)
      st16(q, pack(v, bf16_t{}));
    else
      *reinterpret_cast<uint2*>(q) = make_uint2(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]));
  }
}

// C neighbouring sums of row m from column n on: bias, pre-activation out,
// activation, residual, result.  g.vec: every row of y, pre and r starts on 16 bytes.
template <int C>
__device__ __forceinline__ void finish(const Linear& g, int64_t m, int n, float* v) {
  if (n >= g.N) return;
  const bool whole = g.vec && n + C <= g.N;
  const int cnt = min(C, g.N - n);
  if (g.bias) {
#pragma unroll
    for (int c = 0; c < C; ++c) v[c] += ld_elem(g.bias, min(n + c, g.N - 1), g.bias_dt);
  }
  if (g.pre) {
    if (whole) {
      st_vec<C>(g.pre, m * g.ldp + n, DT_BF16, v);
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
  if (g.res) {
    if (whole) {
      float r[C];
      ld_vec<C>(g.res, m * g.ldr + n, g.out_dt, r);
#pragma unroll
      for (int c = 0; c < C; ++c) v[c] += r[c];
    } else {
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (c < cnt) v[c] += ld_elem(g.res, m * g.ldr + n + c, g.out_dt);
    }
  }
  if (whole) {
    st_vec<C>(g.y, m * g.ldy + n, g.out_dt, v);
  } else {
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (c < cnt) st_elem(g.y, m * g.ldy + n + c, g.out_dt, v[c]);
  }
}

// ---------------------------------------------------------------- tiles
// One tile of C over one share of K; with several shares the fp32 sums go to
// g.part [shares][M][ldpart] and finish_kernel adds them.
template <class TL, bool AK, bool BK>
__global__ __launch_bounds__(TL::THREADS) void linear_tile_kernel(Linear g) {
  constexpr int kLds = TL::MAIN_LDS > buf::Epilogue<TL>::kBytes ? TL::MAIN_LDS : buf::Epilogue<TL>::kBytes;
  __shared__ __attribute__((aligned(1024))) char lds[kLds];
  const int t = xcd_order(blockIdx.x, gridDim.x);
  const int tiles = g.tiles_m * g.tiles_n;
  const int share = t / tiles;
  if (share >= g.shares) return;
  int mt, nt;
  dense_tile(t - share * tiles, g.tiles_m, g.tiles_n, mt, nt);
  const int m0 = mt * TL::BM, n0 = nt * TL::BN;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int k0 = share * g.share_k, kn = min(g.share_k, g.K - k0);
  buf::ARows<TL, AK> a;
  buf::BRows<TL, BK> b;
  a.init(static_cast<const uint16_t*>(g.x) + (AK ? k0 * g.ldx : k0), m0, (int)g.M, g.ldx, kn, wave, lane);
  b.init(static_cast<const uint16_t*>(g.w) + (BK ? k0 * g.ldw : k0), n0, g.N, g.ldw, kn, wave, lane);
  Acc<TL> acc;
  acc.zero();
  buf::mainloop<TL, AK, BK, false>(a, b, (kn + 63) / 64, lds, acc);
  const int rows = min((int)g.M - m0, TL::BM);
  if (g.shares > 1) {
    float* part = g.part + (int64_t)share * g.M * g.ldpart;
    buf::Epilogue<TL>::run(acc, lds, rows, [&](int r, int c, float* v) {
      if (n0 + c < g.N) st_vec<8>(part, (int64_t)(m0 + r) * g.ldpart + n0 + c, DT_F32, v);
    });
  } else {
    buf::Epilogue<TL>::run(acc, lds, rows, [&](int r, int c, float* v) { finish<8>(g, m0 + r, n0 + c, v); });
  }
}

// Sums of the shares, in their order, then the epilogue: 8 columns a thread.
__global__ __launch_bounds__(256) void linear_finish_kernel(Linear g) {
  const int64_t chunks = g.ldpart / 8;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= g.M * chunks) return;
  const int64_t m = i / chunks;
  const int n = (int)(i - m * chunks) * 8;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < g.shares; ++s) {
    float u[8];
    ld_vec<8>(g.part, ((int64_t)s * g.M + m) * g.ldpart + n, DT_F32, u);
#pragma unroll
    for (int c = 0; c < 8; ++c) v[c] += u[c];
  }
  finish<8>(g, m, n, v);
}

// ------------------------------------------------------------- few rows
constexpr int kSkinnyWaves = 4;
constexpr int kSkinnyRows = 64;

typedef u32x4_t u32x4_any_t __attribute__((aligned(2)));
// 16 bytes at any even address
__device__ __forceinline__ uint4 ld16_any(const uint16_t* p) {
  const u32x4_t v = *reinterpret_cast<const u32x4_any_t*>(p);
  return make_uint4(v.x, v.y, v.z, v.w);
}
// 8 values from k on, zeros from K on
__device__ __forceinline__ uint4 ld8_until(const uint16_t* row, int k, int K) {
  if (k + 8 <= K) return ld16_any(row + k);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = k + 2 * i < K ? row[k + 2 * i] : 0, hi = k + 2 * i + 1 < K ? row[k + 2 * i + 1] : 0;
    w[i] = lo | hi << 16;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// MB blocks of 16 rows of x by 16 rows of W.  The weights are the first
// operand, so a lane ends with 4 neighbouring columns of row lane & 15.
template <int MB>
__global__ __launch_bounds__(64 * kSkinnyWaves) void linear_skinny_kernel(Linear g) {
  __shared__ f32x4_t part[kSkinnyWaves][MB][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n0 = blockIdx.x * 16;
  const int at = (lane >> 4) * 8;
  const uint16_t* w = static_cast<const uint16_t*>(g.w) + (int64_t)min(n0 + (lane & 15), g.N - 1) * g.ldw;
  const uint16_t* x[MB];
#pragma unroll
  for (int b = 0; b < MB; ++b) {
    const int64_t m = b * 16 + (lane & 15);
    x[b] = static_cast<const uint16_t*>(g.x) + (m < g.M ? m : g.M - 1) * g.ldx;
  }
  f32x4_t acc[MB];
#pragma unroll
  for (int b = 0; b < MB; ++b) acc[b] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  auto step = [&](const uint4& a, const uint4& v, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, v), c,
                                                   0, 0, 0);
  };
  const int whole = g.K & ~127;
#pragma unroll 2
  for (int k = wave * 128; k < whole; k += kSkinnyWaves * 128) {
    uint4 a[4], v[MB][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = ld16_any(w + k + 32 * i + at);
#pragma unroll
    for (int b = 0; b < MB; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) v[b][i] = ld16_any(x[b] + k + 32 * i + at);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int b = 0; b < MB; ++b) acc[b] = step(a[i], v[b][i], acc[b]);
  }
  // fewer than 128 values of K are left: a block of 32 a wavefront
  {
    const int k = whole + wave * 32;
    if (k < g.K) {
      const uint4 a = ld8_until(w, k + at, g.K);
#pragma unroll
      for (int b = 0; b < MB; ++b) acc[b] = step(a, ld8_until(x[b], k + at, g.K), acc[b]);
    }
  }
#pragma unroll
  for (int b = 0; b < MB; ++b) part[wave][b][lane] = acc[b];
  __syncthreads();
  for (int b = wave; b < MB; b += kSkinnyWaves) {
    f32x4_t s = part[0][b][lane];
#pragma unroll
    for (int j = 1; j < kSkinnyWaves; ++j) s += part[j][b][lane];
    const int m = b * 16 + (lane & 15);
    float v[4] = {s[0], s[1], s[2], s[3]};
    if (m < g.M) finish<4>(g, m, n0 + (lane >> 4) * 4, v);
  }
}
static_assert(kSkinnyWaves * 32 == 128, "the rest of K is one block of 32 a wavefront");

// -------------------------------------------------------- copies, slopes
// Rows [rows][cols] into rows of ldd (a multiple of 8), zeros past cols.
__global__ __launch_bounds__(256) void pack_rows_kernel(const uint16_t* __restrict__ src, int64_t rows, int cols,
                                                        int64_t lds, uint16_t* __restrict__ dst, int64_t ldd) {
  const int64_t chunks = ldd / 8;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= rows * chunks) return;
  const int64_t r = i / chunks;
  const int c = (int)(i - r * chunks) * 8;
  st16(dst + r * ldd + c, ld8_until(src + r * lds, c, cols));
}

// d = dy act'(pre) as bf16 rows of ldd (zeros past N), and sums of d (before
// its rounding) over the rows of each block of kSlopeRows: part [blocks][N].
constexpr int kSlopeRows = 64;
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
  int vec;         // rows of dy and pre start on 16 bytes
};
// 256 threads: 16 chunks of 8 columns x 16 row lanes
__global__ __launch_bounds__(256) void slope_kernel(Slope p) {
  __shared__ float red[16][16 * 8 + 4];
  const int cx = threadIdx.x & 15, ry = threadIdx.x >> 4;
  const int n = (blockIdx.x * 16 + cx) * 8;
  const int64_t r0 = (int64_t)blockIdx.y * kSlopeRows;
  float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  const bool whole = p.vec && n + 8 <= p.N;
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

// db[n] = sum of part[.][n], in order: 64 columns x 4 interleaved row lanes.
__global__ __launch_bounds__(256) void bias_grad_kernel(const float* __restrict__ part, int64_t blocks, int N,
                                                        float* __restrict__ db) {
  __shared__ float red[4][64];
  const int c = threadIdx.x & 63, r = threadIdx.x >> 6;
  const int n = blockIdx.x * 64 + c;
  float s = 0.0f;
  if (n < N)
    for (int64_t b = r; b < blocks; b += 4) s += part[b * N + n];
  red[r][c] = s;
  __syncthreads();
  if (r == 0 && n < N) db[n] = (red[0][c] + red[1][c]) + (red[2][c] + red[3][c]);
}

unsigned grid8(int64_t n) { return (unsigned)((n + 7) & ~int64_t(7)); }

template <class TL, bool AK, bool BK>
hipError_t launch_tiles(const Linear& g, hipStream_t s) {
  linear_tile_kernel<TL, AK, BK><<<grid8((int64_t)g.tiles_m * g.tiles_n * g.shares), TL::THREADS, 0, s>>>(g);
  return hipGetLastError();
}

}  // namespace

bool linear_skinny(int64_t M) { return M <= kSkinnyRows; }

// Tile and shares of K.  A big tile keeps a CU busy by itself, two small ones
// share one; the K of few tiles is shared so that every CU has work, with at
// least 4 K tiles a share.
LinearPlan linear_plan(int64_t M, int64_t N, int64_t K) {
  LinearPlan p{};
  const int64_t big = cdiv64(M, 256) * cdiv64(N, 256), small = cdiv64(M, 128) * cdiv64(N, 128);
  p.big = big >= 192;
  p.shares = 1;
  if (!p.big) {
    const int64_t kt = cdiv64(K, 64);
    int64_t want = 512 / small;
    if (want > kt / 4) want = kt / 4;
    if (want > 1) p.shares = (int)want;
  }
  p.share_k = (int)(cdiv64(cdiv64(K, 64), p.shares) * 64);
  p.shares = (int)cdiv64(K > 0 ? K : 1, p.share_k > 0 ? p.share_k : 1);
  if (p.share_k < 1) p.share_k = 64;
  p.part_bytes = p.shares > 1 ? (int64_t)p.shares * M * ((N + 7) & ~int64_t(7)) * 4 : 0;
  return p;
}

hipError_t launch_linear_tiles(const Linear& in, bool a_kmajor, bool b_kmajor, hipStream_t s) {
  if (in.M <= 0 || in.N <= 0) return hipSuccess;
  Linear g = in;
  const LinearPlan p = linear_plan(g.M, g.N, g.K);
  const int bm = p.big ? 256 : 128;
  g.tiles_m = (int)cdiv64(g.M, bm);
  g.tiles_n = (int)cdiv64(g.N, bm);
  g.shares = p.shares;
  g.share_k = p.share_k;
  g.ldpart = (g.N + 7) & ~int64_t(7);
  hipError_t e;
  if (p.big)
    e = a_kmajor ? launch_tiles<BigTile, true, true>(g, s)
        : b_kmajor ? launch_tiles<BigTile, false, true>(g, s) : launch_tiles<BigTile, false, false>(g, s);
  else
    e = a_kmajor ? launch_tiles<SmallTile, true, true>(g, s)
        : b_kmajor ? launch_tiles<SmallTile, false, true>(g, s) : launch_tiles<SmallTile, false, false>(g, s);
  if (e != hipSuccess || g.shares == 1) return e;
  linear_finish_kernel<<<(unsigned)cdiv64(g.M * (g.ldpart / 8), 256), 256, 0, s>>>(g);
  return hipGetLastError();
}

hipError_t launch_linear_skinny(const Linear& g, hipStream_t s) {
  if (g.M <= 0 || g.N <= 0) return hipSuccess;
  const dim3 grid((unsigned)cdiv64(g.N, 16));
  if (g.M <= 16)
    linear_skinny_kernel<1><<<grid, 64 * kSkinnyWaves, 0, s>>>(g);
  else if (g.M <= 32)
    linear_skinny_kernel<2><<<grid, 64 * kSkinnyWaves, 0, s>>>(g);
  else
    linear_skinny_kernel<4><<<grid, 64 * kSkinnyWaves, 0, s>>>(g);
  return hipGetLastError();
}

hipError_t launch_pack_rows(const void* src, int64_t rows, int cols, int64_t ld, void* dst, int64_t ldd,
                            hipStream_t s) {
  if (rows <= 0 || ldd <= 0) return hipSuccess;
  pack_rows_kernel<<<(unsigned)cdiv64(rows * (ldd / 8), 256), 256, 0, s>>>(
      static_cast<const uint16_t*>(src), rows, cols, ld, static_cast<uint16_t*>(dst), ldd);
  return hipGetLastError();
}

int64_t slope_blocks(int64_t M) { return cdiv64(M, kSlopeRows); }

hipError_t launch_slope(const void* dy, int64_t ldy, int dy_dt, const void* pre, int64_t ldp, int act, int64_t M,
                        int N, void* d, int64_t ldd, float* part, float* db, hipStream_t s) {
  if (N <= 0) return hipSuccess;
  auto on16 = [](const void* p, int64_t ld, int64_t size) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * size % 16 == 0;
  };
  if (M > 0) {
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
    p.vec = on16(dy, ldy, dy_dt == DT_F32 ? 4 : 2) && (act == ACT_NONE || on16(pre, ldp, 2));
    slope_kernel<<<dim3((unsigned)cdiv64(N, 128), (unsigned)slope_blocks(M)), 256, 0, s>>>(p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (db) bias_grad_kernel<<<(unsigned)cdiv64(N, 64), 256, 0, s>>>(part, M > 0 ? slope_blocks(M) : 0, N, db);
  return hipGetLastError();
}

}  // namespace moe
