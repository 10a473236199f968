// Newton-Schulz iteration on batches of matrices: X = G / (|G| + eps), then
// steps of A = X X^T, B = b A + c A A, X = a X + B X, which moves every
// singular value s by a s + b s^3 + c s^5.  X is m x n with m <= n (G
// transposed where it is taller than wide).
//
// The three products run on fp16 matrix instructions (gemm_buf.h) with fp32
// sums.  X itself stays in fp32, and the diagonals of A and B, where their
// weight is, in fp32 as well; the products see X, and A and B off their
// diagonals, rounded to fp16 (11 bits).  Then the rounding touches neither the
// a X + diag(B) X that carries small singular values nor the cancellation
// between a and diag(B), and the result is off by 3e-4 to 1.5e-3 of its norm
// over five steps of the usual coefficients, whatever the spectrum, less than
// its final rounding to bf16.  (fp16 X alone: 1.2e-3 to 0.12, for a matrix of
// nearly rank one; bf16 products: 1.4e-3 to 2e-2 with X in fp32.)  Matrices
// with a side below kSplitSide, where one direction of a few is a large part of
// A's rows (up to 1e-2), also take what X's rounding leaves, as a second fp16
// number, in both products with X: 1e-3 at most.
// fp16's range is no matter: the host bounds the singular values of every
// step and scales X, A and B by powers of two to fill it.
//
// A and B are symmetric: only tiles on and below the diagonal are computed,
// and written to both places.
#include "common.h"
#include "gemm_buf.h"
#include "kernels.h"

namespace moe {
namespace {

using core::Acc;
using core::acc_col;
using core::acc_row;
using core::xcd_order;

using BigTile = core::Tile<256, 256, 4, 2, 64, 2, 3>;
using SmallTile = core::Tile<128, 128, 2, 2, 64, 2, 2>;

int64_t cdiv64(int64_t a, int64_t b) { return (a + b - 1) / b; }

__device__ __forceinline__ uint32_t f16_pair(float lo, float hi) {
  typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, f16x2_t{(_Float16)lo, (_Float16)hi});
}
__device__ __forceinline__ float f16_at(uint32_t pair, int hi) {
  return (float)__builtin_bit_cast(_Float16, (uint16_t)(hi ? pair >> 16 : pair & 0xFFFF));
}

__device__ __forceinline__ float load_in(const void* p, int64_t i, int dt) {
  return dt == DT_F32 ? static_cast<const float*>(p)[i] : bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
}

// Sum over a workgroup of 256 threads, in every thread, in a fixed order.
__device__ __forceinline__ double block_sum(double v, double* part) {
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  return (part[0] + part[1]) + (part[2] + part[3]);
}

// part[matrix][chunk] = sum of squares of kNormRows rows' share of G, in fp64
// (squares of small or large gradients leave fp32's range).
constexpr int kNormChunks = 64;
__global__ __launch_bounds__(256) void ortho_norm_kernel(Ortho p) {
  __shared__ double part[4];
  const int64_t b = blockIdx.x / kNormChunks;
  const int chunk = blockIdx.x % kNormChunks;
  const int64_t base = (p.b0 + b) * p.stride_g;
  const int64_t total = (int64_t)p.M * p.N;
  const int64_t per = (total + kNormChunks - 1) / kNormChunks;
  const int64_t first = chunk * per, end = first + per < total ? first + per : total;
  double s = 0.0;
  int64_t i = first + threadIdx.x;
  int64_t r = i / p.N;
  int c = (int)(i - r * p.N);
  for (; i < end; i += 256) {
    const double v = load_in(p.g, base + r * p.ldg + c, p.dt);
    s = fma(v, v, s);
    c += 256;
    while (c >= p.N) {
      c -= p.N;
      ++r;
    }
  }
  s = block_sum(s, part);
  if (threadIdx.x == 0) p.norm[b * kNormChunks + chunk] = s;
}

// X = G / (|G| + eps) in fp32 and scaled fp16, 64 x 64 values a workgroup,
// zeros in columns n .. np.
__global__ __launch_bounds__(256) void ortho_init_kernel(Ortho p) {
  __shared__ float tile[64][65];
  const int cols = p.np / 64, tiles = cols * ((p.m + 63) / 64);
  const int64_t b = blockIdx.x / tiles;
  const int t = blockIdx.x % tiles;
  const int r0 = t / cols * 64, c0 = t % cols * 64;
  double ss = 0.0;
  for (int i = 0; i < kNormChunks; ++i) ss += p.norm[b * kNormChunks + i];
  const double den = sqrt(ss) + (double)p.eps;
  const double inv = den > 0.0 ? 1.0 / den : 0.0;
  const int64_t gbase = (p.b0 + b) * p.stride_g;
  const int lx = threadIdx.x & 63, ly = threadIdx.x >> 6;
  // read along G's rows
  for (int i = ly; i < 64; i += 4) {
    const int x_r = p.tall ? r0 + lx : r0 + i, x_c = p.tall ? c0 + i : c0 + lx;  // place in X
    float v = 0.0f;
    if (x_r < p.m && x_c < p.n)
      v = (float)((double)load_in(p.g, gbase + (int64_t)(p.tall ? x_c : x_r) * p.ldg + (p.tall ? x_r : x_c), p.dt) * inv);
    if (p.tall)
      tile[lx][i] = v;
    else
      tile[i][lx] = v;
  }
  __syncthreads();
  float* x32 = p.x32 + b * (int64_t)p.m * p.np;
  uint16_t* x16 = p.x16[0] + b * (int64_t)p.m * p.np;
  for (int i = ly; i < 64; i += 4) {
    const int r = r0 + i;
    if (r >= p.m) break;
    const float v = tile[i][lx];
    const int64_t at = (int64_t)r * p.np + c0 + lx;
    const _Float16 h = (_Float16)(v * p.sx);
    x32[at] = v;
    x16[at] = __builtin_bit_cast(uint16_t, h);
    if (p.split) p.lo16[0][b * (int64_t)p.m * p.np + at] = __builtin_bit_cast(uint16_t, (_Float16)(v * p.sx - (float)h));
  }
}

// kB false: A = X X^T, of X in one fp16 number or two (kSplit: h h^T + h l^T +
// l h^T);  true: B = b A + c A A, from A off its diagonal (R) and its diagonal
// d: A A = R R + (d_i + d_j) R_ij + [i = j] d_i^2.
template <class TL, bool kB, bool kSplit>
__global__ __launch_bounds__(TL::THREADS) void ortho_gram_kernel(Ortho p) {
  static_assert(TL::BM == TL::BN, "square tiles of a symmetric product");
  constexpr int kLds = TL::MAIN_LDS > buf::Epilogue<TL>::kBytes ? TL::MAIN_LDS : buf::Epilogue<TL>::kBytes;
  __shared__ __attribute__((aligned(1024))) char lds[kLds];
  const int t = xcd_order(blockIdx.x, gridDim.x);
  const int b = t / p.gram_tiles;
  if (b >= p.count) return;
  // tile (mt, nt), nt <= mt, number mt (mt + 1) / 2 + nt
  const int q = t - b * p.gram_tiles;
  int mt = __builtin_amdgcn_readfirstlane((int)((sqrtf(8.0f * q + 1.0f) - 1.0f) * 0.5f));
  while ((mt + 1) * (mt + 2) / 2 <= q) ++mt;
  while (mt * (mt + 1) / 2 > q) --mt;
  const int nt = q - mt * (mt + 1) / 2;
  const int m0 = mt * TL::BM, n0 = nt * TL::BN;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave / TL::WGN, wn = wave % TL::WGN;
  const int K = kB ? p.mp : p.np;
  const int64_t at = (int64_t)b * p.m * K;
  const uint16_t* X = (kB ? p.a16 : p.x16[p.cur]) + at;
  Acc<TL> acc;
  acc.zero();
  for (int pass = 0; pass < (kSplit && !kB ? 3 : 1); ++pass) {
    const uint16_t* lo = kSplit && !kB ? p.lo16[p.cur] + at : X;
    buf::ARows<TL, false> a;
    buf::BRows<TL, false> w;
    a.init(pass == 2 ? lo : X, m0, p.m, K, K, wave, lane);
    w.init(pass == 1 ? lo : X, n0, p.m, K, K, wave, lane);
    buf::mainloop<TL, false, false, true>(a, w, K / 64, lds, acc);
  }
  const float* dA = p.da + (int64_t)b * p.m;
  float* dOut = (kB ? p.db : p.da) + (int64_t)b * p.m;
  uint16_t* C = (kB ? p.b16 : p.a16) + (int64_t)b * p.m * p.mp;
  // a lane holds rows row .. row + 3 of one column: the transposed place,
  // 4 neighbouring values
#pragma unroll
  for (int ni = 0; ni < TL::NI; ++ni) {
    const int col = n0 + acc_col<TL>(wn, ni, lane);
    const bool in_c = col < p.m;
    float dc = 0.0f;
    if constexpr (kB) dc = dA[min(col, p.m - 1)];
#pragma unroll
    for (int mi = 0; mi < TL::MI; ++mi) {
      const int row = m0 + acc_row<TL>(wm, mi, lane, 0);  // a multiple of 4, as mp is
      f32x4_t& v = acc.v[mi][ni];
      if constexpr (kB) {
        uint2 rw = make_uint2(0, 0);
        f32x4_t dr = {0.f, 0.f, 0.f, 0.f};
        if (in_c && row < p.mp) {
          rw = *reinterpret_cast<const uint2*>(p.a16 + ((int64_t)b * p.m + col) * p.mp + row);
#pragma unroll
          for (int r = 0; r < 4; ++r) dr[r] = dA[min(row + r, p.m - 1)];
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float R = f16_at(r < 2 ? rw.x : rw.y, r & 1) * p.inv_sa;
          const bool diag = row + r == col;
          const float A = diag ? dc : R;
          const float A2 = v[r] * (p.inv_sa * p.inv_sa) + (diag ? dc * dc : (dc + dr[r]) * R);
          v[r] = p.cb * A + p.cc * A2;
        }
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] *= p.inv_sx * p.inv_sx;
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const bool diag = row + r == col;
        if (diag && in_c) dOut[col] = v[r];
        v[r] = diag ? 0.0f : v[r] * (kB ? p.sb : p.sa);
      }
      if (in_c && row < p.mp)
        *reinterpret_cast<uint2*>(C + (int64_t)col * p.mp + row) = make_uint2(f16_pair(v[0], v[1]), f16_pair(v[2], v[3]));
    }
  }
  if (mt == nt) return;
  // below the diagonal: rows of the tile itself (its columns are all below m)
  buf::Epilogue<TL>::run(acc, lds, min(TL::BM, p.m - m0), [&](int r, int c, float* v) {
    st16(C + (int64_t)(m0 + r) * p.mp + n0 + c,
         make_uint4(f16_pair(v[0], v[1]), f16_pair(v[2], v[3]), f16_pair(v[4], v[5]), f16_pair(v[6], v[7])));
  });
}

// X = a X + B X = (a + d_i) X_i + (R X)_i, R being B off its diagonal d.
// kLast 0: into X; 1: the result, as G lies; 2: the result, transposed.
template <class TL, int kLast, bool kSplit>
__global__ __launch_bounds__(TL::THREADS) void ortho_update_kernel(Ortho p) {
  constexpr int kLds = TL::MAIN_LDS > buf::Epilogue<TL>::kBytes ? TL::MAIN_LDS : buf::Epilogue<TL>::kBytes;
  __shared__ __attribute__((aligned(1024))) char lds[kLds];
  const int t = xcd_order(blockIdx.x, gridDim.x);
  const int tiles = p.tiles_m * p.tiles_n;
  const int b = t / tiles;
  if (b >= p.count) return;
  int mt, nt;
  core::dense_tile(t - b * tiles, p.tiles_m, p.tiles_n, mt, nt);
  const int m0 = mt * TL::BM, n0 = nt * TL::BN;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t xo = (int64_t)b * p.m * p.np;
  Acc<TL> acc;
  acc.zero();
  for (int pass = 0; pass < (kSplit ? 2 : 1); ++pass) {
    buf::ARows<TL, false> a;
    buf::BRows<TL, true> w;
    a.init(p.b16 + (int64_t)b * p.m * p.mp, m0, p.m, p.mp, p.mp, wave, lane);
    w.init((pass == 1 ? p.lo16[p.cur] : p.x16[p.cur]) + xo, n0, p.np, p.np, p.m, wave, lane);
    buf::mainloop<TL, false, true, true>(a, w, p.mp / 64, lds, acc);
  }
  const float* dB = p.db + (int64_t)b * p.m;
  const float* x32 = p.x32 + xo;
  const float inv = p.inv_sb * p.inv_sx;
  if constexpr (kLast == 2) {
    // a lane holds 4 neighbouring values of a row of the transposed result
    const int wm = wave / TL::WGN, wn = wave % TL::WGN;
    uint16_t* out = p.out + (p.b0 + b) * p.stride_o;
#pragma unroll
    for (int mi = 0; mi < TL::MI; ++mi) {
      const int row = m0 + acc_row<TL>(wm, mi, lane, 0);
      float d[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) d[r] = p.ca + dB[min(row + r, p.m - 1)];
#pragma unroll
      for (int ni = 0; ni < TL::NI; ++ni) {
        const int col = n0 + acc_col<TL>(wn, ni, lane);
        if (col >= p.n || row >= p.m) continue;
        float v[4];
#pragma unroll
        for (int r = 0; r < 4; ++r)
          v[r] = p.scale * fmaf(d[r], x32[(int64_t)min(row + r, p.m - 1) * p.np + col], acc.v[mi][ni][r] * inv);
        uint16_t* o = out + (int64_t)col * p.ldo + row;
        if (p.vec_out && row + 4 <= p.m) {
          *reinterpret_cast<uint2*>(o) = make_uint2(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]));
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (row + r < p.m) o[r] = f32_to_bf16(v[r]);
        }
      }
    }
  } else {
    buf::Epilogue<TL>::run(acc, lds, min(TL::BM, p.m - m0), [&](int r, int c, float* v) {
      const int row = m0 + r, col = n0 + c;
      if (col >= p.np) return;
      const int64_t at = (int64_t)row * p.np + col;
      const float d = p.ca + dB[row];
      float x[8];
      unpack(ld16(x32 + at), x, float{});
      unpack(ld16(x32 + at + 4), x + 4, float{});
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = fmaf(d, x[i], v[i] * inv);
      if constexpr (kLast == 0) {
        st16(p.x32 + xo + at, pack(x, float{}));
        st16(p.x32 + xo + at + 4, pack(x + 4, float{}));
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= p.sx_next;
        const uint4 h = make_uint4(f16_pair(x[0], x[1]), f16_pair(x[2], x[3]), f16_pair(x[4], x[5]), f16_pair(x[6], x[7]));
        st16(p.x16[1 - p.cur] + xo + at, h);
        if constexpr (kSplit) {
          const uint32_t w4[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] -= f16_at(w4[i / 2], i & 1);
          st16(p.lo16[1 - p.cur] + xo + at,
               make_uint4(f16_pair(x[0], x[1]), f16_pair(x[2], x[3]), f16_pair(x[4], x[5]), f16_pair(x[6], x[7])));
        }
      } else {
        if (col >= p.n) return;
        uint16_t* o = p.out + (p.b0 + b) * p.stride_o + (int64_t)row * p.ldo + col;
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= p.scale;
        if (p.vec_out && col + 8 <= p.n) {
          st16(o, pack(x, bf16_t{}));
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (col + i < p.n) o[i] = f32_to_bf16(x[i]);
        }
      }
    });
  }
}

unsigned grid8(int64_t n) { return (unsigned)((n + 7) & ~int64_t(7)); }

template <class TL, bool kSplit>
hipError_t run_step(const Ortho& p, bool last, hipStream_t s) {
  const unsigned gram = grid8((int64_t)p.gram_tiles * p.count), all = grid8((int64_t)p.tiles_m * p.tiles_n * p.count);
  ortho_gram_kernel<TL, false, kSplit><<<gram, TL::THREADS, 0, s>>>(p);
  ortho_gram_kernel<TL, true, false><<<gram, TL::THREADS, 0, s>>>(p);
  if (!last)
    ortho_update_kernel<TL, 0, kSplit><<<all, TL::THREADS, 0, s>>>(p);
  else if (!p.tall)
    ortho_update_kernel<TL, 1, kSplit><<<all, TL::THREADS, 0, s>>>(p);
  else
    ortho_update_kernel<TL, 2, kSplit><<<all, TL::THREADS, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace

int ortho_norm_chunks() { return kNormChunks; }

constexpr int kSplitSide = 256;
bool ortho_split(int64_t m) { return m < kSplitSide; }

// Matrices at a time: enough tiles of the update for several rounds of the
// chip, so that more would only need more workspace.
int64_t ortho_group(int64_t batch, int64_t m, int64_t n) {
  const int64_t tiles = cdiv64(m, 128) * cdiv64(n, 128);
  int64_t g = 8192 / tiles;
  if (g < 1) g = 1;
  return batch < g ? batch : g;
}

hipError_t launch_orthogonalize(const Ortho& in, const OrthoStep* step, int steps, int64_t batch, int64_t group,
                                hipStream_t s) {
  for (int64_t b0 = 0; b0 < batch; b0 += group) {
    Ortho p = in;
    p.b0 = b0;
    p.count = (int)(batch - b0 < group ? batch - b0 : group);
    p.sx = step[0].sx;
    p.split = ortho_split(p.m);
    ortho_norm_kernel<<<(unsigned)(p.count * kNormChunks), 256, 0, s>>>(p);
    ortho_init_kernel<<<(unsigned)((int64_t)p.count * (p.np / 64) * cdiv64(p.m, 64)), 256, 0, s>>>(p);
    const bool big = !p.split && (int64_t)cdiv64(p.m, 256) * cdiv64(p.m, 256) * p.count >= 256;
    const int tile = big ? 256 : 128;
    const int64_t tm = cdiv64(p.m, tile);
    p.gram_tiles = (int)(tm * (tm + 1) / 2);
    p.tiles_m = (int)tm;
    p.tiles_n = (int)cdiv64(p.np, tile);
    for (int k = 0; k < steps; ++k) {
      const OrthoStep& c = step[k];
      p.cur = k & 1;
      p.ca = c.a;
      p.cb = c.b;
      p.cc = c.c;
      p.sx = c.sx;
      p.inv_sx = 1.0f / c.sx;
      p.sa = c.sa;
      p.inv_sa = 1.0f / c.sa;
      p.sb = c.sb;
      p.inv_sb = 1.0f / c.sb;
      p.sx_next = k + 1 < steps ? step[k + 1].sx : 1.0f;
      const bool last = k + 1 == steps;
      const hipError_t e = big ? run_step<BigTile, false>(p, last, s)
                           : p.split ? run_step<SmallTile, true>(p, last, s) : run_step<SmallTile, false>(p, last, s);
      if (e != hipSuccess) return e;
    }
  }
  return hipGetLastError();
}

}  // namespace moe
