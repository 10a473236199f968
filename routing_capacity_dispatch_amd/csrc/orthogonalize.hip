// Newton-Schulz iteration on batches of matrices: X = G / (|G| + eps), then
// steps of A = X X^T, B = b A + c A A, X = a X + B X, which moves every
// singular value s by a s + b s^3 + c s^5.  X is m x n with m <= n (G
// transposed where it is taller than wide).
//
// The three products run on fp16 matrix instructions (gemm_buf.h) with fp32
// sums.  X itself is held in two fp16 numbers, h + l (22 bits), and the diagonals
// of A and B, where their weight is, in fp32; the products see h, and A and B off
// their diagonals, rounded to fp16 (11 bits).
//
// An update is a (h + l) + B h: the polynomial of h and a times l.  h = X - l has
// singular values of l's size where X has none; they grow by a as l's own do, and
// the two cancel.  A part of B times a part of l only, as its diagonal (which would
// spare a full-rank X the rounding: there B is mostly diagonal), breaks that, and
// what is left grows by `a` in every later step: up to 4e-2 of the result's norm
// where a few rows carry the matrix.  So l's diagonal term has the weight 1 / (the
// later steps' gains), which keeps what it leaves at the last step's size.  The
// result is off by 2e-4 to 2e-3 of its norm over five steps of the usual
// coefficients, up to 3.5e-3 where a few rows or values of one magnitude carry the
// matrix and 5e-3 where a handful of values do; its final rounding to bf16 is
// 1.7e-3.  (h alone: 1.2e-3 to 0.12, for a matrix of nearly rank one; bf16 products:
// 1.4e-3 to 2e-2.)  Matrices with a side below kSplitSide, where one direction of a
// few is a large part of A's rows, take l as well in both products with X: 3.5e-3
// at most.  Larger ones would come to half of the above by that, for about twice
// the matrix instructions.
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
using SmallTile = core::Tile<128, 128, 4, 2, 64, 2, 2>;
using MidTile = core::Tile<128, 128, 4, 2, 64, 5>;
using DeepTile = core::Tile<64, 64, 2, 2, 64, 5>;

int64_t cdiv64(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int kNormChunks = 256;  // most shares of a matrix's norm

__device__ __forceinline__ uint32_t f16_pair(float lo, float hi) {
  typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, f16x2_t{(_Float16)lo, (_Float16)hi});
}
__device__ __forceinline__ float f16_at(uint32_t pair, int hi) {
  return (float)__builtin_bit_cast(_Float16, (uint16_t)(hi ? pair >> 16 : pair & 0xFFFF));
}

// 8 values of G from element i on, of which n (at least 1) are there; zeros after them
__device__ __forceinline__ void load_in(const void* p, int64_t i, int n, int dt, float* v) {
  if (n >= 8) {
    if (dt == DT_F32) {
      const uint16_t* q = reinterpret_cast<const uint16_t*>(static_cast<const float*>(p) + i);
      unpack(buf::ld16_any(q), v, float{});
      unpack(buf::ld16_any(q + 8), v + 4, float{});
    } else {
      unpack(buf::ld16_any(static_cast<const uint16_t*>(p) + i), v, bf16_t{});
    }
  } else {
#pragma unroll
    for (int c = 0; c < 8; ++c)
      v[c] = c >= n ? 0.0f
             : dt == DT_F32 ? static_cast<const float*>(p)[i + c] : bf16_to_f32(static_cast<const uint16_t*>(p)[i + c]);
  }
}

// Sum over a workgroup of 256 threads, in every thread, in a fixed order.
__device__ __forceinline__ double block_sum(double v, double* part) {
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  return (part[0] + part[1]) + (part[2] + part[3]);
}

// norm[matrix][chunk] = sum of squares of a share of G, in fp64 (squares of
// small or large gradients leave fp32's range).
__global__ __launch_bounds__(256) void ortho_norm_kernel(Ortho p) {
  __shared__ double part[4];
  const int64_t b = blockIdx.x / p.chunks;
  const int chunk = blockIdx.x % p.chunks;
  const int64_t base = (p.b0 + b) * p.stride_g;
  const uint32_t per_row = (p.N + 7) / 8;
  const uint32_t total = (uint32_t)p.M * per_row;  // at most 2^29
  const uint32_t per = (total + p.chunks - 1) / p.chunks;
  const uint32_t first = chunk * per, end = min(first + per, total);
  double s = 0.0;
#pragma unroll 4
  for (uint32_t u = first + threadIdx.x; u < end; u += 256) {
    const uint32_t r = u / per_row, c = (u - r * per_row) * 8;
    float v[8];
    load_in(p.g, base + (int64_t)r * p.ldg + c, p.N - (int)c, p.dt, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fma((double)v[i], (double)v[i], s);
  }
  s = block_sum(s, part);
  if (threadIdx.x == 0) p.norm[b * kNormChunks + chunk] = s;
}

// 8 neighbouring values of X (times its scale) as h and l.
__device__ __forceinline__ uint4 f16_pack(const float* v) {
  return make_uint4(f16_pair(v[0], v[1]), f16_pair(v[2], v[3]), f16_pair(v[4], v[5]), f16_pair(v[6], v[7]));
}
__device__ __forceinline__ void f16_unpack(const uint4& q, float* v) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = f16_at(w[i / 2], i & 1);
}
__device__ __forceinline__ void store_x(uint16_t* h, uint16_t* l, float* v) {
  const uint4 q = f16_pack(v);
  st16(h, q);
  float r[8];
  f16_unpack(q, r);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] -= r[i];
  st16(l, f16_pack(v));
}

// X = G / (|G| + eps), 64 x 64 values a workgroup, zeros in columns n .. np.
__global__ __launch_bounds__(256) void ortho_init_kernel(Ortho p) {
  __shared__ float tile[64][65];
  __shared__ double part[4];
  const int cols = p.np / 64, tiles = cols * ((p.m + 63) / 64);
  const int64_t b = blockIdx.x / tiles;
  const int t = blockIdx.x % tiles;
  const int r0 = t / cols * 64, c0 = t % cols * 64;
  const double ss = block_sum((int)threadIdx.x < p.chunks ? p.norm[b * kNormChunks + threadIdx.x] : 0.0, part);
  const double den = sqrt(ss) + (double)p.eps;
  const double scale = den > 0.0 ? 1.0 / den : 0.0;
  const int64_t gbase = (p.b0 + b) * p.stride_g;
  const int64_t xbase = b * (int64_t)p.m * p.np;
  float v[2][8];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = (threadIdx.x >> 3) + 32 * i, c = (threadIdx.x & 7) * 8;
    const int gr = (p.tall ? c0 : r0) + row, gc = (p.tall ? r0 : c0) + c;  // in G
    if (gr < p.M && gc < p.N) {
      load_in(p.g, gbase + (int64_t)gr * p.ldg + gc, p.N - gc, p.dt, v[i]);
#pragma unroll
      for (int q = 0; q < 8; ++q) v[i][q] = (float)((double)v[i][q] * scale);
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q) v[i][q] = 0.0f;
    }
    if (p.tall) {
#pragma unroll
      for (int q = 0; q < 8; ++q) tile[c + q][row] = v[i][q];
    }
  }
  if (p.tall) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int q = 0; q < 8; ++q) v[i][q] = tile[(threadIdx.x >> 3) + 32 * i][(threadIdx.x & 7) * 8 + q];
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = r0 + (threadIdx.x >> 3) + 32 * i;
    if (r >= p.m) break;
    const int64_t at = xbase + (int64_t)r * p.np + c0 + (threadIdx.x & 7) * 8;
#pragma unroll
    for (int q = 0; q < 8; ++q) v[i][q] *= p.sx;
    store_x(p.x16[0] + at, p.lo16[0] + at, v[i]);
  }
}

// acc += A B^T of fp16 operands by the tile's schedule
template <class TL, bool BK, class SA, class SB>
__device__ __forceinline__ void products(const SA& a, const SB& b, int K, char* lds, Acc<TL>& acc) {
  if constexpr (TL::NS == 2)
    buf::mainloop<TL, false, BK, true>(a, b, K / 64, lds, acc);
  else
    buf::mainloop_pipe<TL, false, BK, true>(a, b, K / 64, lds, acc);
}

// kB false: A = X X^T, of X in one fp16 number or two (kSplit: h h^T + h l^T +
// l h^T);  true: B = b A + c A A, from A off its diagonal (R) and its diagonal
// d: A A = R R + (d_i + d_j) R_ij + [i = j] d_i^2.
// t: number of the tile among those of all matrices.
template <class TL, bool kB, bool kSplit>
__device__ __forceinline__ void gram_tile(const Ortho& p, int t, char* lds) {
  static_assert(TL::BM == TL::BN, "square tiles of a symmetric product");
  const int b = t / p.gram_tiles;
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
    products<TL, false>(a, w, K, lds, acc);
  }
  const float* dA = p.da + (int64_t)b * p.m;
  float* dOut = (kB ? p.db : p.da) + (int64_t)b * p.m;
  uint16_t* C = (kB ? p.b16 : p.a16) + (int64_t)b * p.m * p.mp;
  // a lane holds rows row .. row + 3 of one column: the transposed place, 4
  // neighbouring values.  What it reads of A is fetched a column ahead, before
  // the stores that the compiler would not move loads across.
  float dr[TL::MI][4], dc[TL::NI];
  uint2 ahead[2][TL::MI];
  auto fetch = [&](int ni, uint2 (&to)[TL::MI]) {
    const int col = min(n0 + acc_col<TL>(wn, ni, lane), p.m - 1);
#pragma unroll
    for (int mi = 0; mi < TL::MI; ++mi) {
      const int row = min(m0 + acc_row<TL>(wm, mi, lane, 0), p.mp - 4);
      to[mi] = *reinterpret_cast<const uint2*>(p.a16 + ((int64_t)b * p.m + col) * p.mp + row);
    }
  };
  if constexpr (kB) {
#pragma unroll
    for (int mi = 0; mi < TL::MI; ++mi)
#pragma unroll
      for (int r = 0; r < 4; ++r) dr[mi][r] = dA[min(m0 + acc_row<TL>(wm, mi, lane, r), p.m - 1)];
#pragma unroll
    for (int ni = 0; ni < TL::NI; ++ni) dc[ni] = dA[min(n0 + acc_col<TL>(wn, ni, lane), p.m - 1)];
    fetch(0, ahead[0]);
  }
#pragma unroll
  for (int ni = 0; ni < TL::NI; ++ni) {
    if constexpr (kB) {
      if (ni + 1 < TL::NI) fetch(ni + 1, ahead[(ni + 1) & 1]);
    }
    const int col = n0 + acc_col<TL>(wn, ni, lane);
    const bool in_c = col < p.m;
#pragma unroll
    for (int mi = 0; mi < TL::MI; ++mi) {
      const int row = m0 + acc_row<TL>(wm, mi, lane, 0);  // a multiple of 4, as mp is
      f32x4_t& v = acc.v[mi][ni];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const bool diag = row + r == col;
        if constexpr (kB) {
          const uint2 rw = ahead[ni & 1][mi];
          const float R = f16_at(r < 2 ? rw.x : rw.y, r & 1) * p.inv_sa;
          const float A = diag ? dc[ni] : R;
          const float A2 = v[r] * (p.inv_sa * p.inv_sa) + (diag ? dc[ni] * dc[ni] : (dc[ni] + dr[mi][r]) * R);
          v[r] = p.cb * A + p.cc * A2;
        } else {
          v[r] *= p.inv_sx * p.inv_sx;
        }
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
    st16(C + (int64_t)(m0 + r) * p.mp + n0 + c, f16_pack(v));
  });
}

// X = a X + B X = (a + d_i) h_i + (a + w d_i) l_i + (R X)_i, R being B off its
// diagonal d; R X of h and l and w = 1 with kSplit, else of h and w as above.
// kLast 0: into X; 1: the result, as G lies; 2: the result, transposed.
template <class TL, int kLast, bool kSplit>
__device__ __forceinline__ void update_tile(const Ortho& p, int t, char* lds) {
  const int tiles = p.tiles_m * p.tiles_n;
  const int b = t / tiles;
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
    products<TL, true>(a, w, p.mp, lds, acc);
  }
  const float* dB = p.db + (int64_t)b * p.m;
  const uint16_t* xh = p.x16[p.cur] + xo;
  const uint16_t* xl = p.lo16[p.cur] + xo;
  const float inv = p.inv_sb * p.inv_sx;
  if constexpr (kLast == 2) {
    // a lane holds 4 neighbouring values of a row of the transposed result
    const int wm = wave / TL::WGN, wn = wave % TL::WGN;
    uint16_t* out = p.out + (p.b0 + b) * p.stride_o;
#pragma unroll
    for (int mi = 0; mi < TL::MI; ++mi) {
      const int row = m0 + acc_row<TL>(wm, mi, lane, 0);
      float dh[4], dl[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float d = dB[min(row + r, p.m - 1)];
        dh[r] = (p.ca + d) * p.inv_sx;
        dl[r] = fmaf(p.low, d, p.ca) * p.inv_sx;
      }
#pragma unroll
      for (int ni = 0; ni < TL::NI; ++ni) {
        const int col = n0 + acc_col<TL>(wn, ni, lane);
        if (col >= p.n || row >= p.m) continue;
        float v[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int64_t at = (int64_t)min(row + r, p.m - 1) * p.np + col;
          v[r] = p.scale * fmaf(dh[r], f16_at(xh[at], 0), fmaf(dl[r], f16_at(xl[at], 0), acc.v[mi][ni][r] * inv));
        }
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
    struct Ahead {
      uint4 h, l;
      float d;
    };
    buf::Epilogue<TL>::template run<Ahead>(
        acc, lds, min(TL::BM, p.m - m0),
        [&](int r, int c) {
          const int64_t at = (int64_t)(m0 + r) * p.np + min(n0 + c, p.np - 8);
          return Ahead{ld16(xh + at), ld16(xl + at), dB[m0 + r]};
        },
        [&](int r, int c, float* v, const Ahead& q) {
          const int row = m0 + r, col = n0 + c;
          if (col >= p.np) return;
          const float dh = (p.ca + q.d) * p.inv_sx, dl = fmaf(p.low, q.d, p.ca) * p.inv_sx;
          float x[8], y[8];
          f16_unpack(q.h, x);
          f16_unpack(q.l, y);
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = fmaf(dh, x[i], fmaf(dl, y[i], v[i] * inv));
          if constexpr (kLast == 0) {
            const int64_t at = xo + (int64_t)row * p.np + col;
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] *= p.sx_next;
            store_x(p.x16[1 - p.cur] + at, p.lo16[1 - p.cur] + at, x);
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

// One phase of a step on some matrices.
enum Phase : int { PHASE_A = 0, PHASE_B = 1, PHASE_X = 2, PHASE_OUT = 3, PHASE_OUT_T = 4 };

template <class TL, int kPhase, bool kSplit>
__device__ __forceinline__ void phase_tile(const Ortho& p, int t, char* lds) {
  if constexpr (kPhase == PHASE_A)
    gram_tile<TL, false, kSplit>(p, t, lds);
  else if constexpr (kPhase == PHASE_B)
    gram_tile<TL, true, kSplit>(p, t, lds);
  else
    update_tile<TL, kPhase - PHASE_X, kSplit>(p, t, lds);
}
__host__ __device__ inline int phase_tiles(const Ortho& p, int phase) {
  return (phase <= PHASE_B ? p.gram_tiles : p.tiles_m * p.tiles_n) * p.count;
}

template <class TL>
constexpr int tile_lds() {
  return TL::MAIN_LDS > buf::Epilogue<TL>::kBytes ? TL::MAIN_LDS : buf::Epilogue<TL>::kBytes;
}

template <class TL, int kPhase, bool kSplit>
__global__ __launch_bounds__(TL::THREADS) void ortho_phase_kernel(Ortho p) {
  __shared__ __attribute__((aligned(1024))) char lds[tile_lds<TL>()];
  const int t = xcd_order(blockIdx.x, gridDim.x);
  if (t < phase_tiles(p, kPhase)) phase_tile<TL, kPhase, kSplit>(p, t, lds);
}

unsigned grid8(int64_t n) { return (unsigned)((n + 7) & ~int64_t(7)); }

template <class TL>
void set_tiles(Ortho& p) {
  const int64_t t = cdiv64(p.m, TL::BM);
  p.gram_tiles = (int)(t * (t + 1) / 2);
  p.tiles_m = (int)t;
  p.tiles_n = (int)cdiv64(p.np, TL::BN);
}

template <class TL, int kPhase, bool kSplit>
void run_phase_of(const Ortho& p, hipStream_t s) {
  ortho_phase_kernel<TL, kPhase, kSplit><<<grid8(phase_tiles(p, kPhase)), TL::THREADS, 0, s>>>(p);
}
template <class TL>
void run_phase(Ortho p, int phase, hipStream_t s) {
  constexpr bool kSplit = TL::BM < 256;
  set_tiles<TL>(p);
  const bool split = kSplit && p.split;
  if (phase == PHASE_A)
    split ? run_phase_of<TL, PHASE_A, kSplit>(p, s) : run_phase_of<TL, PHASE_A, false>(p, s);
  else if (phase == PHASE_B)
    run_phase_of<TL, PHASE_B, false>(p, s);
  else if (phase == PHASE_X)
    split ? run_phase_of<TL, PHASE_X, kSplit>(p, s) : run_phase_of<TL, PHASE_X, false>(p, s);
  else if (phase == PHASE_OUT)
    split ? run_phase_of<TL, PHASE_OUT, kSplit>(p, s) : run_phase_of<TL, PHASE_OUT, false>(p, s);
  else
    split ? run_phase_of<TL, PHASE_OUT_T, kSplit>(p, s) : run_phase_of<TL, PHASE_OUT_T, false>(p, s);
}
void run_class(const Ortho& p, int cls, int phase, hipStream_t s) {
  if (cls == TILE_BIG)
    run_phase<BigTile>(p, phase, s);
  else if (cls == TILE_SMALL)
    run_phase<SmallTile>(p, phase, s);
  else if (cls == TILE_MID)
    run_phase<MidTile>(p, phase, s);
  else
    run_phase<DeepTile>(p, phase, s);
}

void set_step(Ortho& p, const OrthoStep* step, int steps, int k) {
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
  p.low = p.split ? 1.0f : c.low;
}

}  // namespace

int ortho_norm_chunks() { return kNormChunks; }

constexpr int kSplitSide = 256;
bool ortho_split(int64_t m) { return m < kSplitSide; }

namespace {
// Tile sizes as of other products (100 matrices of 300 x 300: 330 us, 571 with
// big tiles); the big one is not for two fp16 numbers of X.
int class_of(int64_t big, int64_t small, bool split) { return tile_class(split ? 0 : big, small); }
int gram_class(const Ortho& p) {
  auto tiles = [&](int64_t side) { return cdiv64(p.m, side) * (cdiv64(p.m, side) + 1) / 2 * p.count; };
  return class_of(tiles(256), tiles(128), p.split);
}
// (Up to 8 K tiles an update is mostly its epilogue, which two workgroups a CU hide:
// 64 x 512 x 512 441 us, 459 with big tiles; 64 x 1024 x 1024 2415 and 2370.)
int update_class(const Ortho& p) {
  auto tiles = [&](int64_t side) { return cdiv64(p.m, side) * cdiv64(p.np, side) * p.count; };
  return class_of(tiles(256), tiles(128), p.split || p.mp <= 512);
}
}  // namespace

OrthoForm ortho_form(const Ortho& in, int64_t count) {
  Ortho p = in;
  p.count = (int)count;
  p.split = ortho_split(p.m);
  return OrthoForm{gram_class(p), update_class(p), p.split};
}

// Matrices at a time: enough tiles of the update for several rounds of the
// chip, so that more would only need more workspace.
int64_t ortho_group(int64_t batch, int64_t m, int64_t n) {
  const int64_t tiles = cdiv64(m, 128) * cdiv64(n, 128);
  int64_t g = 8192 / tiles;
  if (g < 1) g = 1;
  return batch < g ? batch : g;
}

// One phase a launch.  Two of them in one, two halves of the matrices a phase
// apart, so that one's traffic would run under the other's matrix instructions, is
// slower mostly: its rounds of the chip are others, by chance fewer or more (12 x
// 2048 x 3584: 3951 us, 4378 one by one; 8 x 2048 x 4096 3035 and 3123; 32 x 1024 x
// 2048 2020 and 2040; but 7 x 2048 x 4096 2722 and 2559, 64 x 1024 x 1024 2445 and
// 2390, 58 x 1024 x 2560 4919 and 4228, 4 x 2048 x 8192 3406 and 2945).
hipError_t launch_orthogonalize(const Ortho& in, const OrthoStep* step, int steps, int64_t batch, int64_t group,
                                hipStream_t s) {
  for (int64_t b0 = 0; b0 < batch; b0 += group) {
    Ortho p = in;
    p.b0 = b0;
    p.count = (int)(batch - b0 < group ? batch - b0 : group);
    p.sx = step[0].sx;
    const OrthoForm form = ortho_form(p, p.count);
    p.split = form.split;
    p.chunks = p.count > 1024 / kNormChunks ? (p.count > 1024 / 16 ? 16 : 1024 / p.count) : kNormChunks;
    ortho_norm_kernel<<<(unsigned)(p.count * p.chunks), 256, 0, s>>>(p);
    ortho_init_kernel<<<(unsigned)((int64_t)p.count * (p.np / 64) * cdiv64(p.m, 64)), 256, 0, s>>>(p);
    const int out = p.tall ? PHASE_OUT_T : PHASE_OUT;
    for (int k = 0; k < steps; ++k) {
      set_step(p, step, steps, k);
      run_class(p, form.gram, PHASE_A, s);
      run_class(p, form.gram, PHASE_B, s);
      run_class(p, form.update, k + 1 < steps ? PHASE_X : out, s);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipGetLastError();
}

}  // namespace moe
