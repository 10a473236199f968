// Matrix core products C = A * B^T over operands of any size: the tiles,
// LDS layout and mid-tile barrier schedule of gemm_core.h, with operands read
// through buffer descriptors, so that rows past an operand's end and values
// past K come back as zeros and no operand needs padding in memory.
//
// An operand is row-major ([rows][K], K contiguous) or K-major ([K][rows],
// the transposed operand of a gradient's product).  Its base and rows are
// 16-byte aligned, and a row-major one has K a multiple of 8, so that a
// 16-byte chunk lies inside K or outside as a whole.  A descriptor's extent
// ends with the aligned 16 bytes that hold the operand's last value: nothing
// further is read.
#pragma once

#include "common.h"
#include "gemm_core.h"

namespace moe {
namespace buf {

using core::Acc;
using core::Frags;

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));

// One 16-byte-per-lane buffer -> LDS load: lane l's 16 bytes land at
// lds_wave_base + 16 l, zeros where its offset is outside the descriptor.
// (The wait state between a write of M0 and a load that reads it is the s_nop.)
__device__ __forceinline__ void lds_load16(i32x4_t rsrc, uint32_t voff, char* lds_wave_base) {
  const uint32_t l = __builtin_amdgcn_readfirstlane(
      static_cast<uint32_t>(reinterpret_cast<uintptr_t>((MOE_LDS char*)lds_wave_base)));
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(l), "v"(voff), "s"(rsrc)
               : "memory", "m0");
}

// Rows of one operand for one workgroup's tile: INS load instructions per
// wavefront and K tile.  kMajor: rows run along K.
template <class TL, int INS, int X, bool kMajor>
struct Rows {
  uint64_t base;      // first byte of the tile's rows (row-major) or columns (K-major) at K = 0
  int64_t extent;     // bytes from base to the end of the operand's last value the tile may read
  int64_t kstep;      // bytes between K tiles
  int K;
  uint32_t off[INS];  // per lane
  uint32_t col;       // row-major: first k of this lane's chunk in a K tile

  // ptr: the operand; r0: the tile's first row; rows: rows of the operand; ld in elements
  __device__ __forceinline__ void init(const void* ptr, int r0, int rows, int64_t ld, int K_, int wave, int lane) {
    K = K_;
    if constexpr (kMajor) {
      base = reinterpret_cast<uint64_t>(ptr) + (int64_t)r0 * 2;
      // up to the end of the 16 bytes that hold the last value (a load is all
      // or nothing per 4 bytes; the columns that follow it are never stored)
      extent = K > 0 ? (((int64_t)(K - 1) * ld + (rows - r0)) * 2 + 15) & ~int64_t(15) : 0;
      kstep = TL::BK * ld * 2;
      in_scalar();
      col = 0;
#pragma unroll
      for (int i = 0; i < INS; ++i) {
        const int k = core::kload_row<TL, X>(i, wave, lane);
        const int c = core::kload_col<X>(k, lane);
        // columns past the operand's own would reach into the next k-row
        off[i] = r0 + c / 2 < rows ? (uint32_t)(k * ld * 2) + c : kOut;
      }
    } else {
      base = reinterpret_cast<uint64_t>(ptr) + (int64_t)r0 * ld * 2;
      const int n = min(rows - r0, X);
      extent = (((int64_t)(n - 1) * ld + K) * 2 + 15) & ~int64_t(15);
      kstep = TL::RB;
      in_scalar();
      const int c = core::load_col<TL>(lane);
      col = c / 2;
#pragma unroll
      for (int i = 0; i < INS; ++i) {
        const int r = core::load_row<TL>(i, wave, lane);
        off[i] = r < n ? (uint32_t)(r * ld * 2) + c : kOut;
      }
    }
  }
  // base and extent in scalar registers, so that every descriptor is made there
  __device__ __forceinline__ void in_scalar() {
    base = reinterpret_cast<uint64_t>(core::uniform_ptr(reinterpret_cast<const char*>(base)));
    extent = (int64_t)reinterpret_cast<uint64_t>(core::uniform_ptr(reinterpret_cast<const char*>(extent)));
  }
  static constexpr uint32_t kOut = 0x80000000u;  // outside every descriptor
  // Descriptor of K tile j, and whether this lane's chunk lies inside K.
  struct TileAt {
    i32x4_t rsrc;
    bool in;
  };
  __device__ __forceinline__ TileAt tile(int j) const {
    const uint64_t b = base + (int64_t)j * kstep;
    // made of kernel arguments and block indices in scalar arithmetic (which
    // has no 64-bit comparison: the bytes left are clamped by their halves)
    const int64_t left = extent - (int64_t)j * kstep;
    const int hi = (int)(left >> 32), lo = (int)left;
    const int bytes = hi < 0 ? 0 : (hi > 0 || lo < 0) ? 0x7FFFFFFF : lo;
    TileAt t;
    t.rsrc = i32x4_t{(int)(uint32_t)b, (int)((uint32_t)(b >> 32) & 0xFFFFu), bytes, 0x00020000};
    t.in = kMajor || col + j * TL::BK < (uint32_t)K;
    return t;
  }
  __device__ __forceinline__ void load(const TileAt& t, int i, char* dst) const {
    lds_load16(t.rsrc, kMajor || t.in ? off[i] : kOut, dst);
  }
};

template <class TL, bool kAMajor>
using ARows = Rows<TL, TL::A_INS, TL::BM, kAMajor>;
template <class TL, bool kBMajor>
using BRows = Rows<TL, TL::B_INS, TL::BN, kBMajor>;

template <class TL, bool kHalf>
__device__ __forceinline__ void mfma_frags(const Frags<TL>& f, Acc<TL>& acc) {
  if constexpr (!kHalf) {
    core::mfma_frags<TL>(f, acc);
  } else {
#pragma unroll
    for (int mi = 0; mi < TL::MI; ++mi)
#pragma unroll
      for (int ni = 0; ni < TL::NI; ++ni)
        acc.v[mi][ni] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
            __builtin_bit_cast(f16x8_t, f.a[mi]), __builtin_bit_cast(f16x8_t, f.b[ni]), acc.v[mi][ni], 0, 0, 0);
  }
}

template <class TL, bool AK, bool BK>
__device__ __forceinline__ void interleave() {
  constexpr int NR = core::frag_reads<TL, AK, BK>(), NM = TL::MI * TL::NI;
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, NM / NR, 0);
    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
  }
  __builtin_amdgcn_sched_group_barrier(0x008, NM - (NM / NR) * NR, 0);
}

// acc += A B^T over ktiles K tiles of 64 (fp16 operands with kHalf, else
// bf16): gemm_core's schedule of one barrier per K tile, in its middle, with
// 2 A stages and NSB (2 or 3) B stages.  Ends with a barrier.
template <class TL, bool AK, bool BK, bool kHalf, class SA, class SB>
__device__ __forceinline__ void mainloop(const SA& a, const SB& b, int ktiles, char* lds, Acc<TL>& acc) {
  static_assert(TL::KS == 2 && TL::NS == 2 && (TL::NSB == 2 || TL::NSB == 3), "64-wide K tiles, 2 A stages");
  constexpr int PA = TL::A_INS, PB = TL::B_INS, DB = TL::NSB - 1;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave / TL::WGN, wn = wave % TL::WGN;
  char* lds_a = lds;
  char* lds_b = lds + TL::B_BASE;
  if (ktiles <= 0) return;
  auto issue_a = [&](int j) {
    const auto t = a.tile(j);
#pragma unroll
    for (int i = 0; i < PA; ++i) a.load(t, i, lds_a + (j & 1) * TL::A_BYTES + (i * TL::NW + wave) * 1024);
  };
  auto issue_b = [&](int j, int stage) {
    const auto t = b.tile(j);
#pragma unroll
    for (int i = 0; i < PB; ++i) b.load(t, i, lds_b + stage * TL::B_BYTES + (i * TL::NW + wave) * 1024);
  };
  // issue order: A0 B0 A1 B1 [B2] | A2 B(NSB) | A3 B(NSB+1) | ...
  issue_a(0);
  issue_b(0, 0);
  if (ktiles > 1) {
    issue_a(1);
    issue_b(1, 1);
  }
  if (DB == 2 && ktiles > 2) issue_b(2, 2);
  if (DB == 2 && ktiles > 2)
    core::wait_loads<PA + 2 * PB>();
  else if (ktiles > 1)
    core::wait_loads<PA + PB>();
  else
    core::wait_loads<0>();
  Frags<TL> f0, f1;
  core::read_frags<TL, AK, BK>(lds_a, lds_b, 0, f0, wm, wn, lane);
  int sb = 0;  // B stage of tile kt
  int kt = 0;
  for (; kt + 1 < ktiles; ++kt) {
    int sb1 = sb + 1;
    if (sb1 == TL::NSB) sb1 = 0;
    // phase 1: MFMAs of (kt, first half) | reads of (kt, second half)
    core::read_frags<TL, AK, BK>(lds_a + (kt & 1) * TL::A_BYTES, lds_b + sb * TL::B_BYTES, 1, f1, wm, wn, lane);
    mfma_frags<TL, kHalf>(f0, acc);
    interleave<TL, AK, BK>();
    // landed: A(kt+1), B(kt+1); still in flight, where B runs 2 ahead: B(kt+2)
    if (DB == 2 && kt + 2 < ktiles)
      core::wait_loads<PB>();
    else
      core::wait_loads<0>();
    // phase 3: the next loads into tile kt's stages, MFMAs of (kt, second
    // half) | reads of (kt+1, first half)
    core::set_prio<1>();
    if (kt + 2 < ktiles) issue_a(kt + 2);
    if (kt + TL::NSB < ktiles) issue_b(kt + TL::NSB, sb);
    core::read_frags<TL, AK, BK>(lds_a + ((kt + 1) & 1) * TL::A_BYTES, lds_b + sb1 * TL::B_BYTES, 0, f0, wm, wn, lane);
    mfma_frags<TL, kHalf>(f1, acc);
    interleave<TL, AK, BK>();
    core::set_prio<0>();
    sb = sb1;
  }
  mfma_frags<TL, kHalf>(f0, acc);
  core::read_frags<TL, AK, BK>(lds_a + ((ktiles - 1) & 1) * TL::A_BYTES, lds_b + sb * TL::B_BYTES, 1, f0, wm, wn, lane);
  mfma_frags<TL, kHalf>(f0, acc);
  __builtin_amdgcn_sched_barrier(0);
  __syncthreads();
}

// The same with TL::NS stages of both operands, NS - 1 of them in flight, for
// tiles that leave room for two workgroups a CU (one's epilogue then runs
// under the other's matrix instructions) or that are few, so that each waits
// for its loads alone.  One barrier per K tile; the fragments of the next one
// are read among the matrix instructions of this one.
template <class TL, bool AK, bool BK, bool kHalf, class SA, class SB>
__device__ __forceinline__ void mainloop_pipe(const SA& a, const SB& b, int ktiles, char* lds, Acc<TL>& acc) {
  static_assert(TL::NSB == TL::NS && (TL::NS - 1) * (TL::A_INS + TL::B_INS) < 64,
                "as many stages of B as of A, and loads that the wait can count");
  constexpr int P = TL::A_INS + TL::B_INS, NS = TL::NS, KS = TL::KS;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave / TL::WGN, wn = wave % TL::WGN;
  char* lds_a = lds;
  char* lds_b = lds + TL::B_BASE;
  if (ktiles <= 0) return;
  auto issue = [&](int j, int stage) {
    const auto ta = a.tile(j);
    const auto tb = b.tile(j);
#pragma unroll
    for (int i = 0; i < TL::A_INS; ++i) a.load(ta, i, lds_a + stage * TL::A_BYTES + (i * TL::NW + wave) * 1024);
#pragma unroll
    for (int i = 0; i < TL::B_INS; ++i) b.load(tb, i, lds_b + stage * TL::B_BYTES + (i * TL::NW + wave) * 1024);
  };
  // at most `tiles` tiles of this wavefront's loads still in flight, then a barrier
  auto wait_tiles = [&](int tiles) {
    if (NS >= 5 && tiles >= 4)
      core::wait_loads<4 * P>();
    else if (NS >= 4 && tiles >= 3)
      core::wait_loads<3 * P>();
    else if (NS >= 3 && tiles >= 2)
      core::wait_loads<2 * P>();
    else if (tiles >= 1)
      core::wait_loads<P>();
    else
      core::wait_loads<0>();
  };
#pragma unroll
  for (int j = 0; j < NS; ++j)
    if (j < ktiles) issue(j, j);
  wait_tiles(min(NS - 1, ktiles - 1));
  Frags<TL> f[2][KS];
  auto read = [&](int stage, Frags<TL> (&g)[KS]) {
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
      core::read_frags<TL, AK, BK>(lds_a + stage * TL::A_BYTES, lds_b + stage * TL::B_BYTES, ks, g[ks], wm, wn, lane);
  };
  read(0, f[0]);
  int stage = 0;  // of tile kt
  auto step = [&](int kt, Frags<TL> (&cur)[KS], Frags<TL> (&nxt)[KS]) {
    // landed: tile kt + 1; every wavefront has read tile kt
    wait_tiles(min(NS - 2, ktiles - 2 - kt));
    core::set_prio<1>();
    if (kt + NS < ktiles) issue(kt + NS, stage);
    if (++stage == NS) stage = 0;
    read(stage, nxt);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) mfma_frags<TL, kHalf>(cur[ks], acc);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) interleave<TL, AK, BK>();
    core::set_prio<0>();
  };
  int kt = 0;
  for (; kt + 2 < ktiles; kt += 2) {
    step(kt, f[0], f[1]);
    step(kt + 1, f[1], f[0]);
  }
  if (kt + 1 < ktiles) {
    step(kt, f[0], f[1]);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) mfma_frags<TL, kHalf>(f[1][ks], acc);
  } else {
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) mfma_frags<TL, kHalf>(f[0][ks], acc);
  }
  __builtin_amdgcn_sched_barrier(0);
  __syncthreads();
}

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

// Rows of one operand at any alignment and of any K, by way of registers.
template <class TL, int INS, int X, bool kMajor>
struct RegRows {
  const uint16_t* ptr;  // the tile's first row (column) at K = 0
  int64_t ld;
  int n, K, wave, lane;  // rows of the operand from there on
  __device__ __forceinline__ void init(const void* p, int r0, int rows, int64_t ld_, int K_, int wave_, int lane_) {
    ptr = static_cast<const uint16_t*>(p) + (kMajor ? r0 : r0 * ld_);
    ld = ld_;
    n = rows - r0;
    K = K_;
    wave = wave_;
    lane = lane_;
  }
  // kLast: the last K tile, in which K ends.  Before it, rows past the
  // operand's are read as its last and columns past it as the first or as what
  // follows in memory (there is another k-row, and a k-row has at least 8
  // values): their results are not stored.
  template <bool kLast>
  __device__ __forceinline__ uint4 load(int j, int i) const {
    if constexpr (kMajor) {
      const int kr = core::kload_row<TL, X>(i, wave, lane), k = j * TL::BK + kr, c = core::kload_col<X>(kr, lane) / 2;
      if constexpr (!kLast) return ld16_any(ptr + k * ld + (c < n ? c : 0));
      return k < K ? ld8_until(ptr + k * ld, c, n) : make_uint4(0, 0, 0, 0);
    } else {
      const int r = core::load_row<TL>(i, wave, lane), k = j * TL::BK + core::load_col<TL>(lane) / 2;
      if constexpr (!kLast) return ld16_any(ptr + min(r, n - 1) * ld + k);
      return r < n ? ld8_until(ptr + r * ld, k, K) : make_uint4(0, 0, 0, 0);
    }
  }
};
template <class TL, bool kAMajor>
using ARegs = RegRows<TL, TL::A_INS, TL::BM, kAMajor>;
template <class TL, bool kBMajor>
using BRegs = RegRows<TL, TL::B_INS, TL::BN, kBMajor>;

// acc += A B^T over such operands: four K tiles' loads in flight in registers,
// two stages of LDS, one barrier per K tile.
template <class TL, bool AK, bool BK, bool kHalf, class SA, class SB>
__device__ __forceinline__ void mainloop_regs(const SA& a, const SB& b, int ktiles, char* lds, Acc<TL>& acc) {
  constexpr int D = 4;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave / TL::WGN, wn = wave % TL::WGN;
  char* lds_a = lds;
  char* lds_b = lds + TL::B_BASE;
  uint4 ra[D][TL::A_INS], rb[D][TL::B_INS];
  auto load = [&](int j, int s) {
    if (j + 1 < ktiles) {
#pragma unroll
      for (int i = 0; i < TL::A_INS; ++i) ra[s][i] = a.template load<false>(j, i);
#pragma unroll
      for (int i = 0; i < TL::B_INS; ++i) rb[s][i] = b.template load<false>(j, i);
    } else if (j < ktiles) {
#pragma unroll
      for (int i = 0; i < TL::A_INS; ++i) ra[s][i] = a.template load<true>(j, i);
#pragma unroll
      for (int i = 0; i < TL::B_INS; ++i) rb[s][i] = b.template load<true>(j, i);
    }
  };
  // tile j's registers to LDS, and the loads of tile j + D into them
  auto stage = [&](int j, int s) {
    char* sa = lds_a + (s & 1) * TL::A_BYTES;
    char* sb = lds_b + (s & 1) * TL::B_BYTES;
#pragma unroll
    for (int i = 0; i < TL::A_INS; ++i) st16(sa + (i * TL::NW + wave) * 1024 + lane * 16, ra[s][i]);
#pragma unroll
    for (int i = 0; i < TL::B_INS; ++i) st16(sb + (i * TL::NW + wave) * 1024 + lane * 16, rb[s][i]);
    load(j + D, s);
  };
  Frags<TL> f[TL::KS];
  auto read = [&](int s) {
    __syncthreads();
#pragma unroll
    for (int ks = 0; ks < TL::KS; ++ks)
      core::read_frags<TL, AK, BK>(lds_a + (s & 1) * TL::A_BYTES, lds_b + (s & 1) * TL::B_BYTES, ks, f[ks], wm, wn, lane);
  };
  if (ktiles <= 0) return;
#pragma unroll
  for (int s = 0; s < D; ++s) load(s, s);
  stage(0, 0);
  read(0);
  for (int j = 0; j < ktiles; j += D) {
#pragma unroll
    for (int s = 0; s < D; ++s)
      if (j + s < ktiles) {
        // the next tile goes to the other stage while this one's products run
        if (j + s + 1 < ktiles) stage(j + s + 1, (s + 1) % D);
#pragma unroll
        for (int ks = 0; ks < TL::KS; ++ks) mfma_frags<TL, kHalf>(f[ks], acc);
        if (j + s + 1 < ktiles) read((s + 1) % D);
      }
  }
  __syncthreads();
}

// LDS written by lanes of a wavefront is read by others of the same one.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// A wavefront's own accumulator tile, `kRows` rows of WN columns at a time,
// through LDS as fp32 (no barrier: each wavefront has its own part), so that
// a lane then meets neighbouring columns: f(row in the workgroup's tile, first
// column in the tile, 8 values).  Rows at or past `rows` are skipped.
template <class TL>
struct Epilogue {
  static constexpr int kRows = 16;
  static constexpr int kLd = TL::WN + 4;  // floats: the 4 row groups of a 16 x 16 block fall on different banks
  static constexpr int kBytes = TL::NW * kRows * kLd * 4;
  static constexpr int kLpr = TL::WN / 8;        // lanes a row
  static constexpr int kRpi = 64 / kLpr;         // rows at a time
  static constexpr int kIts = kRows / kRpi;
  // First of the 8 columns that this lane meets, in every row.
  __device__ __forceinline__ static int column() {
    return ((threadIdx.x >> 6) % TL::WGN) * TL::WN + ((threadIdx.x & 63) % kLpr) * 8;
  }
  // load(row, column) -> X: what the epilogue reads there, fetched one block
  // of kRows ahead (before the stores of the last one, which a load issued
  // later would have to wait for).  f(row, column, 8 values, X).
  template <class X, class Load, class F>
  __device__ __forceinline__ static void run(const Acc<TL>& acc, char* lds, int rows, Load&& load, F&& f) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wm = wave / TL::WGN;
    float* mine = reinterpret_cast<float*>(lds) + wave * kRows * kLd;
    const int r0 = lane / kLpr, c = (lane % kLpr) * 8, col = column();
    X x[2][kIts];
    auto fetch = [&](int mi, X (&to)[kIts]) {
#pragma unroll
      for (int i = 0; i < kIts; ++i) {
        const int row = wm * TL::WM + mi * 16 + i * kRpi + r0;
        if (row < rows) to[i] = load(row, col);
      }
    };
    fetch(0, x[0]);
#pragma unroll
    for (int mi = 0; mi < TL::MI; ++mi) {
      if (mi + 1 < TL::MI) fetch(mi + 1, x[(mi + 1) & 1]);
#pragma unroll
      for (int ni = 0; ni < TL::NI; ++ni)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          mine[((lane >> 4) * 4 + r) * kLd + ni * 16 + (lane & 15)] = acc.v[mi][ni][r];
      wave_sync();
#pragma unroll
      for (int i = 0; i < kIts; ++i) {
        const int row = i * kRpi + r0;
        const f32x4_t lo = *reinterpret_cast<const f32x4_t*>(mine + row * kLd + c);
        const f32x4_t hi = *reinterpret_cast<const f32x4_t*>(mine + row * kLd + c + 4);
        float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        const int at = wm * TL::WM + mi * 16 + row;
        if (at < rows) f(at, col, v, x[mi & 1][i]);
      }
      wave_sync();
    }
  }
  struct None {};
  template <class F>
  __device__ __forceinline__ static void run(const Acc<TL>& acc, char* lds, int rows, F&& f) {
    run<None>(acc, lds, rows, [](int, int) { return None{}; }, [&](int r, int c, float* v, None) { f(r, c, v); });
  }
};

}  // namespace buf
}  // namespace moe
