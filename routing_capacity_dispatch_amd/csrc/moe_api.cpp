// Host side of the C ABI: validation, capacity plan, workspace carving and
// the launch sequence of the branch.  No allocation, no host synchronisation.
#include "moe.h"

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <mutex>

#include "kernels.h"

#define MOE_API extern "C" __attribute__((visibility("default")))

namespace {

constexpr int64_t kI32Max = 2147483647;
constexpr int32_t kMaxWidth = 1 << 20;  // largest d_model, d_latent, d_ff, d_ff_shared
// Most entries of a grouped GEMM's tile list: its grid (one 512-thread
// workgroup per entry, rounded up to a multiple of 8) stays below 2^32
// work-items.
constexpr int64_t kMaxListEntries = (int64_t(1) << 23) - 8;

// Stages of moe_forward, in launch order: latent GEMM, router GEMM, top-k,
// slot assignment, row scatter, receiver binning, expert row lists, expert
// gate/up GEMM, expert down GEMM, combine, shared gate/up GEMM, output GEMM.
constexpr int kStages = 12;

// Records stage boundary i (event i) on the stream when events are given.
struct Marks {
  void* const* ev;
  int n;
  int next;
  hipError_t mark(hipStream_t s) {
    if (!ev || next >= n) return hipSuccess;
    return hipEventRecord(static_cast<hipEvent_t>(ev[next++]), s);
  }
};


int64_t align256(int64_t x) { return (x + 255) & ~int64_t(255); }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Bump allocator over the caller's workspace.
struct Carver {
  char* base;
  int64_t used;
  void* take(int64_t bytes) {
    void* p = base ? base + used : nullptr;
    used += align256(bytes);
    return p;
  }
};

bool aligned256(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 255) == 0; }

// Sizes every entry point needs.  top_k is the number of assignments per
// token; only selection (moe_route, moe_forward) also needs top_k <= E.
moe_status check_route_shape(const moe_config* c) {
  if (!c) return MOE_ERR_INVALID_ARG;
  if (c->T < 0 || c->n_experts < 1 || c->top_k < 1) return MOE_ERR_INVALID_ARG;
  if (c->T * (int64_t)c->n_experts > kI32Max * 64) return MOE_ERR_UNSUPPORTED;
  if (c->T * (int64_t)c->top_k > kI32Max) return MOE_ERR_INVALID_ARG;
  if (c->n_experts > 1024 || c->top_k > 64) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Capacity with exact integer arithmetic: ceil(num * Tw * k / (den * n)).
int64_t capacity(int64_t num, int64_t den, int64_t Tw, int64_t k, int64_t n) {
  const __int128 a = (__int128)num * Tw * k;
  const __int128 b = (__int128)den * n;
  return (int64_t)((a + b - 1) / b);
}

// The routed experts' grouped GEMMs take 256-row tiles instead of 192-row
// ones when an expert's expected rows ceil(T k / E) reach kTallRows: both
// tiles then pad an expert by a few per cent at most, and the taller tile
// does more MFMA work per staged operand byte.  A function of the config
// only, so the plan's workspace sizes and every launch agree.
constexpr int64_t kTallRows = 4096;
bool tall_tiles(const moe_config* c) {
  return ceil_div(c->T * (int64_t)c->top_k, c->n_experts) >= kTallRows;
}

// Upper bounds of the ragged GEMMs' tile lists: expert e has
// ceil(count_e / bm) <= count_e / bm + 1 M tiles.
void dropless_entries(const moe_config* c, int64_t* ent0, int64_t* ent1) {
  const int64_t n = c->T * (int64_t)c->top_k;
  const int64_t bm = moe::ragged_tile_rows(tall_tiles(c));
  const int64_t mt = ceil_div(n, bm) + c->n_experts;
  *ent0 = mt * ceil_div(c->d_ff, moe::ragged_gate_up_cols());
  *ent1 = mt * ceil_div(c->d_latent, moe::ragged_down_cols());
}

// Tile-list bounds of the capped path's grouped GEMMs: expert e holds at
// most max_rows kept rows, and sum_e count_e <= E * max_rows.
void capped_entries(const moe_config* c, int64_t max_rows, int64_t* ent0, int64_t* ent1) {
  const int64_t bm = moe::ragged_tile_rows(tall_tiles(c));
  const int64_t E = c->n_experts;
  const int64_t per = ceil_div(max_rows, bm);
  const int64_t mt = per * E < ceil_div(E * max_rows, bm) + E ? per * E : ceil_div(E * max_rows, bm) + E;
  *ent0 = mt * ceil_div(c->d_ff, moe::ragged_gate_up_cols());
  *ent1 = mt * ceil_div(c->d_latent, moe::ragged_down_cols());
}

// Tile-list bounds of the backward's grouped dgrad GEMMs over R padded
// rows: sum_e ceil(rows_e / bm) <= R / bm + E M tiles.
void backward_entries(const moe_config* c, int64_t R, int64_t* pre, int64_t* dh, int64_t* du) {
  const int64_t mt = ceil_div(R, moe::bwd_dgrad_rows()) + c->n_experts;
  *pre = mt * ceil_div(c->d_ff, moe::ragged_gate_up_cols());
  *dh = mt * ceil_div(c->d_ff, moe::bwd_dgrad_cols());
  *du = mt * ceil_div(c->d_latent, moe::bwd_dgrad_cols());
}

moe_status plan_impl(const moe_config* c, moe_plan* p) {
  if (!c || !p) return MOE_ERR_INVALID_ARG;
  moe_status st = check_route_shape(c);
  if (st != MOE_OK) return st;
  if (c->d_model < 1 || c->d_latent < 1 || c->d_ff < 1 || c->n_pools < 1 || c->n_waves < 1 ||
      c->n_shared < 0 || (c->n_shared > 0 && c->d_ff_shared < 1))
    return MOE_ERR_INVALID_ARG;
  if (c->n_experts % c->n_pools) return MOE_ERR_INVALID_ARG;
  if (c->send_cap_num < 0 || c->send_cap_den < 1 || c->recv_cap_num < 0 || c->recv_cap_den < 1 ||
      c->cap_send_rows < 0 || c->cap_recv_rows < 0)
    return MOE_ERR_INVALID_ARG;
  if (c->dtype != MOE_F32 && c->dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
  if (c->reserved != 0) return MOE_ERR_INVALID_ARG;
  if (c->d_model % 64 || c->d_latent % 64 || c->d_ff % 64 ||
      (c->n_shared > 0 && c->d_ff_shared % 64))
    return MOE_ERR_UNSUPPORTED;
  // widths up to 2^20: with T * k < 2^31 and every capacity product below
  // 2^31, each workspace size below stays far inside int64
  if (c->d_model > kMaxWidth || c->d_latent > kMaxWidth || c->d_ff > kMaxWidth ||
      (c->n_shared > 0 && c->d_ff_shared > kMaxWidth))
    return MOE_ERR_UNSUPPORTED;
  if (c->n_shared > 3) return MOE_ERR_UNSUPPORTED;
  if (c->n_waves > 65535) return MOE_ERR_UNSUPPORTED;  // the slot scan's grid has one row per wave

  const int64_t T = c->T, W = c->n_waves, E = c->n_experts, P = c->n_pools, k = c->top_k;
  const int64_t Tw = ceil_div(T, W);
  const int64_t cs = c->cap_send_rows ? c->cap_send_rows
                                      : capacity(c->send_cap_num, c->send_cap_den, Tw, k, P);
  const int64_t cr = c->cap_recv_rows ? c->cap_recv_rows
                                      : capacity(c->recv_cap_num, c->recv_cap_den, Tw, k, E);
  // every index the kernels form stays inside int32 (each capacity first, so
  // no product can overflow: W, P, E < 2^17)
  if (cs > kI32Max || cr > kI32Max || W * P * cs > kI32Max || W * E * cr > kI32Max)
    return MOE_ERR_UNSUPPORTED;
  const int64_t eb = c->dtype == MOE_BF16 ? 2 : 4;
  const int64_t L = c->d_latent, F = c->d_ff;
  const int64_t S = c->n_shared, Fs = c->d_ff_shared;

  // the bf16 GEMMs address each operand buffer as a scalar base plus a
  // 32-bit lane offset: every buffer read from one base stays below 4 GiB
  if (c->dtype == MOE_BF16) {
    const int64_t kLim = int64_t(1) << 32;
    const int64_t D = c->d_model;
    const int64_t pools = W * P * align256(cs * L * 2 + cs * 4);
    const int64_t widest = D > L ? D : L;
    if (T * widest * 2 >= kLim || T * S * Fs * 2 >= kLim || pools >= kLim || F * L * 2 >= kLim ||
        L * D * 2 >= kLim || Fs * D * 2 >= kLim)
      return MOE_ERR_UNSUPPORTED;
  }

  p->tokens_per_wave = Tw;
  p->cap_send = cs;
  p->cap_recv = cr;
  p->experts_per_pool = E / P;
  p->elem_bytes = eb;
  p->row_bytes = L * eb;
  p->ids_offset = cs * L * eb;
  p->pool_block_bytes = align256(p->ids_offset + cs * 4);
  p->pools_bytes = W * P * p->pool_block_bytes;
  p->expert_out_bytes = align256(W * P * cs * L * eb);
  p->max_expert_rows = W * cr;

  Carver d{nullptr, 0};
  d.take(W * 3 * 8);  // per-wave counters
  d.take(W * moe::assign_chunks(Tw, k) * (int64_t)(E + P) * 4);  // per-chunk key counts of the slot scan
  p->dispatch_ws_bytes = d.used;

  Carver x{nullptr, 0};
  if (c->dtype == MOE_BF16) {
    int64_t e0, e1;
    capped_entries(c, W * cr, &e0, &e1);
    if (e0 > kMaxListEntries || e1 > kMaxListEntries) return MOE_ERR_UNSUPPORTED;
    x.take((E + 1) * 4);          // expert-major row offsets
    x.take(E * W * cr * 4);       // flat pool-row index of each kept row
    x.take(e0 * 12);              // gate/up tile list
    x.take(e1 * 12);              // down tile list
    x.take(8);                    // list lengths
    x.take(E * W * cr * F * eb);  // SwiGLU hidden rows, expert-major
  } else {
    x.take(E * W * cr * 4);       // expert row lists
    x.take(E * 4);                // rows per expert
    x.take(E * W * cr * F * eb);  // SwiGLU hidden rows
  }
  p->experts_ws_bytes = x.used;

  Carver f{nullptr, 0};
  f.take(T * L * eb);         // z
  f.take(T * E * 4);          // logits
  f.take(T * k * 4);          // topk
  f.take(T * k * 4);          // gates
  f.take(T * k * 4);          // pool_slot
  f.take(T * k * 4);          // recv_slot
  f.take(W * P * 4);          // pool_count
  f.take(W * E * 4);          // expert_count
  f.take(W * E * cr * 4);     // bank_rows
  f.take(p->pools_bytes);     // pools
  f.take(p->expert_out_bytes);
  f.take(T * L * eb);         // y_latent
  f.take(T * S * Fs * eb);    // shared hidden
  f.take(3 * 8);              // counters
  f.take(p->dispatch_ws_bytes);
  f.take(p->experts_ws_bytes);
  p->forward_ws_bytes = f.used;

  // dropless ragged variant
  const int64_t n = T * k;
  int64_t ent0, ent1;
  dropless_entries(c, &ent0, &ent1);
  if (ent0 > kMaxListEntries || ent1 > kMaxListEntries) return MOE_ERR_UNSUPPORTED;
  const int64_t nblk = moe::ragged_sort_blocks(n);
  p->dropless_rows = n;
  Carver dd{nullptr, 0};
  dd.take(nblk * E * 4);  // per-chunk histograms
  dd.take(nblk * E * 4);  // per-chunk bases
  p->dropless_dispatch_ws_bytes = dd.used;
  Carver dx{nullptr, 0};
  dx.take(ent0 * 12);     // gate/up tile list
  dx.take(ent1 * 12);     // down tile list
  dx.take(8);             // list lengths
  dx.take(n * F * eb);    // SwiGLU hidden rows
  p->dropless_experts_ws_bytes = dx.used;
  Carver df{nullptr, 0};
  df.take(T * L * eb);    // z
  df.take(T * E * 4);     // logits
  df.take(T * k * 4);     // topk
  df.take(T * k * 4);     // gates
  df.take(T * k * 4);     // row_of
  df.take((E + 1) * 4);   // expert offsets
  df.take(n * L * eb);    // xs
  df.take(n * L * eb);    // expert_out
  df.take(T * L * eb);    // y_latent
  df.take(T * S * Fs * eb);
  df.take(3 * 8);
  df.take(p->dropless_dispatch_ws_bytes);
  df.take(p->dropless_experts_ws_bytes);
  p->dropless_forward_ws_bytes = df.used;

  // backward of the routed path: expert e's kept rows, rounded up to 64
  const int64_t kept_max = T * k < E * W * cr ? T * k : E * W * cr;
  const int64_t R = kept_max + 63 * E;
  int64_t bpre, bdh, bdu;
  backward_entries(c, R, &bpre, &bdh, &bdu);
  if (R > kI32Max || bpre > kMaxListEntries || bdh > kMaxListEntries || bdu > kMaxListEntries)
    return MOE_ERR_UNSUPPORTED;
  p->backward_rows = R;
  Carver bx{nullptr, 0};
  bx.take(E * 4);           // rows per expert
  bx.take((E + 1) * 4);     // padded offsets
  bx.take(R * 4);           // pool row of each padded row
  bx.take(bpre * 12);       // recompute tile list
  bx.take(bdh * 12);        // dh tile list
  bx.take(bdu * 12);        // du tile list
  bx.take(16);              // list lengths
  bx.take(R * L * 2);       // u rows
  bx.take(R * L * 2);       // do rows
  bx.take(R * F * 2);       // dh
  bx.take(R * 2 * F * 2);   // da | db
  bx.take(R * F * 2);       // h
  p->experts_bwd_ws_bytes = bx.used;
  // ... and for the dropless variant, over its T*k rows
  const int64_t Rd = n + 63 * E;
  int64_t dpre, ddh, ddu;
  backward_entries(c, Rd, &dpre, &ddh, &ddu);
  if (Rd > kI32Max || dpre > kMaxListEntries || ddh > kMaxListEntries || ddu > kMaxListEntries)
    return MOE_ERR_UNSUPPORTED;
  p->dropless_backward_rows = Rd;
  Carver dbx{nullptr, 0};
  dbx.take(E * 4);
  dbx.take((E + 1) * 4);
  dbx.take(Rd * 4);
  dbx.take(dpre * 12);
  dbx.take(ddh * 12);
  dbx.take(ddu * 12);
  dbx.take(16);
  dbx.take(Rd * L * 2);
  dbx.take(Rd * L * 2);
  dbx.take(Rd * F * 2);
  dbx.take(Rd * 2 * F * 2);
  dbx.take(Rd * F * 2);
  p->dropless_experts_bwd_ws_bytes = dbx.used;
  Carver dbb{nullptr, 0};
  dbb.take(T * k * 4);       // d_gates
  dbb.take(n * L * eb);      // d_expert_out
  dbb.take(n * L * eb);      // d_xs
  dbb.take(p->dropless_experts_bwd_ws_bytes);
  p->dropless_backward_ws_bytes = dbb.used;
  Carver bb{nullptr, 0};
  bb.take(T * k * 4);              // d_gates
  bb.take(p->expert_out_bytes);    // d_expert_out
  bb.take(p->expert_out_bytes);    // d_pool_rows
  bb.take(p->experts_bwd_ws_bytes);
  p->backward_ws_bytes = bb.used;
  return MOE_OK;
}

moe_status hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

moe::DispatchArgs dispatch_args(const moe_config* c, const moe_plan& p, const int32_t* topk,
                                void* pools, int32_t* pool_slot, int32_t* recv_slot,
                                int32_t* pool_count, int64_t* wave_counts, int64_t* counts) {
  moe::DispatchArgs a{};
  a.topk = topk;
  a.T = c->T;
  a.k = c->top_k;
  a.E = c->n_experts;
  a.P = c->n_pools;
  a.W = c->n_waves;
  a.Tw = p.tokens_per_wave;
  a.cap_send = p.cap_send;
  a.cap_recv = p.cap_recv;
  a.pool_slot = pool_slot;
  a.recv_slot = recv_slot;
  a.pool_count = pool_count;
  a.pools = static_cast<char*>(pools);
  a.block_bytes = p.pool_block_bytes;
  a.ids_offset = p.ids_offset;
  a.row_bytes = p.row_bytes;
  a.wave_counts = wave_counts;
  a.counts = counts;
  return a;
}

moe_status run_dispatch(const moe_config* c, const moe_plan& p, const int32_t* topk, const void* z,
                        void* pools, int32_t* pool_slot, int32_t* recv_slot, int32_t* bank_rows,
                        int32_t* pool_count, int32_t* expert_count, int64_t* counts, void* ws,
                        hipStream_t s, Marks* m) {
  Carver cv{static_cast<char*>(ws), 0};
  int64_t* wave_counts = static_cast<int64_t*>(cv.take(c->n_waves * 3 * 8));
  moe::DispatchArgs a =
      dispatch_args(c, p, topk, pools, pool_slot, recv_slot, pool_count, wave_counts, counts);
  a.n_chunks = moe::assign_chunks(p.tokens_per_wave, c->top_k);
  a.chunk_counts = static_cast<int32_t*>(
      cv.take(c->n_waves * (int64_t)a.n_chunks * (c->n_experts + c->n_pools) * 4));
  hipError_t e = moe::launch_assign(a, s);
  if (e == hipSuccess && m) e = m->mark(s);
  if (e == hipSuccess) e = moe::launch_scatter_rows(a, z, s);
  if (e == hipSuccess && m) e = m->mark(s);
  if (e == hipSuccess) e = moe::launch_recv_bin(a, bank_rows, expert_count, s);
  if (e == hipSuccess && m) e = m->mark(s);
  return hip_status(e);
}

moe_status run_experts(const moe_config* c, const moe_plan& p, const void* pools,
                       const int32_t* bank_rows, const int32_t* expert_count, const void* wg,
                       const void* wu, const void* wd, void* expert_out, void* ws,
                       hipStream_t s, Marks* m) {
  const int E = c->n_experts;
  const int max_rows = (int)p.max_expert_rows;
  Carver cv{static_cast<char*>(ws), 0};
  if (c->dtype == MOE_BF16) {
    // expert-major row lists, then the grouped GEMMs over device-built tile
    // lists (rows gathered from the pools, outputs scattered back to them)
    int64_t ent0, ent1;
    capped_entries(c, max_rows, &ent0, &ent1);
    int32_t* offsets = static_cast<int32_t*>(cv.take((int64_t)(E + 1) * 4));
    int32_t* gidx = static_cast<int32_t*>(cv.take((int64_t)E * max_rows * 4));
    int32_t* list0 = static_cast<int32_t*>(cv.take(ent0 * 12));
    int32_t* list1 = static_cast<int32_t*>(cv.take(ent1 * 12));
    int32_t* ntiles = static_cast<int32_t*>(cv.take(8));
    char* H = static_cast<char*>(cv.take((int64_t)E * max_rows * c->d_ff * p.elem_bytes));
    const int tn0 = (int)ceil_div(c->d_ff, moe::ragged_gate_up_cols());
    const int tn1 = (int)ceil_div(c->d_latent, moe::ragged_down_cols());
    hipError_t e = moe::launch_expert_gidx(bank_rows, expert_count, E, c->n_pools, c->n_waves, p.cap_send,
                                           p.cap_recv, offsets, gidx, s);
    if (e == hipSuccess)
      e = moe::launch_ragged_tiles(offsets, E, moe::ragged_tile_rows(tall_tiles(c)), tn0, tn1, list0, list1,
                                   ntiles, s);
    if (e == hipSuccess && m) e = m->mark(s);
    if (e != hipSuccess) return MOE_ERR_HIP;
    moe::RaggedGemm g{};
    g.A = static_cast<const char*>(pools);
    g.a_row_bytes = p.row_bytes;
    g.a_index = gidx;
    g.a_block_rows = (int)p.cap_send;
    g.a_block_bytes = p.pool_block_bytes;
    g.offsets = offsets;
    g.list = list0;
    g.ntiles = ntiles;
    g.W0 = static_cast<const char*>(wg);
    g.W1 = static_cast<const char*>(wu);
    g.E = E;
    g.F = c->d_ff;
    g.K = c->d_latent;
    g.C = H;
    g.c_row_bytes = (int64_t)c->d_ff * p.elem_bytes;
    e = moe::launch_ragged_gate_up_bf16(g, ent0, tall_tiles(c), s);
    if (e == hipSuccess && m) e = m->mark(s);
    if (e != hipSuccess) return MOE_ERR_HIP;
    moe::RaggedGemm d{};
    d.A = H;
    d.a_row_bytes = (int64_t)c->d_ff * p.elem_bytes;
    d.offsets = offsets;
    d.list = list1;
    d.ntiles = ntiles + 1;
    d.W0 = static_cast<const char*>(wd);
    d.E = E;
    d.K = c->d_ff;
    d.N = c->d_latent;
    d.C = static_cast<char*>(expert_out);
    d.c_row_bytes = p.row_bytes;
    d.c_index = gidx;
    e = moe::launch_ragged_down_bf16(d, ent1, tall_tiles(c), s);
    if (e == hipSuccess && m) e = m->mark(s);
    return hip_status(e);
  }
  int32_t* erow = static_cast<int32_t*>(cv.take((int64_t)E * max_rows * 4));
  int32_t* rows_total = static_cast<int32_t*>(cv.take((int64_t)E * 4));
  void* H = cv.take((int64_t)E * max_rows * c->d_ff * p.elem_bytes);
  hipError_t e = moe::launch_expert_rows(bank_rows, expert_count, E, c->n_pools, c->n_waves,
                                         p.cap_send, p.cap_recv, erow, rows_total, max_rows, s);
  if (e == hipSuccess && m) e = m->mark(s);
  if (e != hipSuccess) return MOE_ERR_HIP;
  moe::ExpertGateUp gu{};
  gu.pools = static_cast<const char*>(pools);
  gu.block_bytes = p.pool_block_bytes;
  gu.row_bytes = p.row_bytes;
  gu.cap_send = (int)p.cap_send;
  gu.erow = erow;
  gu.rows_total = rows_total;
  gu.E = E;
  gu.max_rows = max_rows;
  gu.F = c->d_ff;
  gu.L = c->d_latent;
  gu.Wg = wg;
  gu.Wu = wu;
  gu.H = H;
  e = moe::launch_expert_gate_up(c->dtype, gu, s);
  if (e == hipSuccess && m) e = m->mark(s);
  if (e != hipSuccess) return MOE_ERR_HIP;
  moe::ExpertDown dn{};
  dn.H = H;
  dn.erow = erow;
  dn.rows_total = rows_total;
  dn.E = E;
  dn.max_rows = max_rows;
  dn.F = c->d_ff;
  dn.L = c->d_latent;
  dn.Wd = wd;
  dn.out = expert_out;
  e = moe::launch_expert_down(c->dtype, dn, s);
  if (e == hipSuccess && m) e = m->mark(s);
  return hip_status(e);
}

moe_status run_combine(const moe_config* c, const moe_plan& p, const void* expert_out,
                       const int32_t* topk, const int32_t* pool_slot, const int32_t* recv_slot,
                       const float* gates, void* y_latent, hipStream_t s, int64_t y_pitch = 0) {
  moe::CombineArgs a{};
  a.expert_out = static_cast<const char*>(expert_out);
  a.topk = topk;
  a.pool_slot = pool_slot;
  a.recv_slot = recv_slot;
  a.gates = gates;
  a.T = c->T;
  a.Tw = p.tokens_per_wave;
  a.k = c->top_k;
  a.E = c->n_experts;
  a.P = c->n_pools;
  a.cap_send = p.cap_send;
  a.row_bytes = p.row_bytes;
  a.y = y_latent;
  a.y_pitch = y_pitch;
  return hip_status(moe::launch_combine(c->dtype, a, s));
}

}  // namespace

MOE_API const char* moe_status_string(moe_status s) {
  switch (s) {
    case MOE_OK: return "MOE_OK";
    case MOE_ERR_INVALID_ARG: return "MOE_ERR_INVALID_ARG: invalid argument";
    case MOE_ERR_UNSUPPORTED: return "MOE_ERR_UNSUPPORTED: unsupported shape";
    case MOE_ERR_WORKSPACE: return "MOE_ERR_WORKSPACE: workspace too small or misaligned";
    case MOE_ERR_HIP: return "MOE_ERR_HIP: kernel launch failed";
  }
  return "unknown moe_status";
}

MOE_API int32_t moe_version(void) { return 100; }

MOE_API moe_status moe_make_plan(const moe_config* cfg, moe_plan* plan) {
  return plan_impl(cfg, plan);
}

MOE_API moe_status moe_route(const moe_config* cfg, const float* logits, const float* bias,
                             int32_t* topk_idx, float* gates, void* stream) {
  moe_status st = check_route_shape(cfg);
  if (st != MOE_OK) return st;
  if (cfg->top_k > cfg->n_experts) return MOE_ERR_INVALID_ARG;
  if (cfg->T > 0 && (!logits || !topk_idx || !gates)) return MOE_ERR_INVALID_ARG;
  return hip_status(moe::launch_topk_gates(logits, bias, cfg->T, cfg->n_experts, cfg->top_k,
                                           topk_idx, gates, static_cast<hipStream_t>(stream)));
}

static moe_status check_bias_update(const moe_config* cfg, int32_t n_bins) {
  moe_status st = check_route_shape(cfg);
  if (st != MOE_OK) return st;
  if (cfg->T < 1 || cfg->top_k > cfg->n_experts) return MOE_ERR_INVALID_ARG;
  if (n_bins < 1 || n_bins > moe::bias_max_bins()) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

MOE_API moe_status moe_router_bias_ws_bytes(const moe_config* cfg, int32_t n_bins, size_t* bytes) {
  moe_status st = check_bias_update(cfg, n_bins);
  if (st != MOE_OK) return st;
  if (!bytes) return MOE_ERR_INVALID_ARG;
  *bytes = (size_t)moe::bias_ws_bytes(cfg->T, cfg->n_experts, n_bins);
  return MOE_OK;
}

static moe_status bias_update_impl(const moe_config* cfg, const float* logits, int32_t n_bins, float* bias_next,
                                   int32_t* hist, float* lohi, void* ws, size_t ws_bytes, void* stream,
                                   void* const* events) {
  moe_status st = check_bias_update(cfg, n_bins);
  if (st != MOE_OK) return st;
  if (!logits || !bias_next) return MOE_ERR_INVALID_ARG;
  if (!ws || !aligned256(ws) || (int64_t)ws_bytes < moe::bias_ws_bytes(cfg->T, cfg->n_experts, n_bins))
    return MOE_ERR_WORKSPACE;
  return hip_status(moe::launch_bias_update(logits, cfg->T, cfg->n_experts, cfg->top_k, n_bins, bias_next, hist,
                                            lohi, ws, static_cast<hipStream_t>(stream), events));
}

MOE_API moe_status moe_router_bias_update(const moe_config* cfg, const float* logits, int32_t n_bins,
                                          float* bias_next, int32_t* hist, float* lohi, void* ws,
                                          size_t ws_bytes, void* stream) {
  return bias_update_impl(cfg, logits, n_bins, bias_next, hist, lohi, ws, ws_bytes, stream, nullptr);
}

MOE_API int32_t moe_router_bias_stage_count(void) { return 4; }

MOE_API moe_status moe_router_bias_update_profiled(const moe_config* cfg, const float* logits, int32_t n_bins,
                                                   float* bias_next, int32_t* hist, float* lohi, void* ws,
                                                   size_t ws_bytes, void* stream, void* const* stage_events,
                                                   int32_t n_events) {
  if (!stage_events || n_events < 5) return MOE_ERR_INVALID_ARG;
  return bias_update_impl(cfg, logits, n_bins, bias_next, hist, lohi, ws, ws_bytes, stream, stage_events);
}

MOE_API moe_status moe_dispatch(const moe_config* cfg, const int32_t* topk_idx, const void* z,
                                void* pools, int32_t* pool_slot, int32_t* recv_slot,
                                int32_t* bank_rows, int32_t* pool_count, int32_t* expert_count,
                                int64_t* counts, void* ws, size_t ws_bytes, void* stream) {
  moe_plan p;
  moe_status st = plan_impl(cfg, &p);
  if (st != MOE_OK) return st;
  if (!pool_count || !expert_count || !counts) return MOE_ERR_INVALID_ARG;
  if ((p.pools_bytes > 0 && !pools) || (p.cap_recv > 0 && !bank_rows)) return MOE_ERR_INVALID_ARG;
  if (cfg->T > 0 && (!topk_idx || !z || !pool_slot || !recv_slot)) return MOE_ERR_INVALID_ARG;
  if (!ws || (int64_t)ws_bytes < p.dispatch_ws_bytes || !aligned256(ws)) return MOE_ERR_WORKSPACE;
  return run_dispatch(cfg, p, topk_idx, z, pools, pool_slot, recv_slot, bank_rows, pool_count,
                      expert_count, counts, ws, static_cast<hipStream_t>(stream), nullptr);
}

// ---- dispatch without allocation -----------------------------------------
// The scratch of moe_dispatch_noalloc (per-wave counters and per-chunk key
// counts, the same bytes moe_dispatch takes as its workspace) lives in this
// file-scope device array: every GPU the library runs on holds one copy at
// its own address until the process ends.  In host code the array's name is
// a host-side stand-in, never a device address: only the pointer that
// hipGetSymbolAddress returns for the current device is handed to kernels.
namespace {

constexpr int64_t kNoallocScratchBytes = int64_t(4) << 20;
constexpr int kMaxDevices = 64;
__device__ __align__(256) char noalloc_scratch[kNoallocScratchBytes];

std::mutex g_scratch_mu;
void* g_scratch_ptr[kMaxDevices] = {};

// The current device's copy of the array, looked up once per device (with
// that device current) on the first call that runs there.
moe_status noalloc_scratch_ptr(void** out) {
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return MOE_ERR_HIP;
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (!g_scratch_ptr[dev]) {
    void* ptr = nullptr;
    if (hipGetSymbolAddress(&ptr, HIP_SYMBOL(noalloc_scratch)) != hipSuccess || !ptr) return MOE_ERR_HIP;
    g_scratch_ptr[dev] = ptr;
  }
  *out = g_scratch_ptr[dev];
  return MOE_OK;
}

}  // namespace

MOE_API int64_t moe_dispatch_noalloc_scratch_bytes(void) { return kNoallocScratchBytes; }

MOE_API moe_status moe_dispatch_noalloc(const moe_config* cfg, const int32_t* topk_idx, const void* z,
                                        void* pools, int32_t* pool_slot, int32_t* recv_slot,
                                        int32_t* bank_rows, int32_t* pool_count, int32_t* expert_count,
                                        int64_t* counts, void* stream) {
  moe_plan p;
  moe_status st = plan_impl(cfg, &p);
  if (st != MOE_OK) return st;
  if (!pool_count || !expert_count || !counts) return MOE_ERR_INVALID_ARG;
  if ((p.pools_bytes > 0 && !pools) || (p.cap_recv > 0 && !bank_rows)) return MOE_ERR_INVALID_ARG;
  if (cfg->T > 0 && (!topk_idx || !z || !pool_slot || !recv_slot)) return MOE_ERR_INVALID_ARG;
  if (p.dispatch_ws_bytes > kNoallocScratchBytes) return MOE_ERR_WORKSPACE;
  void* scratch = nullptr;
  st = noalloc_scratch_ptr(&scratch);
  if (st != MOE_OK) return st;
  // the kernels clear what they accumulate into (the first workgroup of the
  // count pass zeroes the per-wave counters; every chunk count that is read
  // is written first), so the array's previous contents do not matter
  return run_dispatch(cfg, p, topk_idx, z, pools, pool_slot, recv_slot, bank_rows, pool_count,
                      expert_count, counts, scratch, static_cast<hipStream_t>(stream), nullptr);
}

MOE_API moe_status moe_experts(const moe_config* cfg, const void* pools, const int32_t* bank_rows,
                               const int32_t* expert_count, const void* w_gate, const void* w_up,
                               const void* w_down, void* expert_out, void* ws, size_t ws_bytes,
                               void* stream) {
  moe_plan p;
  moe_status st = plan_impl(cfg, &p);
  if (st != MOE_OK) return st;
  if (!expert_count || !w_gate || !w_up || !w_down) return MOE_ERR_INVALID_ARG;
  if ((p.pools_bytes > 0 && (!pools || !expert_out)) || (p.cap_recv > 0 && !bank_rows))
    return MOE_ERR_INVALID_ARG;
  if (!ws || (int64_t)ws_bytes < p.experts_ws_bytes || !aligned256(ws)) return MOE_ERR_WORKSPACE;
  return run_experts(cfg, p, pools, bank_rows, expert_count, w_gate, w_up, w_down, expert_out, ws,
                     static_cast<hipStream_t>(stream), nullptr);
}

MOE_API moe_status moe_combine(const moe_config* cfg, const void* expert_out,
                               const int32_t* topk_idx, const int32_t* pool_slot,
                               const int32_t* recv_slot, const float* gates, void* y_latent,
                               void* stream) {
  moe_plan p;
  moe_status st = plan_impl(cfg, &p);
  if (st != MOE_OK) return st;
  // pool-shaped buffers are empty when the sender capacity is 0: then they may be null
  if (cfg->T > 0 && ((p.expert_out_bytes > 0 && !expert_out) || !topk_idx || !pool_slot || !recv_slot || !gates ||
                     !y_latent))
    return MOE_ERR_INVALID_ARG;
  return run_combine(cfg, p, expert_out, topk_idx, pool_slot, recv_slot, gates, y_latent,
                     static_cast<hipStream_t>(stream));
}

namespace {

moe_status forward_impl(const moe_config* cfg, const moe_weights* w, const void* x, void* y,
                        const moe_taps* taps, int64_t* counts, void* ws, size_t ws_bytes,
                        void* stream, void* const* events, int n_events) {
  moe_plan p;
  moe_status st = plan_impl(cfg, &p);
  if (st != MOE_OK) return st;
  if (cfg->top_k > cfg->n_experts) return MOE_ERR_INVALID_ARG;
  // the router GEMM writes fp32 logit rows in 16-byte chunks
  if (cfg->n_experts % 4) return MOE_ERR_UNSUPPORTED;
  if (!w) return MOE_ERR_INVALID_ARG;
  if (!w->w_latent || !w->w_router || !w->w_gate || !w->w_up || !w->w_down || !w->w_up_proj)
    return MOE_ERR_INVALID_ARG;
  if (cfg->n_shared > 0 && (!w->ws_gate || !w->ws_up || !w->ws_down)) return MOE_ERR_INVALID_ARG;
  if (cfg->T > 0 && (!x || !y)) return MOE_ERR_INVALID_ARG;
  if (!ws || (int64_t)ws_bytes < p.forward_ws_bytes || !aligned256(ws)) return MOE_ERR_WORKSPACE;

  const moe_taps none{};
  const moe_taps& tp = taps ? *taps : none;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int64_t T = cfg->T, W = cfg->n_waves, E = cfg->n_experts, P = cfg->n_pools,
                k = cfg->top_k;
  const int64_t L = cfg->d_latent, D = cfg->d_model, S = cfg->n_shared, Fs = cfg->d_ff_shared;
  const int64_t eb = p.elem_bytes;
  const int dt = cfg->dtype;

  Carver cv{static_cast<char*>(ws), 0};
  auto pick = [&](void* tap, int64_t bytes) {
    void* q = cv.take(bytes);
    return tap ? tap : q;
  };
  void* z = pick(tp.z, T * L * eb);
  float* logits = static_cast<float*>(pick(tp.logits, T * E * 4));
  int32_t* topk = static_cast<int32_t*>(pick(tp.topk_idx, T * k * 4));
  float* gates = static_cast<float*>(pick(tp.gates, T * k * 4));
  int32_t* pool_slot = static_cast<int32_t*>(pick(tp.pool_slot, T * k * 4));
  int32_t* recv_slot = static_cast<int32_t*>(pick(tp.recv_slot, T * k * 4));
  int32_t* pool_count = static_cast<int32_t*>(pick(tp.pool_count, W * P * 4));
  int32_t* expert_count = static_cast<int32_t*>(pick(tp.expert_count, W * E * 4));
  int32_t* bank_rows = static_cast<int32_t*>(pick(tp.bank_rows, W * E * p.cap_recv * 4));
  void* pools = pick(tp.pools, p.pools_bytes);
  void* expert_out = pick(tp.expert_out, p.expert_out_bytes);
  void* y_lat = pick(tp.y_latent, T * L * eb);
  void* hs = cv.take(T * S * Fs * eb);
  // Without a y_latent tap, y_lat and the shared hidden rows are the two
  // column blocks of one [T][L + S*Fs] buffer (it fits in the two carves
  // above), so the output projection reads one A operand over all its K
  // ranges.
  int64_t ylat_ld = L, hs_ld = S * Fs;
  if (!tp.y_latent && S > 0 && T * (L + S * Fs) * eb < (int64_t(1) << 32)) {
    hs = static_cast<char*>(y_lat) + L * eb;
    ylat_ld = hs_ld = L + S * Fs;
  }
  int64_t* cnt = static_cast<int64_t*>(pick(counts, 3 * 8));
  void* dws = cv.take(p.dispatch_ws_bytes);
  void* xws = cv.take(p.experts_ws_bytes);

  Marks mk{events, n_events, 0};
  Marks* m = &mk;
  hipError_t e = m->mark(s);  // start of stage 0
  if (e != hipSuccess) return MOE_ERR_HIP;
  // latent projection z = x W_lat^T
  moe::GemmDense g{};
  g.nseg = 1;
  g.seg[0] = {x, D, w->w_latent, D, (int)D};
  g.C = z;
  g.ldc = L;
  g.M = (int)T;
  g.N = (int)L;
  e = moe::launch_gemm_dense(dt, dt, g, s);
  if (e == hipSuccess) e = m->mark(s);
  if (e != hipSuccess) return MOE_ERR_HIP;
  // router logits (fp32) = z W_r^T
  g.seg[0] = {z, L, w->w_router, L, (int)L};
  g.C = logits;
  g.ldc = E;
  g.N = (int)E;
  e = moe::launch_gemm_dense(dt, moe::DT_F32, g, s);
  if (e == hipSuccess) e = m->mark(s);
  if (e != hipSuccess) return MOE_ERR_HIP;
  e = moe::launch_topk_gates(logits, w->router_bias, T, (int)E, (int)k, topk, gates, s);
  if (e == hipSuccess) e = m->mark(s);
  if (e != hipSuccess) return MOE_ERR_HIP;
  st = run_dispatch(cfg, p, topk, z, pools, pool_slot, recv_slot, bank_rows, pool_count,
                    expert_count, cnt, dws, s, m);
  if (st != MOE_OK) return st;
  st = run_experts(cfg, p, pools, bank_rows, expert_count, w->w_gate, w->w_up, w->w_down,
                   expert_out, xws, s, m);
  if (st != MOE_OK) return st;
  st = run_combine(cfg, p, expert_out, topk, pool_slot, recv_slot, gates, y_lat, s, ylat_ld * eb);
  if (st == MOE_OK && m->mark(s) != hipSuccess) st = MOE_ERR_HIP;
  if (st != MOE_OK) return st;
  // shared experts' hidden rows: silu(x Wg_s^T) * (x Wu_s^T), [T][S*Fs]
  if (S > 0) {
    e = moe::launch_swiglu_dense(dt, x, D, w->ws_gate, w->ws_up, (int)S, (int)Fs, (int)D, (int)T,
                                 hs, hs_ld, s);
    if (e != hipSuccess) return MOE_ERR_HIP;
  }
  if (m->mark(s) != hipSuccess) return MOE_ERR_HIP;
  // y = y_lat W_up^T + sum_s hs_s Wd_s^T: one accumulation over K segments
  moe::GemmDense o{};
  o.nseg = 1 + (int)S;
  o.seg[0] = {y_lat, ylat_ld, w->w_up_proj, L, (int)L};
  for (int sh = 0; sh < S; ++sh)
    o.seg[1 + sh] = {static_cast<const char*>(hs) + sh * Fs * eb, hs_ld,
                     static_cast<const char*>(w->ws_down) + sh * D * Fs * eb, Fs, (int)Fs};
  o.C = y;
  o.ldc = D;
  o.M = (int)T;
  o.N = (int)D;
  e = moe::launch_gemm_dense(dt, dt, o, s);
  if (e == hipSuccess) e = m->mark(s);
  return hip_status(e);
}

}  // namespace

MOE_API moe_status moe_forward(const moe_config* cfg, const moe_weights* w, const void* x, void* y,
                               const moe_taps* taps, int64_t* counts, void* ws, size_t ws_bytes,
                               void* stream) {
  return forward_impl(cfg, w, x, y, taps, counts, ws, ws_bytes, stream, nullptr, 0);
}

MOE_API moe_status moe_forward_profiled(const moe_config* cfg, const moe_weights* w, const void* x,
                                        void* y, const moe_taps* taps, int64_t* counts, void* ws,
                                        size_t ws_bytes, void* stream, void* const* stage_events,
                                        int32_t n_events) {
  if (n_events < 0 || (n_events > 0 && !stage_events)) return MOE_ERR_INVALID_ARG;
  for (int i = 0; i < n_events; ++i)
    if (!stage_events[i]) return MOE_ERR_INVALID_ARG;
  return forward_impl(cfg, w, x, y, taps, counts, ws, ws_bytes, stream, stage_events, n_events);
}

MOE_API int32_t moe_forward_stage_count(void) { return kStages; }

// ------------------------------------------------------------------ dropless
namespace {

constexpr int kDroplessStages = 11;

moe_status check_dropless(const moe_config* cfg, moe_plan* p) {
  moe_status st = plan_impl(cfg, p);
  if (st != MOE_OK) return st;
  if (cfg->dtype != MOE_BF16) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// xs null: only the rows' places are found.
moe_status run_dispatch_dropless(const moe_config* c, const moe_plan& p, const int32_t* topk, const void* z,
                                 void* xs, int32_t* row_of, int32_t* offsets, int64_t* counts, void* ws,
                                 hipStream_t s, Marks* m) {
  const int64_t n = p.dropless_rows;
  const int64_t nblk = moe::ragged_sort_blocks(n);
  Carver cv{static_cast<char*>(ws), 0};
  int32_t* hist = static_cast<int32_t*>(cv.take(nblk * c->n_experts * 4));
  int32_t* base = static_cast<int32_t*>(cv.take(nblk * c->n_experts * 4));
  hipError_t e = moe::launch_ragged_sort(topk, n, c->n_experts, hist, base, offsets, row_of, counts, s);
  if (e == hipSuccess && m) e = m->mark(s);
  if (e == hipSuccess && xs) e = moe::launch_ragged_scatter(z, row_of, c->T, c->top_k, p.row_bytes, xs, s);
  if (e == hipSuccess && m) e = m->mark(s);
  return hip_status(e);
}

moe_status run_experts_dropless(const moe_config* c, const moe_plan& p, const void* xs,
                                const int32_t* offsets, const void* wg, const void* wu, const void* wd,
                                void* out, void* ws, hipStream_t s, Marks* m) {
  int64_t ent0, ent1;
  dropless_entries(c, &ent0, &ent1);
  const int64_t n = p.dropless_rows;
  Carver cv{static_cast<char*>(ws), 0};
  int32_t* list0 = static_cast<int32_t*>(cv.take(ent0 * 12));
  int32_t* list1 = static_cast<int32_t*>(cv.take(ent1 * 12));
  int32_t* ntiles = static_cast<int32_t*>(cv.take(8));
  char* H = static_cast<char*>(cv.take(n * c->d_ff * p.elem_bytes));
  const int tn0 = (int)ceil_div(c->d_ff, moe::ragged_gate_up_cols());
  const int tn1 = (int)ceil_div(c->d_latent, moe::ragged_down_cols());
  hipError_t e = moe::launch_ragged_tiles(offsets, c->n_experts, moe::ragged_tile_rows(tall_tiles(c)), tn0, tn1,
                                          list0, list1, ntiles, s);
  if (e == hipSuccess && m) e = m->mark(s);
  if (e != hipSuccess) return MOE_ERR_HIP;
  moe::RaggedGemm g{};
  g.A = static_cast<const char*>(xs);
  g.a_row_bytes = p.row_bytes;
  g.offsets = offsets;
  g.list = list0;
  g.ntiles = ntiles;
  g.W0 = static_cast<const char*>(wg);
  g.W1 = static_cast<const char*>(wu);
  g.E = c->n_experts;
  g.F = c->d_ff;
  g.K = c->d_latent;
  g.N = 0;
  g.C = H;
  g.c_row_bytes = (int64_t)c->d_ff * p.elem_bytes;
  e = moe::launch_ragged_gate_up_bf16(g, ent0, tall_tiles(c), s);
  if (e == hipSuccess && m) e = m->mark(s);
  if (e != hipSuccess) return MOE_ERR_HIP;
  moe::RaggedGemm d{};
  d.A = H;
  d.a_row_bytes = (int64_t)c->d_ff * p.elem_bytes;
  d.offsets = offsets;
  d.list = list1;
  d.ntiles = ntiles + 1;
  d.W0 = static_cast<const char*>(wd);
  d.W1 = nullptr;
  d.E = c->n_experts;
  d.F = 0;
  d.K = c->d_ff;
  d.N = c->d_latent;
  d.C = static_cast<char*>(out);
  d.c_row_bytes = p.row_bytes;
  e = moe::launch_ragged_down_bf16(d, ent1, tall_tiles(c), s);
  if (e == hipSuccess && m) e = m->mark(s);
  return hip_status(e);
}

moe_status forward_dropless_impl(const moe_config* cfg, const moe_weights* w, const void* x, void* y,
                                 const moe_dropless_taps* taps, int64_t* counts, void* ws, size_t ws_bytes,
                                 void* stream, void* const* events, int n_events) {
  moe_plan p;
  moe_status st = check_dropless(cfg, &p);
  if (st != MOE_OK) return st;
  if (cfg->top_k > cfg->n_experts) return MOE_ERR_INVALID_ARG;
  if (cfg->n_experts % 4) return MOE_ERR_UNSUPPORTED;
  if (!w) return MOE_ERR_INVALID_ARG;
  if (!w->w_latent || !w->w_router || !w->w_gate || !w->w_up || !w->w_down || !w->w_up_proj)
    return MOE_ERR_INVALID_ARG;
  if (cfg->n_shared > 0 && (!w->ws_gate || !w->ws_up || !w->ws_down)) return MOE_ERR_INVALID_ARG;
  if (cfg->T > 0 && (!x || !y)) return MOE_ERR_INVALID_ARG;
  if (!ws || (int64_t)ws_bytes < p.dropless_forward_ws_bytes || !aligned256(ws)) return MOE_ERR_WORKSPACE;

  const moe_dropless_taps none{};
  const moe_dropless_taps& tp = taps ? *taps : none;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int64_t T = cfg->T, E = cfg->n_experts, k = cfg->top_k;
  const int64_t L = cfg->d_latent, D = cfg->d_model, S = cfg->n_shared, Fs = cfg->d_ff_shared;
  const int64_t eb = p.elem_bytes, n = p.dropless_rows;
  const int dt = cfg->dtype;

  Carver cv{static_cast<char*>(ws), 0};
  auto pick = [&](void* tap, int64_t bytes) {
    void* q = cv.take(bytes);
    return tap ? tap : q;
  };
  void* z = pick(tp.z, T * L * eb);
  float* logits = static_cast<float*>(pick(tp.logits, T * E * 4));
  int32_t* topk = static_cast<int32_t*>(pick(tp.topk_idx, T * k * 4));
  float* gates = static_cast<float*>(pick(tp.gates, T * k * 4));
  int32_t* row_of = static_cast<int32_t*>(pick(tp.row_of, T * k * 4));
  int32_t* offsets = static_cast<int32_t*>(pick(tp.expert_offsets, (E + 1) * 4));
  void* xs = pick(tp.xs, n * L * eb);
  void* out = pick(tp.expert_out, n * L * eb);
  void* y_lat = pick(tp.y_latent, T * L * eb);
  void* hs = cv.take(T * S * Fs * eb);
  // Without a y_latent tap, y_lat and the shared hidden rows are the two
  // column blocks of one [T][L + S*Fs] buffer (it fits in the two carves
  // above), so the output projection reads one A operand over all its K
  // ranges.
  int64_t ylat_ld = L, hs_ld = S * Fs;
  if (!tp.y_latent && S > 0 && T * (L + S * Fs) * eb < (int64_t(1) << 32)) {
    hs = static_cast<char*>(y_lat) + L * eb;
    ylat_ld = hs_ld = L + S * Fs;
  }
  int64_t* cnt = static_cast<int64_t*>(pick(counts, 3 * 8));
  void* dws = cv.take(p.dropless_dispatch_ws_bytes);
  void* xws = cv.take(p.dropless_experts_ws_bytes);

  Marks mk{events, n_events, 0};
  Marks* m = &mk;
  hipError_t e = m->mark(s);
  if (e != hipSuccess) return MOE_ERR_HIP;
  moe::GemmDense g{};
  g.nseg = 1;
  g.seg[0] = {x, D, w->w_latent, D, (int)D};
  g.C = z;
  g.ldc = L;
  g.M = (int)T;
  g.N = (int)L;
  e = moe::launch_gemm_dense(dt, dt, g, s);
  if (e == hipSuccess) e = m->mark(s);
  if (e != hipSuccess) return MOE_ERR_HIP;
  g.seg[0] = {z, L, w->w_router, L, (int)L};
  g.C = logits;
  g.ldc = E;
  g.N = (int)E;
  e = moe::launch_gemm_dense(dt, moe::DT_F32, g, s);
  if (e == hipSuccess) e = m->mark(s);
  if (e != hipSuccess) return MOE_ERR_HIP;
  e = moe::launch_topk_gates(logits, w->router_bias, T, (int)E, (int)k, topk, gates, s);
  if (e == hipSuccess) e = m->mark(s);
  if (e != hipSuccess) return MOE_ERR_HIP;
  st = run_dispatch_dropless(cfg, p, topk, z, xs, row_of, offsets, cnt, dws, s, m);
  if (st != MOE_OK) return st;
  st = run_experts_dropless(cfg, p, xs, offsets, w->w_gate, w->w_up, w->w_down, out, xws, s, m);
  if (st != MOE_OK) return st;
  e = moe::launch_ragged_combine(dt, out, row_of, gates, T, (int)k, p.row_bytes, y_lat, s, ylat_ld * eb);
  if (e == hipSuccess) e = m->mark(s);
  if (e != hipSuccess) return MOE_ERR_HIP;
  if (S > 0) {
    e = moe::launch_swiglu_dense(dt, x, D, w->ws_gate, w->ws_up, (int)S, (int)Fs, (int)D, (int)T, hs, hs_ld,
                                 s);
    if (e != hipSuccess) return MOE_ERR_HIP;
  }
  if (m->mark(s) != hipSuccess) return MOE_ERR_HIP;
  moe::GemmDense o{};
  o.nseg = 1 + (int)S;
  o.seg[0] = {y_lat, ylat_ld, w->w_up_proj, L, (int)L};
  for (int sh = 0; sh < S; ++sh)
    o.seg[1 + sh] = {static_cast<const char*>(hs) + sh * Fs * eb, hs_ld,
                     static_cast<const char*>(w->ws_down) + sh * D * Fs * eb, Fs, (int)Fs};
  o.C = y;
  o.ldc = D;
  o.M = (int)T;
  o.N = (int)D;
  e = moe::launch_gemm_dense(dt, dt, o, s);
  if (e == hipSuccess) e = m->mark(s);
  return hip_status(e);
}

}  // namespace

MOE_API moe_status moe_dispatch_dropless(const moe_config* cfg, const int32_t* topk_idx, const void* z,
                                         void* xs, int32_t* row_of, int32_t* expert_offsets,
                                         int64_t* counts, void* ws, size_t ws_bytes, void* stream) {
  moe_plan p;
  moe_status st = check_dropless(cfg, &p);
  if (st != MOE_OK) return st;
  if (!expert_offsets) return MOE_ERR_INVALID_ARG;
  if (cfg->T > 0 && (!topk_idx || !z || !xs || !row_of)) return MOE_ERR_INVALID_ARG;
  if (p.dropless_dispatch_ws_bytes > 0 &&
      (!ws || (int64_t)ws_bytes < p.dropless_dispatch_ws_bytes || !aligned256(ws)))
    return MOE_ERR_WORKSPACE;
  return run_dispatch_dropless(cfg, p, topk_idx, z, xs, row_of, expert_offsets, counts, ws,
                               static_cast<hipStream_t>(stream), nullptr);
}

MOE_API moe_status moe_experts_dropless(const moe_config* cfg, const void* xs, const int32_t* expert_offsets,
                                        const void* w_gate, const void* w_up, const void* w_down,
                                        void* expert_out, void* ws, size_t ws_bytes, void* stream) {
  moe_plan p;
  moe_status st = check_dropless(cfg, &p);
  if (st != MOE_OK) return st;
  if (!expert_offsets || !w_gate || !w_up || !w_down) return MOE_ERR_INVALID_ARG;
  if (cfg->T > 0 && (!xs || !expert_out)) return MOE_ERR_INVALID_ARG;
  if (!ws || (int64_t)ws_bytes < p.dropless_experts_ws_bytes || !aligned256(ws)) return MOE_ERR_WORKSPACE;
  return run_experts_dropless(cfg, p, xs, expert_offsets, w_gate, w_up, w_down, expert_out, ws,
                              static_cast<hipStream_t>(stream), nullptr);
}

MOE_API moe_status moe_combine_dropless(const moe_config* cfg, const void* expert_out, const int32_t* row_of,
                                        const float* gates, void* y_latent, void* stream) {
  moe_plan p;
  moe_status st = check_dropless(cfg, &p);
  if (st != MOE_OK) return st;
  if (cfg->T > 0 && (!expert_out || !row_of || !gates || !y_latent)) return MOE_ERR_INVALID_ARG;
  return hip_status(moe::launch_ragged_combine(cfg->dtype, expert_out, row_of, gates, cfg->T, cfg->top_k,
                                               p.row_bytes, y_latent, static_cast<hipStream_t>(stream)));
}

MOE_API moe_status moe_forward_dropless(const moe_config* cfg, const moe_weights* w, const void* x, void* y,
                                        const moe_dropless_taps* taps, int64_t* counts, void* ws,
                                        size_t ws_bytes, void* stream) {
  return forward_dropless_impl(cfg, w, x, y, taps, counts, ws, ws_bytes, stream, nullptr, 0);
}

MOE_API int32_t moe_forward_dropless_stage_count(void) { return kDroplessStages; }

MOE_API moe_status moe_forward_dropless_profiled(const moe_config* cfg, const moe_weights* w, const void* x,
                                                 void* y, const moe_dropless_taps* taps, int64_t* counts,
                                                 void* ws, size_t ws_bytes, void* stream,
                                                 void* const* stage_events, int32_t n_events) {
  if (n_events < 0 || (n_events > 0 && !stage_events)) return MOE_ERR_INVALID_ARG;
  for (int i = 0; i < n_events; ++i)
    if (!stage_events[i]) return MOE_ERR_INVALID_ARG;
  return forward_dropless_impl(cfg, w, x, y, taps, counts, ws, ws_bytes, stream, stage_events, n_events);
}

// ------------------------------------------------------------------ backward
namespace {

constexpr int kBackwardStages = 11;

moe_status check_backward(const moe_config* cfg, moe_plan* p) {
  moe_status st = plan_impl(cfg, p);
  if (st != MOE_OK) return st;
  if (cfg->dtype != MOE_BF16 || cfg->d_latent % 256 || cfg->d_ff % 256) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status run_combine_bwd(const moe_config* c, const moe_plan& p, const void* expert_out, const int32_t* topk,
                           const int32_t* pool_slot, const int32_t* recv_slot, const float* gates,
                           const void* dy, float* d_gates, void* d_expert_out, hipStream_t s) {
  moe::CombineBwdArgs a{};
  a.expert_out = expert_out;
  a.dy = dy;
  a.topk = topk;
  a.pool_slot = pool_slot;
  a.recv_slot = recv_slot;
  a.gates = gates;
  a.T = c->T;
  a.Tw = p.tokens_per_wave;
  a.k = c->top_k;
  a.E = c->n_experts;
  a.P = c->n_pools;
  a.cap_send = p.cap_send;
  a.row_bytes = p.row_bytes;
  a.d_gates = d_gates;
  a.d_expert_out = d_expert_out;
  return hip_status(moe::launch_combine_bwd(a, s));
}

// Where the experts' backward finds its rows: the capped path's pools and
// bank lists, or the dropless variant's expert-ordered buffers.
struct BwdRows {
  const int32_t* bank_rows;       // capped
  const int32_t* expert_count;
  const int32_t* expert_offsets;  // dropless (non-NULL selects it)
  const void* u;                  // pools, or xs
  const void* d_out;              // d_expert_out
  void* d_in;                     // du out: d_pool_rows, or d_xs
};

moe_status run_experts_bwd(const moe_config* c, const moe_plan& p, const BwdRows& src, const void* wg, const void* wu,
                           const void* wd, void* dwg, void* dwu, void* dwd, void* ws, hipStream_t s, Marks* m) {
  const int E = c->n_experts;
  const bool ragged = src.expert_offsets != nullptr;
  const int64_t L = c->d_latent, F = c->d_ff, R = ragged ? p.dropless_backward_rows : p.backward_rows;
  int64_t epre, edh, edu;
  backward_entries(c, R, &epre, &edh, &edu);
  Carver cv{static_cast<char*>(ws), 0};
  int32_t* counts = static_cast<int32_t*>(cv.take(E * 4));
  int32_t* offsets = static_cast<int32_t*>(cv.take((int64_t)(E + 1) * 4));
  int32_t* gidx = static_cast<int32_t*>(cv.take(R * 4));
  int32_t* list_pre = static_cast<int32_t*>(cv.take(epre * 12));
  int32_t* list_dh = static_cast<int32_t*>(cv.take(edh * 12));
  int32_t* list_du = static_cast<int32_t*>(cv.take(edu * 12));
  int32_t* ntiles = static_cast<int32_t*>(cv.take(16));
  char* U = static_cast<char*>(cv.take(R * L * 2));
  char* DO = static_cast<char*>(cv.take(R * L * 2));
  char* DH = static_cast<char*>(cv.take(R * F * 2));
  char* DADB = static_cast<char*>(cv.take(R * 2 * F * 2));
  char* H = static_cast<char*>(cv.take(R * F * 2));
  // one M-tile structure serves the recompute (expert tile) and dh (dgrad
  // tile) lists, so the two tiles must have the same row count
  const int bm = moe::bwd_dgrad_rows();
  if (bm != moe::ragged_tile_rows(false)) return MOE_ERR_UNSUPPORTED;
  hipError_t e = ragged ? moe::launch_bwd_layout_ragged(src.expert_offsets, E, p.dropless_rows, counts, offsets,
                                                         gidx, s)
                        : moe::launch_bwd_layout(src.bank_rows, src.expert_count, E, c->n_pools, c->n_waves,
                                                 p.cap_send, p.cap_recv, counts, offsets, gidx, s);
  if (e == hipSuccess)
    e = moe::launch_ragged_tiles(offsets, E, bm, (int)ceil_div(F, moe::ragged_gate_up_cols()),
                                 (int)ceil_div(F, moe::bwd_dgrad_cols()), list_pre, list_dh, ntiles, s);
  if (e == hipSuccess)
    e = moe::launch_ragged_tiles(offsets, E, bm, (int)ceil_div(L, moe::bwd_dgrad_cols()), 0, list_du, list_du,
                                 ntiles + 2, s);
  if (e == hipSuccess && m) e = m->mark(s);
  // u and do rows in the padded expert-major order (zero padding rows)
  const int one_block = 0x7fffffff;  // the dropless buffers are one block of rows
  if (e == hipSuccess)
    e = ragged ? moe::launch_gather_rows(src.u, one_block, 0, p.row_bytes, gidx, offsets + E, R, U, s)
               : moe::launch_gather_rows(src.u, (int)p.cap_send, p.pool_block_bytes, p.row_bytes, gidx, offsets + E,
                                         R, U, s);
  if (e == hipSuccess)
    e = ragged ? moe::launch_gather_rows(src.d_out, one_block, 0, p.row_bytes, gidx, offsets + E, R, DO, s)
               : moe::launch_gather_rows(src.d_out, (int)p.cap_send, p.cap_send * p.row_bytes, p.row_bytes, gidx,
                                         offsets + E, R, DO, s);
  if (e == hipSuccess && m) e = m->mark(s);
  if (e != hipSuccess) return MOE_ERR_HIP;
  // dh = do W_d
  moe::BwdDgrad d{};
  d.A = DO;
  d.a_row_bytes = L * 2;
  d.offsets = offsets;
  d.counts = counts;
  d.list = list_dh;
  d.ntiles = ntiles + 1;
  d.W0 = static_cast<const char*>(wd);
  d.E = E;
  d.K = (int)L;
  d.N = (int)F;
  d.F = (int)F;
  d.C = DH;
  d.c_row_bytes = F * 2;
  e = moe::launch_bwd_dh(d, edh, s);
  if (e == hipSuccess && m) e = m->mark(s);
  if (e != hipSuccess) return MOE_ERR_HIP;
  // recompute a = u W_g^T, b = u W_u^T; SwiGLU backward: da, db, h
  moe::RaggedGemm g{};
  g.A = U;
  g.a_row_bytes = L * 2;
  g.offsets = offsets;
  g.list = list_pre;
  g.ntiles = ntiles;
  g.W0 = static_cast<const char*>(wg);
  g.W1 = static_cast<const char*>(wu);
  g.E = E;
  g.F = (int)F;
  g.K = (int)L;
  g.C = DADB;
  g.c_row_bytes = 2 * F * 2;
  g.dH = DH;
  g.dh_row_bytes = F * 2;
  g.H = H;
  g.h_row_bytes = F * 2;
  e = moe::launch_ragged_swiglu_bwd_bf16(g, epre, s);
  if (e == hipSuccess && m) e = m->mark(s);
  if (e != hipSuccess) return MOE_ERR_HIP;
  // du = da W_g + db W_u, rows back to their pool slots
  moe::BwdDgrad u{};
  u.A = DADB;
  u.a_row_bytes = 2 * F * 2;
  u.a_seg_bytes = F * 2;
  u.offsets = offsets;
  u.counts = counts;
  u.list = list_du;
  u.ntiles = ntiles + 2;
  u.W0 = static_cast<const char*>(wg);
  u.W1 = static_cast<const char*>(wu);
  u.E = E;
  u.K = (int)F;
  u.N = (int)L;
  u.F = (int)F;
  u.C = static_cast<char*>(src.d_in);
  u.c_row_bytes = p.row_bytes;
  u.c_index = gidx;
  e = moe::launch_bwd_du(u, edu, s);
  if (e == hipSuccess && m) e = m->mark(s);
  if (e != hipSuccess) return MOE_ERR_HIP;
  // weight gradients over each expert's padded rows
  const int tile = moe::bwd_wgrad_tile();
  auto wgrad = [&](const char* X, int64_t xr, int64_t xc, const char* Y, int64_t yr, int M, int N, void* C) {
    moe::BwdWgrad w{};
    w.X = X;
    w.x_row_bytes = xr;
    w.x_col_bytes = xc;
    w.Y = Y;
    w.y_row_bytes = yr;
    w.y_col_bytes = 0;
    w.offsets = offsets;
    w.counts = counts;
    w.E = E;
    w.M = M;
    w.N = N;
    w.tiles_m = M / tile;
    w.tiles_n = N / tile;
    w.C = static_cast<char*>(C);
    hipError_t r = moe::launch_bwd_wgrad(w, s);
    if (r == hipSuccess && m) r = m->mark(s);
    return r;
  };
  e = wgrad(DO, L * 2, 0, H, F * 2, (int)L, (int)F, dwd);
  if (e == hipSuccess) e = wgrad(DADB, 2 * F * 2, 0, U, L * 2, (int)F, (int)L, dwg);
  if (e == hipSuccess) e = wgrad(DADB, 2 * F * 2, F * 2, U, L * 2, (int)F, (int)L, dwu);
  return hip_status(e);
}

moe_status run_dispatch_bwd(const moe_config* c, const moe_plan& p, const int32_t* topk, const int32_t* pool_slot,
                            const int32_t* recv_slot, const void* d_pool_rows, void* dz, hipStream_t s) {
  return run_combine(c, p, d_pool_rows, topk, pool_slot, recv_slot, nullptr, dz, s);
}

moe_status backward_impl(const moe_config* cfg, const moe_weights* w, const moe_taps* sv, const void* dy,
                         void* dz, float* d_logits, void* dwg, void* dwu, void* dwd, void* ws, size_t ws_bytes,
                         void* stream, void* const* events, int n_events) {
  moe_plan p;
  moe_status st = check_backward(cfg, &p);
  if (st != MOE_OK) return st;
  if (!w || !sv || !w->w_gate || !w->w_up || !w->w_down || !dwg || !dwu || !dwd || !sv->expert_count)
    return MOE_ERR_INVALID_ARG;
  // pool-shaped buffers are empty when a capacity is 0: then they may be null
  if ((p.pools_bytes > 0 && (!sv->pools || !sv->expert_out)) || (p.cap_recv > 0 && !sv->bank_rows))
    return MOE_ERR_INVALID_ARG;
  if (cfg->T > 0 && (!sv->topk_idx || !sv->gates || !sv->pool_slot || !sv->recv_slot || !dy || !dz || !d_logits))
    return MOE_ERR_INVALID_ARG;
  if (!ws || (int64_t)ws_bytes < p.backward_ws_bytes || !aligned256(ws)) return MOE_ERR_WORKSPACE;
  hipStream_t s = static_cast<hipStream_t>(stream);
  Marks marks{events, n_events, 0};
  Marks* m = events ? &marks : nullptr;
  Carver cv{static_cast<char*>(ws), 0};
  const int64_t T = cfg->T, k = cfg->top_k;
  float* d_gates = static_cast<float*>(cv.take(T * k * 4));
  void* d_expert_out = cv.take(p.expert_out_bytes);
  void* d_pool_rows = cv.take(p.expert_out_bytes);
  void* ews = cv.take(p.experts_bwd_ws_bytes);
  hipError_t e = m ? m->mark(s) : hipSuccess;
  if (e != hipSuccess) return MOE_ERR_HIP;
  st = run_combine_bwd(cfg, p, sv->expert_out, sv->topk_idx, sv->pool_slot, sv->recv_slot, sv->gates, dy, d_gates,
                       d_expert_out, s);
  if (st == MOE_OK && m) st = hip_status(m->mark(s));
  if (st == MOE_OK) {
    const BwdRows src{sv->bank_rows, sv->expert_count, nullptr, sv->pools, d_expert_out, d_pool_rows};
    st = run_experts_bwd(cfg, p, src, w->w_gate, w->w_up, w->w_down, dwg, dwu, dwd, ews, s, m);
  }
  if (st == MOE_OK)
    st = run_dispatch_bwd(cfg, p, sv->topk_idx, sv->pool_slot, sv->recv_slot, d_pool_rows, dz, s);
  if (st == MOE_OK && m) st = hip_status(m->mark(s));
  if (st == MOE_OK)
    st = hip_status(moe::launch_route_bwd(sv->topk_idx, sv->gates, d_gates, T, (int)k, cfg->n_experts, d_logits, s));
  if (st == MOE_OK && m) st = hip_status(m->mark(s));
  return st;
}

}  // namespace

MOE_API moe_status moe_combine_backward(const moe_config* cfg, const void* expert_out, const int32_t* topk_idx,
                                        const int32_t* pool_slot, const int32_t* recv_slot, const float* gates,
                                        const void* dy_latent, float* d_gates, void* d_expert_out, void* stream) {
  moe_plan p;
  moe_status st = check_backward(cfg, &p);
  if (st != MOE_OK) return st;
  if (cfg->T > 0 && ((p.expert_out_bytes > 0 && (!expert_out || !d_expert_out)) || !topk_idx || !pool_slot ||
                     !recv_slot || !gates || !dy_latent || !d_gates))
    return MOE_ERR_INVALID_ARG;
  return run_combine_bwd(cfg, p, expert_out, topk_idx, pool_slot, recv_slot, gates, dy_latent, d_gates,
                         d_expert_out, static_cast<hipStream_t>(stream));
}

MOE_API moe_status moe_experts_backward(const moe_config* cfg, const void* pools, const int32_t* bank_rows,
                                        const int32_t* expert_count, const void* w_gate, const void* w_up,
                                        const void* w_down, const void* d_expert_out, void* d_pool_rows,
                                        void* dw_gate, void* dw_up, void* dw_down, void* ws, size_t ws_bytes,
                                        void* stream) {
  moe_plan p;
  moe_status st = check_backward(cfg, &p);
  if (st != MOE_OK) return st;
  if (!expert_count || !w_gate || !w_up || !w_down || !dw_gate || !dw_up || !dw_down) return MOE_ERR_INVALID_ARG;
  if ((p.pools_bytes > 0 && (!pools || !d_expert_out || !d_pool_rows)) || (p.cap_recv > 0 && !bank_rows))
    return MOE_ERR_INVALID_ARG;
  if (!ws || (int64_t)ws_bytes < p.experts_bwd_ws_bytes || !aligned256(ws)) return MOE_ERR_WORKSPACE;
  const BwdRows src{bank_rows, expert_count, nullptr, pools, d_expert_out, d_pool_rows};
  return run_experts_bwd(cfg, p, src, w_gate, w_up, w_down, dw_gate, dw_up, dw_down, ws,
                         static_cast<hipStream_t>(stream), nullptr);
}

MOE_API moe_status moe_dispatch_backward(const moe_config* cfg, const int32_t* topk_idx, const int32_t* pool_slot,
                                         const int32_t* recv_slot, const void* d_pool_rows, void* dz,
                                         void* stream) {
  moe_plan p;
  moe_status st = check_backward(cfg, &p);
  if (st != MOE_OK) return st;
  if (cfg->T > 0 && (!topk_idx || !pool_slot || !recv_slot || (p.expert_out_bytes > 0 && !d_pool_rows) || !dz))
    return MOE_ERR_INVALID_ARG;
  return run_dispatch_bwd(cfg, p, topk_idx, pool_slot, recv_slot, d_pool_rows, dz,
                          static_cast<hipStream_t>(stream));
}

MOE_API moe_status moe_route_backward(const moe_config* cfg, const int32_t* topk_idx, const float* gates,
                                      const float* d_gates, float* d_logits, void* stream) {
  moe_status st = check_route_shape(cfg);
  if (st != MOE_OK) return st;
  if (cfg->T > 0 && (!topk_idx || !gates || !d_gates || !d_logits)) return MOE_ERR_INVALID_ARG;
  return hip_status(moe::launch_route_bwd(topk_idx, gates, d_gates, cfg->T, cfg->top_k, cfg->n_experts, d_logits,
                                          static_cast<hipStream_t>(stream)));
}

MOE_API moe_status moe_backward_routed(const moe_config* cfg, const moe_weights* w, const moe_taps* saved,
                                       const void* dy_latent, void* dz, float* d_logits, void* dw_gate,
                                       void* dw_up, void* dw_down, void* ws, size_t ws_bytes, void* stream) {
  return backward_impl(cfg, w, saved, dy_latent, dz, d_logits, dw_gate, dw_up, dw_down, ws, ws_bytes, stream,
                       nullptr, 0);
}

MOE_API int32_t moe_backward_routed_stage_count(void) { return kBackwardStages; }

MOE_API moe_status moe_backward_routed_profiled(const moe_config* cfg, const moe_weights* w, const moe_taps* saved,
                                                const void* dy_latent, void* dz, float* d_logits, void* dw_gate,
                                                void* dw_up, void* dw_down, void* ws, size_t ws_bytes,
                                                void* stream, void* const* stage_events, int32_t n_events) {
  if (n_events < 0 || (n_events > 0 && !stage_events)) return MOE_ERR_INVALID_ARG;
  for (int i = 0; i < n_events; ++i)
    if (!stage_events[i]) return MOE_ERR_INVALID_ARG;
  return backward_impl(cfg, w, saved, dy_latent, dz, d_logits, dw_gate, dw_up, dw_down, ws, ws_bytes, stream,
                       stage_events, n_events);
}

// ------------------------------------------------------------------ dropless backward
namespace {

moe_status run_combine_bwd_dropless(const moe_config* c, const moe_plan& p, const void* expert_out,
                                    const int32_t* row_of, const float* gates, const void* dy, float* d_gates,
                                    void* d_expert_out, hipStream_t s) {
  moe::CombineBwdArgs a{};
  a.expert_out = expert_out;
  a.dy = dy;
  a.row_of = row_of;
  a.gates = gates;
  a.T = c->T;
  a.Tw = p.tokens_per_wave > 0 ? p.tokens_per_wave : 1;
  a.k = c->top_k;
  a.E = c->n_experts;
  a.P = c->n_pools;
  a.cap_send = p.cap_send;
  a.row_bytes = p.row_bytes;
  a.d_gates = d_gates;
  a.d_expert_out = d_expert_out;
  return hip_status(moe::launch_combine_bwd(a, s));
}

moe_status backward_dropless_impl(const moe_config* cfg, const moe_weights* w, const moe_dropless_taps* sv,
                                  const void* dy, void* dz, float* d_logits, void* dwg, void* dwu, void* dwd,
                                  void* ws, size_t ws_bytes, void* stream, void* const* events, int n_events) {
  moe_plan p;
  moe_status st = check_backward(cfg, &p);
  if (st != MOE_OK) return st;
  if (!w || !sv || !w->w_gate || !w->w_up || !w->w_down || !dwg || !dwu || !dwd || !sv->expert_offsets)
    return MOE_ERR_INVALID_ARG;
  if (cfg->T > 0 && (!sv->topk_idx || !sv->gates || !sv->row_of || !sv->xs || !sv->expert_out || !dy || !dz ||
                     !d_logits))
    return MOE_ERR_INVALID_ARG;
  if (!ws || (int64_t)ws_bytes < p.dropless_backward_ws_bytes || !aligned256(ws)) return MOE_ERR_WORKSPACE;
  hipStream_t s = static_cast<hipStream_t>(stream);
  Marks marks{events, n_events, 0};
  Marks* m = events ? &marks : nullptr;
  Carver cv{static_cast<char*>(ws), 0};
  const int64_t T = cfg->T, k = cfg->top_k, n = p.dropless_rows;
  float* d_gates = static_cast<float*>(cv.take(T * k * 4));
  void* d_expert_out = cv.take(n * p.row_bytes);
  void* d_xs = cv.take(n * p.row_bytes);
  void* ews = cv.take(p.dropless_experts_bwd_ws_bytes);
  hipError_t e = m ? m->mark(s) : hipSuccess;
  if (e != hipSuccess) return MOE_ERR_HIP;
  st = run_combine_bwd_dropless(cfg, p, sv->expert_out, sv->row_of, sv->gates, dy, d_gates, d_expert_out, s);
  if (st == MOE_OK && m) st = hip_status(m->mark(s));
  if (st == MOE_OK) {
    const BwdRows src{nullptr, nullptr, sv->expert_offsets, sv->xs, d_expert_out, d_xs};
    st = run_experts_bwd(cfg, p, src, w->w_gate, w->w_up, w->w_down, dwg, dwu, dwd, ews, s, m);
  }
  if (st == MOE_OK)
    st = hip_status(moe::launch_ragged_combine(cfg->dtype, d_xs, sv->row_of, nullptr, T, (int)k, p.row_bytes, dz, s));
  if (st == MOE_OK && m) st = hip_status(m->mark(s));
  if (st == MOE_OK)
    st = hip_status(moe::launch_route_bwd(sv->topk_idx, sv->gates, d_gates, T, (int)k, cfg->n_experts, d_logits, s));
  if (st == MOE_OK && m) st = hip_status(m->mark(s));
  return st;
}

}  // namespace

MOE_API moe_status moe_combine_backward_dropless(const moe_config* cfg, const void* expert_out,
                                                 const int32_t* row_of, const float* gates, const void* dy_latent,
                                                 float* d_gates, void* d_expert_out, void* stream) {
  moe_plan p;
  moe_status st = check_backward(cfg, &p);
  if (st != MOE_OK) return st;
  if (cfg->T > 0 && (!expert_out || !row_of || !gates || !dy_latent || !d_gates || !d_expert_out))
    return MOE_ERR_INVALID_ARG;
  return run_combine_bwd_dropless(cfg, p, expert_out, row_of, gates, dy_latent, d_gates, d_expert_out,
                                  static_cast<hipStream_t>(stream));
}

MOE_API moe_status moe_experts_backward_dropless(const moe_config* cfg, const void* xs, const int32_t* expert_offsets,
                                                 const void* w_gate, const void* w_up, const void* w_down,
                                                 const void* d_expert_out, void* d_xs, void* dw_gate, void* dw_up,
                                                 void* dw_down, void* ws, size_t ws_bytes, void* stream) {
  moe_plan p;
  moe_status st = check_backward(cfg, &p);
  if (st != MOE_OK) return st;
  if (!expert_offsets || !w_gate || !w_up || !w_down || !dw_gate || !dw_up || !dw_down) return MOE_ERR_INVALID_ARG;
  if (cfg->T > 0 && (!xs || !d_expert_out || !d_xs)) return MOE_ERR_INVALID_ARG;
  if (!ws || (int64_t)ws_bytes < p.dropless_experts_bwd_ws_bytes || !aligned256(ws)) return MOE_ERR_WORKSPACE;
  const BwdRows src{nullptr, nullptr, expert_offsets, xs, d_expert_out, d_xs};
  return run_experts_bwd(cfg, p, src, w_gate, w_up, w_down, dw_gate, dw_up, dw_down, ws,
                         static_cast<hipStream_t>(stream), nullptr);
}

MOE_API moe_status moe_dispatch_backward_dropless(const moe_config* cfg, const int32_t* row_of, const void* d_xs,
                                                  void* dz, void* stream) {
  moe_plan p;
  moe_status st = check_backward(cfg, &p);
  if (st != MOE_OK) return st;
  if (cfg->T > 0 && (!row_of || !d_xs || !dz)) return MOE_ERR_INVALID_ARG;
  return hip_status(moe::launch_ragged_combine(cfg->dtype, d_xs, row_of, nullptr, cfg->T, cfg->top_k, p.row_bytes,
                                               dz, static_cast<hipStream_t>(stream)));
}

MOE_API moe_status moe_backward_dropless(const moe_config* cfg, const moe_weights* w, const moe_dropless_taps* saved,
                                         const void* dy_latent, void* dz, float* d_logits, void* dw_gate,
                                         void* dw_up, void* dw_down, void* ws, size_t ws_bytes, void* stream) {
  return backward_dropless_impl(cfg, w, saved, dy_latent, dz, d_logits, dw_gate, dw_up, dw_down, ws, ws_bytes,
                                stream, nullptr, 0);
}

MOE_API moe_status moe_backward_dropless_profiled(const moe_config* cfg, const moe_weights* w,
                                                  const moe_dropless_taps* saved, const void* dy_latent, void* dz,
                                                  float* d_logits, void* dw_gate, void* dw_up, void* dw_down,
                                                  void* ws, size_t ws_bytes, void* stream,
                                                  void* const* stage_events, int32_t n_events) {
  if (n_events < 0 || (n_events > 0 && !stage_events)) return MOE_ERR_INVALID_ARG;
  for (int i = 0; i < n_events; ++i)
    if (!stage_events[i]) return MOE_ERR_INVALID_ARG;
  return backward_dropless_impl(cfg, w, saved, dy_latent, dz, d_logits, dw_gate, dw_up, dw_down, ws, ws_bytes,
                                stream, stage_events, n_events);
}

// ------------------------------------------------------------------ scored routing
namespace {

constexpr int kMaxGroups = 64;  // one lane of a wavefront per group
constexpr int64_t kMaxScoredTokens = (int64_t(1) << 26) - 4;  // 64 threads each, below 2^32 in a launch

moe_status check_scoring(const moe_config* c, const moe_scoring* sc, moe::ScoreArgs* a) {
  moe_status st = check_route_shape(c);
  if (st != MOE_OK) return st;
  if (!sc || c->top_k > c->n_experts) return MOE_ERR_INVALID_ARG;
  if (sc->score != MOE_SCORE_SOFTMAX && sc->score != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID_ARG;
  if (sc->n_groups < 1 || c->n_experts % sc->n_groups || sc->top_groups < 1 || sc->top_groups > sc->n_groups ||
      sc->group_top < 1 || sc->group_top > 2)
    return MOE_ERR_INVALID_ARG;
  if (sc->top_groups * (c->n_experts / sc->n_groups) < c->top_k) return MOE_ERR_INVALID_ARG;
  if ((sc->renormalise != 0 && sc->renormalise != 1) || sc->reserved != 0) return MOE_ERR_INVALID_ARG;
  if (!(sc->scale - sc->scale == 0.0f)) return MOE_ERR_INVALID_ARG;  // an infinity or a NaN
  if (sc->n_groups > kMaxGroups || c->T > kMaxScoredTokens) return MOE_ERR_UNSUPPORTED;
  a->T = c->T;
  a->E = c->n_experts;
  a->k = c->top_k;
  a->sigmoid = sc->score == MOE_SCORE_SIGMOID;
  a->groups = sc->top_groups == sc->n_groups ? 1 : sc->n_groups;  // every group kept: no limit
  a->top_groups = a->groups == 1 ? 1 : sc->top_groups;
  a->group_top = sc->group_top;
  a->renorm = sc->renormalise;
  a->scale = sc->scale;
  return MOE_OK;
}

}  // namespace

MOE_API moe_status moe_route_scored(const moe_config* cfg, const moe_scoring* scoring, const float* logits,
                                    const float* bias, int32_t* topk_idx, float* gates, void* stream) {
  moe::ScoreArgs a{};
  moe_status st = check_scoring(cfg, scoring, &a);
  if (st != MOE_OK) return st;
  if (cfg->T > 0 && (!logits || !topk_idx || !gates)) return MOE_ERR_INVALID_ARG;
  return hip_status(moe::launch_route_scored(a, logits, bias, topk_idx, gates, static_cast<hipStream_t>(stream)));
}

MOE_API moe_status moe_route_scored_backward(const moe_config* cfg, const moe_scoring* scoring, const float* logits,
                                             const int32_t* topk_idx, const float* d_gates, float* d_logits,
                                             void* stream) {
  moe::ScoreArgs a{};
  moe_status st = check_scoring(cfg, scoring, &a);
  if (st != MOE_OK) return st;
  if (cfg->T > 0 && (!logits || !topk_idx || !d_gates || !d_logits)) return MOE_ERR_INVALID_ARG;
  return hip_status(
      moe::launch_route_scored_bwd(a, logits, topk_idx, d_gates, d_logits, static_cast<hipStream_t>(stream)));
}

// ------------------------------------------------------------------ block-scaled e4m3
namespace {

constexpr int64_t kMaxQuantTiles = (int64_t(1) << 24) - 1;  // 256-thread workgroups of one launch
constexpr int64_t kMaxQuantRows = int64_t(1) << 30;         // rows of an operand of moe_gemm_quant
constexpr int64_t kMaxQuantK = int64_t(1) << 23;            // 256 rows of K bytes stay below 2^31

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool aligned_to(const void* p, int64_t n) { return reinterpret_cast<uintptr_t>(p) % (uintptr_t)n == 0; }
int64_t align128(int64_t x) { return (x + 127) & ~int64_t(127); }

moe_status check_gemm_quant(const moe_quant_gemm* q, moe::QuantGemm* g) {
  if (!q) return MOE_ERR_INVALID_ARG;
  if (q->M < 0 || q->N < 0 || q->K < 0 || q->reserved != 0) return MOE_ERR_INVALID_ARG;
  if (q->out_dtype != MOE_F32 && q->out_dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
  if (q->b_block_rows != 1 && q->b_block_rows != 128) return MOE_ERR_INVALID_ARG;
  if (q->K % 128) return MOE_ERR_INVALID_ARG;
  if (q->M > kMaxQuantRows || q->N > kMaxQuantRows || q->K > kMaxQuantK ||
      ceil_div(q->M, 128) * ceil_div(q->N, 128) > kMaxListEntries)
    return MOE_ERR_UNSUPPORTED;
  const int64_t kb = q->K / 128;
  const int64_t nb = q->b_block_rows == 128 ? kb : q->N;
  if (q->lda < q->K || q->ldb < q->K || q->ldc < q->N || q->a_scale_ld < q->M || q->b_scale_ld < nb)
    return MOE_ERR_INVALID_ARG;
  if (q->lda > kMaxQuantK || q->ldb > kMaxQuantK) return MOE_ERR_UNSUPPORTED;
  if (q->lda % 16 || q->ldb % 16) return MOE_ERR_UNSUPPORTED;
  g->lda = q->lda;
  g->a_scale_ld = q->a_scale_ld;
  g->ldb = q->ldb;
  g->b_scale_ld = q->b_scale_ld;
  g->b_rows = q->b_block_rows;
  g->M = q->M;
  g->N = q->N;
  g->K = (int)q->K;
  g->out_dt = q->out_dtype;
  g->ldc = q->ldc;
  return MOE_OK;
}

// Grouped SwiGLU in e4m3 over expert-ordered bf16 rows: its workspace.
struct QuantExpertsWs {
  char* xq;   // quantised rows
  float* xs;  // and their scales
  char* hq;   // quantised hidden rows
  float* hs;
  float* h;   // few rows per expert: hidden rows in fp32
};
int64_t carve_experts_quant(const moe_config* c, int64_t n, void* ws, QuantExpertsWs* w) {
  const int64_t L = c->d_latent, F = c->d_ff;
  const bool few = moe::few_rows(n, c->n_experts, true);
  Carver cv{static_cast<char*>(ws), 0};
  w->xq = static_cast<char*>(cv.take(n * L));
  w->xs = static_cast<float*>(cv.take(n * (L / 128) * 4));
  w->hq = static_cast<char*>(cv.take(n * F));
  w->hs = static_cast<float*>(cv.take(n * (F / 128) * 4));
  w->h = static_cast<float*>(cv.take(few ? n * F * 4 : 0));
  return cv.used;
}

moe_status check_quant_config(const moe_config* cfg, moe_plan* p) {
  moe_status st = check_dropless(cfg, p);
  if (st != MOE_OK) return st;
  if (cfg->d_latent % 128 || cfg->d_ff % 128) return MOE_ERR_UNSUPPORTED;
  // tiles of 64 rows x 128 columns at the least
  const int64_t widest = cfg->d_latent > cfg->d_ff ? cfg->d_latent : cfg->d_ff;
  if ((ceil_div(p->dropless_rows, 64) + cfg->n_experts) * (widest / 128) > kMaxListEntries) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// xs null: the workspace's xq and xs hold the quantised rows already (not
// where few_rows).
moe_status run_experts_quant(const moe_config* c, const moe_plan& p, const void* xs, const int32_t* offsets,
                             const moe_quant_experts* w, void* out, void* ws, hipStream_t s) {
  const int64_t n = p.dropless_rows, L = c->d_latent, F = c->d_ff;
  QuantExpertsWs q;
  carve_experts_quant(c, n, ws, &q);
  auto quantize = [&](const void* x, int dt, int64_t K, char* to, float* scale) {
    moe::QuantizeArgs z{};
    z.x = x;
    z.rows = n;
    z.cols = z.ld = z.ldq = K;
    z.dt = dt;
    z.block_rows = 1;
    z.q = to;
    z.scale = scale;
    z.scale_ld = n;
    return moe::launch_quantize(z, s);
  };
  hipError_t e;
  if (moe::few_rows(n, c->n_experts, true)) {
    // a token's ids differ, so an expert has at most T rows (more are taken
    // in further passes): fewer staged rows leave room for more workgroups
    const int chunk = (int)(c->T < 16 ? c->T : 16);
    const bool stage_x = moe::few_rows_stage((int)L), stage_h = moe::few_rows_stage((int)F);
    if (!stage_x) {
      e = quantize(xs, moe::DT_BF16, L, q.xq, q.xs);
      if (e != hipSuccess) return MOE_ERR_HIP;
    }
    moe::FewRows u{};
    u.x = stage_x ? xs : q.xq;
    u.ldx = L;
    u.x_scale = q.xs;
    u.x_scale_ld = n;
    u.W0 = static_cast<const char*>(w->q_gate);
    u.s0 = w->s_gate;
    u.W1 = static_cast<const char*>(w->q_up);
    u.s1 = w->s_up;
    u.M = n;
    u.E = c->n_experts;
    u.N = (int)F;
    u.K = (int)L;
    u.chunk = chunk;
    u.offsets = offsets;
    u.out = q.h;
    u.ldo = F;
    e = moe::launch_few_rows(u, true, stage_x, s);
    if (e != hipSuccess) return MOE_ERR_HIP;
    if (!stage_h) {
      e = quantize(q.h, moe::DT_F32, F, q.hq, q.hs);
      if (e != hipSuccess) return MOE_ERR_HIP;
    }
    moe::FewRows d{};
    d.x = stage_h ? static_cast<const void*>(q.h) : q.hq;
    d.ldx = F;
    d.x_scale = q.hs;
    d.x_scale_ld = n;
    d.W0 = static_cast<const char*>(w->q_down);
    d.s0 = w->s_down;
    d.M = n;
    d.E = c->n_experts;
    d.N = (int)L;
    d.K = (int)F;
    d.chunk = chunk;
    d.offsets = offsets;
    d.out = out;
    d.ldo = L;
    return hip_status(moe::launch_few_rows(d, false, stage_h, s));
  }
  e = xs ? quantize(xs, moe::DT_BF16, L, q.xq, q.xs) : hipSuccess;
  if (e != hipSuccess) return MOE_ERR_HIP;
  moe::QuantGateUp u{};
  u.A = q.xq;
  u.lda = L;
  u.a_scale = q.xs;
  u.a_scale_ld = n;
  u.Wg = static_cast<const char*>(w->q_gate);
  u.sg = w->s_gate;
  u.Wu = static_cast<const char*>(w->q_up);
  u.su = w->s_up;
  u.M = n;
  u.E = c->n_experts;
  u.F = (int)F;
  u.K = (int)L;
  u.offsets = offsets;
  u.H = q.hq;
  u.ldh = F;
  u.h_scale = q.hs;
  u.h_scale_ld = n;
  e = moe::launch_quant_gate_up(u, s);
  if (e != hipSuccess) return MOE_ERR_HIP;
  moe::QuantGemm d{};
  d.A = q.hq;
  d.lda = F;
  d.a_scale = q.hs;
  d.a_scale_ld = n;
  d.B = static_cast<const char*>(w->q_down);
  d.ldb = F;
  d.b_scale = w->s_down;
  d.b_scale_ld = F / 128;
  d.b_rows = 128;
  d.M = n;
  d.N = L;
  d.K = (int)F;
  d.out_dt = moe::DT_BF16;
  d.C = out;
  d.ldc = L;
  d.offsets = offsets;
  d.E = c->n_experts;
  d.b_stride = L * F;
  d.b_scale_stride = (L / 128) * (F / 128);
  return hip_status(moe::launch_quant_gemm(d, nullptr, s));
}

bool quant_experts_valid(const moe_quant_experts* w) {
  return w && w->q_gate && w->s_gate && w->q_up && w->s_up && w->q_down && w->s_down && aligned16(w->q_gate) &&
         aligned16(w->q_up) && aligned16(w->q_down);
}

}  // namespace

MOE_API moe_status moe_quantize(int64_t rows, int64_t cols, const void* x, int64_t ldx, int32_t dtype,
                                int32_t block_rows, int32_t transpose, void* q, float* scales, void* stream) {
  if (rows < 0 || cols < 0 || ldx < cols) return MOE_ERR_INVALID_ARG;
  if ((dtype != MOE_F32 && dtype != MOE_BF16) || (block_rows != 1 && block_rows != 128) ||
      (transpose != 0 && transpose != 1))
    return MOE_ERR_INVALID_ARG;
  // a workgroup's rows: 32 where rows are quantised as they lie
  const int64_t tile = block_rows == 1 && !transpose ? 32 : 128;
  if (rows > kMaxQuantRows || cols > kMaxQuantRows || ceil_div(rows, tile) * ceil_div(cols, 128) > kMaxQuantTiles)
    return MOE_ERR_UNSUPPORTED;
  if (rows == 0 || cols == 0) return MOE_OK;
  if (!x || !q || !scales || !aligned16(q) || !aligned_to(x, dtype == MOE_BF16 ? 2 : 4) || !aligned_to(scales, 4))
    return MOE_ERR_INVALID_ARG;
  moe::QuantizeArgs a{};
  a.x = x;
  a.rows = rows;
  a.cols = cols;
  a.ld = ldx;
  a.dt = dtype;
  a.block_rows = block_rows;
  a.transpose = transpose != 0;
  const int64_t R = transpose ? cols : rows, K = transpose ? rows : cols;
  a.q = static_cast<char*>(q);
  a.ldq = align128(K);
  a.scale = scales;
  a.scale_ld = block_rows == 1 ? R : align128(K) / 128;
  return hip_status(moe::launch_quantize(a, static_cast<hipStream_t>(stream)));
}

MOE_API moe_status moe_gemm_quant_ws_bytes(const moe_quant_gemm* gemm, size_t* bytes) {
  moe::QuantGemm g{};
  moe_status st = check_gemm_quant(gemm, &g);
  if (st != MOE_OK) return st;
  if (!bytes) return MOE_ERR_INVALID_ARG;
  *bytes = (size_t)align256(moe::quant_gemm_ws_bytes(g));
  return MOE_OK;
}

MOE_API moe_status moe_gemm_quant(const moe_quant_gemm* gemm, void* ws, size_t ws_bytes, void* stream) {
  moe::QuantGemm g{};
  moe_status st = check_gemm_quant(gemm, &g);
  if (st != MOE_OK) return st;
  if (g.M == 0 || g.N == 0) return MOE_OK;
  if (!gemm->c || !aligned_to(gemm->c, gemm->out_dtype == MOE_BF16 ? 2 : 4)) return MOE_ERR_INVALID_ARG;
  if (g.K > 0 && (!gemm->a || !gemm->a_scale || !gemm->b || !gemm->b_scale || !aligned16(gemm->a) ||
                  !aligned16(gemm->b) || !aligned_to(gemm->a_scale, 4) || !aligned_to(gemm->b_scale, 4)))
    return MOE_ERR_INVALID_ARG;
  const int64_t need = align256(moe::quant_gemm_ws_bytes(g));
  if (need > 0 && (!ws || (int64_t)ws_bytes < need || !aligned256(ws))) return MOE_ERR_WORKSPACE;
  g.A = static_cast<const char*>(gemm->a);
  g.a_scale = gemm->a_scale;
  g.B = static_cast<const char*>(gemm->b);
  g.b_scale = gemm->b_scale;
  g.C = gemm->c;
  return hip_status(moe::launch_quant_gemm(g, ws, static_cast<hipStream_t>(stream)));
}

MOE_API moe_status moe_experts_dropless_quant_ws_bytes(const moe_config* cfg, size_t* bytes) {
  moe_plan p;
  moe_status st = check_quant_config(cfg, &p);
  if (st != MOE_OK) return st;
  if (!bytes) return MOE_ERR_INVALID_ARG;
  QuantExpertsWs q;
  *bytes = (size_t)carve_experts_quant(cfg, p.dropless_rows, nullptr, &q);
  return MOE_OK;
}

MOE_API moe_status moe_experts_dropless_quant(const moe_config* cfg, const void* xs, const int32_t* expert_offsets,
                                              const moe_quant_experts* w, void* expert_out, void* ws,
                                              size_t ws_bytes, void* stream) {
  moe_plan p;
  moe_status st = check_quant_config(cfg, &p);
  if (st != MOE_OK) return st;
  if (!expert_offsets || !quant_experts_valid(w)) return MOE_ERR_INVALID_ARG;
  if (cfg->T == 0) return MOE_OK;
  if (!xs || !expert_out || !aligned16(xs) || !aligned16(expert_out)) return MOE_ERR_INVALID_ARG;
  QuantExpertsWs q;
  if (!ws || (int64_t)ws_bytes < carve_experts_quant(cfg, p.dropless_rows, nullptr, &q) || !aligned256(ws))
    return MOE_ERR_WORKSPACE;
  return run_experts_quant(cfg, p, xs, expert_offsets, w, expert_out, ws, static_cast<hipStream_t>(stream));
}

// ------------------------------------------------------------------ dropless forward in e4m3
namespace {

constexpr int64_t kFewLogitRows = 1024;  // rows of the router product up to which the kernel for few is the faster

struct QuantForwardWs {
  char* xq;       // quantised x and its scales
  float* xs;
  char* z;
  float* logits;
  int32_t* topk;
  float* gates;
  int32_t* row_of;
  int32_t* offsets;
  char* rows;     // xs of the dispatch
  char* expert_out;
  char* y_lat;
  char* cat;      // [T][L + S Fs]: quantised y_lat and shared hidden rows
  float* cat_s;
  float* h;       // few tokens: shared hidden rows in fp32
  int64_t* counts;
  void* dispatch;
  void* experts;
  void* gemm;
};

moe::QuantGemm dense_quant(const char* A, const float* sa, int64_t T, const void* B, const float* sb, int64_t N,
                           int64_t K, void* C) {
  moe::QuantGemm g{};
  g.A = A;
  g.lda = K;
  g.a_scale = sa;
  g.a_scale_ld = T;
  g.B = static_cast<const char*>(B);
  g.ldb = K;
  g.b_scale = sb;
  g.b_scale_ld = K / 128;
  g.b_rows = 128;
  g.M = T;
  g.N = N;
  g.K = (int)K;
  g.out_dt = moe::DT_BF16;
  g.C = C;
  g.ldc = N;
  return g;
}

int64_t carve_forward_quant(const moe_config* c, const moe_plan& p, const moe_dropless_taps& tp, int64_t* counts,
                            void* ws, QuantForwardWs* w) {
  const int64_t T = c->T, D = c->d_model, L = c->d_latent, E = c->n_experts, k = c->top_k, n = p.dropless_rows;
  const int64_t W = L + (int64_t)c->n_shared * c->d_ff_shared;
  Carver cv{static_cast<char*>(ws), 0};
  auto pick = [&](void* tap, int64_t bytes) {
    void* q = cv.take(bytes);
    return tap ? tap : q;
  };
  w->xq = static_cast<char*>(cv.take(T * D));
  w->xs = static_cast<float*>(cv.take(T * (D / 128) * 4));
  w->z = static_cast<char*>(pick(tp.z, T * L * 2));
  w->logits = static_cast<float*>(pick(tp.logits, T * E * 4));
  w->topk = static_cast<int32_t*>(pick(tp.topk_idx, T * k * 4));
  w->gates = static_cast<float*>(pick(tp.gates, T * k * 4));
  w->row_of = static_cast<int32_t*>(pick(tp.row_of, T * k * 4));
  w->offsets = static_cast<int32_t*>(pick(tp.expert_offsets, (E + 1) * 4));
  w->rows = static_cast<char*>(pick(tp.xs, moe::few_rows(n, (int)E, true) ? n * L * 2 : 0));
  w->expert_out = static_cast<char*>(pick(tp.expert_out, n * L * 2));
  w->y_lat = static_cast<char*>(pick(tp.y_latent, T * L * 2));
  w->cat = static_cast<char*>(cv.take(T * W));
  w->cat_s = static_cast<float*>(cv.take(T * (W / 128) * 4));
  w->h = static_cast<float*>(cv.take(moe::few_rows(T, c->n_shared, false) ? T * (W - L) * 4 : 0));
  w->counts = static_cast<int64_t*>(pick(counts, 3 * 8));
  w->dispatch = cv.take(p.dropless_dispatch_ws_bytes);
  QuantExpertsWs x;
  w->experts = cv.take(carve_experts_quant(c, n, nullptr, &x));
  const int64_t g0 = moe::quant_gemm_ws_bytes(dense_quant(nullptr, nullptr, T, nullptr, nullptr, L, D, nullptr));
  const int64_t g1 = moe::quant_gemm_ws_bytes(dense_quant(nullptr, nullptr, T, nullptr, nullptr, D, W, nullptr));
  w->gemm = cv.take(g0 > g1 ? g0 : g1);
  return cv.used;
}

moe_status check_forward_quant(const moe_config* cfg, moe_plan* p) {
  moe_status st = check_quant_config(cfg, p);
  if (st != MOE_OK) return st;
  if (cfg->top_k > cfg->n_experts) return MOE_ERR_INVALID_ARG;
  if (cfg->n_experts % 4 || cfg->d_model % 128 || (cfg->n_shared > 0 && cfg->d_ff_shared % 128))
    return MOE_ERR_UNSUPPORTED;
  // the two dense products and the shared hidden tiles, within the limits of moe_gemm_quant
  const int64_t W = cfg->d_latent + (int64_t)cfg->n_shared * cfg->d_ff_shared;
  const int64_t widest = cfg->d_model > W ? cfg->d_model : W;
  if (widest > kMaxQuantK || cfg->T > kMaxQuantRows || ceil_div(cfg->T, 64) * ceil_div(widest, 128) > kMaxListEntries)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace

MOE_API moe_status moe_forward_dropless_quant_ws_bytes(const moe_config* cfg, size_t* bytes) {
  moe_plan p;
  moe_status st = check_forward_quant(cfg, &p);
  if (st != MOE_OK) return st;
  if (!bytes) return MOE_ERR_INVALID_ARG;
  QuantForwardWs w;
  *bytes = (size_t)carve_forward_quant(cfg, p, moe_dropless_taps{}, nullptr, nullptr, &w);
  return MOE_OK;
}

MOE_API moe_status moe_forward_dropless_quant(const moe_config* cfg, const moe_scoring* scoring,
                                              const moe_quant_weights* w, const void* x, void* y,
                                              const moe_dropless_taps* taps, int64_t* counts, void* ws,
                                              size_t ws_bytes, void* stream) {
  moe_plan p;
  moe_status st = check_forward_quant(cfg, &p);
  if (st != MOE_OK) return st;
  moe::ScoreArgs sc{};
  st = check_scoring(cfg, scoring, &sc);
  if (st != MOE_OK) return st;
  if (!w || !w->q_latent || !w->s_latent || !w->w_router || !quant_experts_valid(&w->experts) || !w->q_output ||
      !w->s_output || !aligned16(w->q_latent) || !aligned16(w->w_router) || !aligned16(w->q_output))
    return MOE_ERR_INVALID_ARG;
  if (cfg->n_shared > 0 && (!w->q_shared_gate || !w->s_shared_gate || !w->q_shared_up || !w->s_shared_up ||
                            !aligned16(w->q_shared_gate) || !aligned16(w->q_shared_up)))
    return MOE_ERR_INVALID_ARG;
  if (cfg->T > 0 && (!x || !y || !aligned16(x) || !aligned16(y))) return MOE_ERR_INVALID_ARG;
  const moe_dropless_taps none{};
  const moe_dropless_taps& tp = taps ? *taps : none;
  for (const void* t : {static_cast<const void*>(tp.logits), static_cast<const void*>(tp.z),
                        static_cast<const void*>(tp.xs), static_cast<const void*>(tp.expert_out),
                        static_cast<const void*>(tp.y_latent)})
    if (!aligned16(t)) return MOE_ERR_INVALID_ARG;
  QuantForwardWs q;
  if (!ws || !aligned256(ws) || (int64_t)ws_bytes < carve_forward_quant(cfg, p, none, nullptr, nullptr, &q))
    return MOE_ERR_WORKSPACE;
  carve_forward_quant(cfg, p, tp, counts, ws, &q);

  hipStream_t s = static_cast<hipStream_t>(stream);
  const int64_t T = cfg->T, D = cfg->d_model, L = cfg->d_latent, E = cfg->n_experts, S = cfg->n_shared;
  const int64_t Fs = S > 0 ? cfg->d_ff_shared : 0, W = L + S * Fs;
  auto quantize = [&](const void* from, int dt, int64_t cols, char* to, int64_t ldq, float* scale) {
    moe::QuantizeArgs a{};
    a.x = from;
    a.rows = T;
    a.cols = a.ld = cols;
    a.dt = dt;
    a.block_rows = 1;
    a.q = to;
    a.ldq = ldq;
    a.scale = scale;
    a.scale_ld = T;
    return moe::launch_quantize(a, s);
  };
  // z, then the router on it
  hipError_t e = quantize(x, moe::DT_BF16, D, q.xq, D, q.xs);
  if (e == hipSuccess)
    e = moe::launch_quant_gemm(dense_quant(q.xq, q.xs, T, w->q_latent, w->s_latent, L, D, q.z), q.gemm, s);
  if (e != hipSuccess) return MOE_ERR_HIP;
  moe::GemmDense r{};
  r.nseg = 1;
  r.seg[0] = {q.z, L, w->w_router, L, (int)L};
  r.C = q.logits;
  r.ldc = E;
  r.M = (int)T;
  r.N = (int)E;
  e = T <= kFewLogitRows ? moe::launch_few_f32out_bf16(r, s) : moe::launch_gemm_dense(moe::DT_BF16, moe::DT_F32, r, s);
  if (e == hipSuccess) e = moe::launch_route_scored(sc, q.logits, w->router_bias, q.topk, q.gates, s);
  if (e != hipSuccess) return MOE_ERR_HIP;
  // the routed path.  Rows are quantised on their way to their experts,
  // except where the bf16 rows are asked for or where the experts' kernels for
  // few rows quantise them
  const bool bf16_rows = tp.xs || moe::few_rows(p.dropless_rows, (int)E, true);
  st = run_dispatch_dropless(cfg, p, q.topk, q.z, bf16_rows ? q.rows : nullptr, q.row_of, q.offsets, q.counts,
                             q.dispatch, s, nullptr);
  if (st != MOE_OK) return st;
  if (T > 0) {
    if (!bf16_rows) {
      QuantExpertsWs x;
      carve_experts_quant(cfg, p.dropless_rows, q.experts, &x);
      e = moe::launch_quantize_scatter(q.z, T, (int)L, q.row_of, cfg->top_k, x.xq, x.xs, p.dropless_rows, s);
      if (e != hipSuccess) return MOE_ERR_HIP;
    }
    st = run_experts_quant(cfg, p, bf16_rows ? q.rows : nullptr, q.offsets, &w->experts, q.expert_out, q.experts, s);
    if (st != MOE_OK) return st;
  }
  e = moe::launch_ragged_combine(moe::DT_BF16, q.expert_out, q.row_of, q.gates, T, cfg->top_k, L * 2, q.y_lat, s);
  if (e == hipSuccess) e = quantize(q.y_lat, moe::DT_BF16, L, q.cat, W, q.cat_s);
  if (e != hipSuccess) return MOE_ERR_HIP;
  // shared hidden rows beside it
  if (S > 0 && T > 0) {
    if (moe::few_rows(T, (int)S, false)) {
      moe::FewRows u{};
      u.x = q.xq;
      u.ldx = D;
      u.x_scale = q.xs;
      u.x_scale_ld = T;
      u.W0 = static_cast<const char*>(w->q_shared_gate);
      u.s0 = w->s_shared_gate;
      u.W1 = static_cast<const char*>(w->q_shared_up);
      u.s1 = w->s_shared_up;
      u.M = T;
      u.E = (int)S;
      u.N = (int)Fs;
      u.K = (int)D;
      u.chunk = 16;
      u.out = q.h;
      u.ldo = S * Fs;
      e = moe::launch_few_rows(u, true, false, s);
      if (e == hipSuccess) e = quantize(q.h, moe::DT_F32, S * Fs, q.cat + L, W, q.cat_s + (L / 128) * T);
    } else {
      moe::QuantGateUp u{};
      u.A = q.xq;
      u.lda = D;
      u.a_scale = q.xs;
      u.a_scale_ld = T;
      u.Wg = static_cast<const char*>(w->q_shared_gate);
      u.sg = w->s_shared_gate;
      u.Wu = static_cast<const char*>(w->q_shared_up);
      u.su = w->s_shared_up;
      u.M = T;
      u.E = (int)S;
      u.F = (int)Fs;
      u.K = (int)D;
      u.H = q.cat + L;
      u.ldh = W;
      u.h_scale = q.cat_s + (L / 128) * T;
      u.h_scale_ld = T;
      e = moe::launch_quant_gate_up(u, s);
    }
    if (e != hipSuccess) return MOE_ERR_HIP;
  }
  return hip_status(moe::launch_quant_gemm(dense_quant(q.cat, q.cat_s, T, w->q_output, w->s_output, D, W, y), q.gemm, s));
}

// ------------------------------------------------------------------ linear layers
namespace {

constexpr int64_t kMaxLd = int64_t(1) << 22;  // 256 rows of 2 bytes stay below 2^31
constexpr int64_t kMaxLinearRows = int64_t(1) << 30;
constexpr int64_t kMaxSlopeRows = 65535 * 32;  // one grid row for 32 rows of d

int64_t align8(int64_t x) { return (x + 7) & ~int64_t(7); }

// a launch has fewer than 2^32 threads: one of every 8 values that are copied
bool copies_fit(int64_t x_rows, int64_t w_rows, int64_t K8) {
  return ceil_div(x_rows * (K8 / 8), 256) + ceil_div(w_rows * (K8 / 8), 256) < (int64_t(1) << 24);
}

// rows can be read by the tiles as they are
bool tile_rows(const void* p, int64_t ld) { return aligned16(p) && ld % 8 == 0; }

moe_status check_linear_sizes(int64_t M, int64_t N, int64_t K) {
  if (M < 0 || N < 0 || K < 0) return MOE_ERR_INVALID_ARG;
  if (M > kMaxLinearRows || N > kMaxLd || K > kMaxLd) return MOE_ERR_UNSUPPORTED;
  const int64_t n = N > K ? N : K;
  if (ceil_div(M, 128) * ceil_div(n, 128) > kMaxListEntries || ceil_div(N, 128) * ceil_div(K, 128) > kMaxListEntries)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status check_ld(int64_t ld, int64_t least) {
  if (ld < least) return MOE_ERR_INVALID_ARG;
  return ld > kMaxLd ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

bool valid_dtype(int32_t d) { return d == MOE_F32 || d == MOE_BF16; }
bool valid_act(int32_t a) { return a >= MOE_ACT_NONE && a <= MOE_ACT_GELU; }
bool on_elem(const void* p, int32_t dtype) { return aligned_to(p, dtype == MOE_F32 ? 4 : 2); }

moe_status check_linear(const moe_linear_args* a) {
  if (!a) return MOE_ERR_INVALID_ARG;
  if (!valid_dtype(a->bias_dtype) || !valid_dtype(a->out_dtype) || !valid_act(a->act) || a->reserved != 0)
    return MOE_ERR_INVALID_ARG;
  moe_status st = check_linear_sizes(a->M, a->N, a->K);
  if (st == MOE_OK) st = check_ld(a->ldx, a->K);
  if (st == MOE_OK) st = check_ld(a->ldw, a->K);
  if (st == MOE_OK) st = check_ld(a->ldy, a->N);
  if (st == MOE_OK && a->residual) st = check_ld(a->ldr, a->N);
  if (st == MOE_OK && a->pre) st = check_ld(a->ldp, a->N);
  if (st != MOE_OK) return st;
  if (!aligned_to(a->x, 2) || !aligned_to(a->w, 2) || !on_elem(a->bias, a->bias_dtype) ||
      !on_elem(a->residual, a->out_dtype) || !on_elem(a->y, a->out_dtype) || !aligned_to(a->pre, 2))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

struct LinearWs {
  moe::LinearPlan plan;
  bool regs;  // the operands are taken as they lie, by way of registers
  bool fits;  // the copies' launch
  void* x;    // copies in whole 16 bytes, or null
  void* w;
  void* part;
};
int64_t carve_linear(const moe_linear_args* a, void* ws, LinearWs* w) {
  Carver cv{static_cast<char*>(ws), 0};
  *w = LinearWs{};
  w->fits = true;
  if (a->M == 0 || a->N == 0 || moe::linear_streams(a->M, a->N, a->K)) return 0;
  const int64_t K8 = align8(a->K);
  const int cls = moe::linear_class(a->M, a->N, a->K, 0, 0, 0);
  w->plan = moe::linear_plan(cls, a->M, a->N, K8, moe::linear_units(cls, a->M, a->N, K8));
  const bool whole = a->K % 8 == 0, x = whole && tile_rows(a->x, a->ldx), y = whole && tile_rows(a->w, a->ldw);
  if (cls == moe::TILE_DEEP) {
    w->regs = !(x && y);
  } else if (a->K > 0) {
    if (!x) w->x = cv.take(a->M * K8 * 2);
    if (!y) w->w = cv.take(a->N * K8 * 2);
    w->fits = copies_fit(x ? 0 : a->M, y ? 0 : a->N, K8);
  }
  if (w->plan.part_bytes) w->part = cv.take(w->plan.part_bytes);
  return cv.used;
}

}  // namespace

MOE_API moe_status moe_linear_ws_bytes(const moe_linear_args* args, size_t* bytes) {
  const moe_status st = check_linear(args);
  if (st != MOE_OK) return st;
  if (!bytes) return MOE_ERR_INVALID_ARG;
  LinearWs w;
  const int64_t need = carve_linear(args, nullptr, &w);
  if (!w.fits) return MOE_ERR_UNSUPPORTED;
  *bytes = (size_t)need;
  return MOE_OK;
}

MOE_API moe_status moe_linear(const moe_linear_args* args, void* ws, size_t ws_bytes, void* stream) {
  const moe_status st = check_linear(args);
  if (st != MOE_OK) return st;
  const moe_linear_args& a = *args;
  if (a.M == 0 || a.N == 0) return MOE_OK;
  if (!a.y || (a.K > 0 && (!a.x || !a.w))) return MOE_ERR_INVALID_ARG;
  LinearWs w;
  const int64_t need = carve_linear(args, nullptr, &w);
  if (!w.fits) return MOE_ERR_UNSUPPORTED;
  if (need > 0 && (!ws || !aligned256(ws) || (int64_t)ws_bytes < need)) return MOE_ERR_WORKSPACE;
  carve_linear(args, need > 0 ? ws : nullptr, &w);
  hipStream_t s = static_cast<hipStream_t>(stream);
  moe::Linear g{};
  g.x = a.x;
  g.ldx = a.ldx;
  g.w = a.w;
  g.ldw = a.ldw;
  g.M = a.M;
  g.N = (int)a.N;
  g.K = (int)a.K;
  g.bias = a.bias;
  g.bias_dt = a.bias_dtype;
  g.res = a.residual;
  g.ldr = a.ldr;
  g.y = a.y;
  g.ldy = a.ldy;
  g.out_dt = a.out_dtype;
  g.pre = a.pre;
  g.ldp = a.ldp;
  g.act = a.act;
  if (moe::linear_streams(a.M, a.N, a.K)) return hip_status(moe::launch_linear_stream(g, s));
  const int64_t K8 = align8(a.K);
  const moe::PackRows px{a.x, a.M, g.K, a.ldx, w.x, K8}, pw{a.w, a.N, g.K, a.ldw, w.w, K8};
  const hipError_t e = moe::launch_pack_rows(px, pw, s);
  if (e != hipSuccess) return MOE_ERR_HIP;
  if (w.x) {
    g.x = w.x;
    g.ldx = K8;
  }
  if (w.w) {
    g.w = w.w;
    g.ldw = K8;
  }
  g.part = static_cast<float*>(w.part);
  return hip_status(moe::launch_linear_tiles(g, w.plan, w.regs, s));
}

namespace {

moe_status check_linear_grad(const moe_linear_grad* a) {
  if (!a) return MOE_ERR_INVALID_ARG;
  if (!valid_dtype(a->dy_dtype) || !valid_act(a->act) || a->reserved != 0) return MOE_ERR_INVALID_ARG;
  moe_status st = check_linear_sizes(a->M, a->N, a->K);
  if (st == MOE_OK && a->M > kMaxSlopeRows) st = MOE_ERR_UNSUPPORTED;
  // both products and the sums of db are one launch
  if (st == MOE_OK &&
      ((a->dw ? ceil_div(a->N, 128) : 0) + (a->dx ? ceil_div(a->M, 128) : 0)) * ceil_div(a->K, 128) +
              (a->db ? ceil_div(a->N, 64) : 0) > kMaxListEntries - 16)
    st = MOE_ERR_UNSUPPORTED;
  if (st == MOE_OK) st = check_ld(a->lddy, a->N);
  if (st == MOE_OK && a->act != MOE_ACT_NONE) st = check_ld(a->ldp, a->N);
  if (st == MOE_OK && a->dw) st = check_ld(a->ldx, a->K);
  if (st == MOE_OK && a->dx) st = check_ld(a->ldw, a->K);
  if (st == MOE_OK && a->dx) st = check_ld(a->lddx, a->K);
  if (st == MOE_OK && a->dw) st = check_ld(a->lddw, a->K);
  if (st != MOE_OK) return st;
  if (!on_elem(a->dy, a->dy_dtype) || !aligned_to(a->pre, 2) || !aligned_to(a->x, 2) || !aligned_to(a->w, 2) ||
      !aligned_to(a->dx, 2) || !aligned_to(a->dw, 2) || !aligned_to(a->db, 4))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

struct LinearGradWs {
  moe::LinearPlan dw, dx;
  bool regs;    // x and w are taken as they lie, by way of registers
  bool fits;    // the copies' launch
  void* d;      // bf16 [M][N rounded up to 8], or null: dy itself
  float* sums;  // partial sums of db
  void* x;      // copies in whole 16 bytes, or null
  void* w;
  void* part_dw;
  void* part_dx;
};
int64_t carve_linear_grad(const moe_linear_grad* a, void* ws, LinearGradWs* w) {
  Carver cv{static_cast<char*>(ws), 0};
  *w = LinearGradWs{};
  const int64_t N8 = align8(a->N), K8 = align8(a->K);
  const bool dx = a->dx != nullptr, dw = a->dw != nullptr;
  const int cls = moe::linear_class(dw ? a->N : 0, a->K, a->M, dx ? a->M : 0, a->K, a->N);
  const double units = (dw ? moe::linear_units(cls, a->N, a->K, a->M) : 0.0) +
                       (dx ? moe::linear_units(cls, a->M, a->K, a->N) : 0.0);
  w->dw = moe::linear_plan(cls, a->N, a->K, a->M, units);
  w->dx = moe::linear_plan(cls, a->M, a->K, a->N, units);
  const bool products = (dx || dw) && a->M > 0 && a->N > 0 && a->K > 0;
  // dy as it is serves as d where no slope and no rounding is due
  const bool own = a->act == MOE_ACT_NONE && a->dy_dtype == MOE_BF16 && tile_rows(a->dy, a->lddy) &&
                   (!dx || a->N % 8 == 0);
  if (products && !own) w->d = cv.take(a->M * N8 * 2);
  if (a->db && a->M > 0) w->sums = static_cast<float*>(cv.take(moe::slope_blocks(a->M) * a->N * 4));
  const bool x = dw && !tile_rows(a->x, a->ldx), y = dx && !tile_rows(a->w, a->ldw);
  // by way of registers a k-row has at least 8 values
  w->regs = cls == moe::TILE_DEEP && (x || y) && (!dw || a->ldx >= 8) && (!dx || a->ldw >= 8);
  if (products && !w->regs) {
    if (x) w->x = cv.take(a->M * K8 * 2);
    if (y) w->w = cv.take(a->N * K8 * 2);
  }
  w->fits = !products || w->regs || copies_fit(x ? a->M : 0, y ? a->N : 0, K8);
  if (dw && w->dw.part_bytes) w->part_dw = cv.take(w->dw.part_bytes);
  if (dx && w->dx.part_bytes) w->part_dx = cv.take(w->dx.part_bytes);
  return cv.used;
}

}  // namespace

MOE_API moe_status moe_linear_backward_ws_bytes(const moe_linear_grad* args, size_t* bytes) {
  const moe_status st = check_linear_grad(args);
  if (st != MOE_OK) return st;
  if (!bytes) return MOE_ERR_INVALID_ARG;
  LinearGradWs w;
  const int64_t need = carve_linear_grad(args, nullptr, &w);
  if (!w.fits) return MOE_ERR_UNSUPPORTED;
  *bytes = (size_t)need;
  return MOE_OK;
}

MOE_API moe_status moe_linear_backward(const moe_linear_grad* args, void* ws, size_t ws_bytes, void* stream) {
  const moe_status st = check_linear_grad(args);
  if (st != MOE_OK) return st;
  const moe_linear_grad& a = *args;
  if (a.M > 0 && a.N > 0) {
    if ((a.dx || a.dw || a.db) && (!a.dy || (a.act != MOE_ACT_NONE && !a.pre))) return MOE_ERR_INVALID_ARG;
    if (a.K > 0 && ((a.dx && !a.w) || (a.dw && !a.x))) return MOE_ERR_INVALID_ARG;
  }
  LinearGradWs w;
  const int64_t need = carve_linear_grad(args, nullptr, &w);
  if (!w.fits) return MOE_ERR_UNSUPPORTED;
  if (need > 0 && (!ws || !aligned256(ws) || (int64_t)ws_bytes < need)) return MOE_ERR_WORKSPACE;
  carve_linear_grad(args, need > 0 ? ws : nullptr, &w);
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int64_t N8 = align8(a.N), K8 = align8(a.K);
  hipError_t e = hipSuccess;
  if (w.d || w.sums)
    e = moe::launch_slope(a.dy, a.lddy, a.dy_dtype, a.pre, a.ldp, a.act, a.M, (int)a.N, w.d, N8, w.sums, s);
  const moe::PackRows px{a.x, a.M, (int)a.K, a.ldx, w.x, K8}, pw{a.w, a.N, (int)a.K, a.ldw, w.w, K8};
  if (e == hipSuccess) e = moe::launch_pack_rows(px, pw, s);
  if (e != hipSuccess) return MOE_ERR_HIP;
  const void* d = w.d ? w.d : a.dy;
  const int64_t ldd = w.d ? N8 : a.lddy;
  moe::LinearGrads g{};
  if (a.dw) {  // d and x, both K-major along M
    moe::Linear& q = g.dw;
    q.x = d;
    q.ldx = ldd;
    q.w = w.x ? w.x : a.x;
    q.ldw = w.x ? K8 : a.ldx;
    q.M = a.N;
    q.N = (int)a.K;
    q.K = (int)a.M;
    q.y = a.dw;
    q.ldy = a.lddw;
    q.out_dt = moe::DT_BF16;
    q.part = static_cast<float*>(w.part_dw);
  }
  if (a.dx) {  // d by W, K-major along N
    moe::Linear& q = g.dx;
    q.x = d;
    q.ldx = ldd;
    q.w = w.w ? w.w : a.w;
    q.ldw = w.w ? K8 : a.ldw;
    q.M = a.M;
    q.N = (int)a.K;
    q.K = (int)a.N;
    q.y = a.dx;
    q.ldy = a.lddx;
    q.out_dt = moe::DT_BF16;
    q.part = static_cast<float*>(w.part_dx);
  }
  g.sums = w.sums;
  g.sum_blocks = w.sums ? moe::slope_blocks(a.M) : 0;
  g.N = (int)a.N;
  g.db = a.db;
  return hip_status(moe::launch_linear_grads(g, w.dw, w.dx, w.regs, s));
}

// ------------------------------------------------------------------ orthogonalised updates
namespace {

constexpr int kMaxOrthoSteps = 64;
constexpr int64_t kMaxOrthoSide = 65536;
constexpr int64_t kMaxOrthoLd = int64_t(1) << 30;
constexpr double kMaxSingular = 1048576.0;

// The largest power of two that takes magnitudes up to `most` to at most half
// of fp16's range.
float fp16_scale(double most) {
  if (!(most > 0.0)) return 1.0f;
  int e = 0;
  frexp(32768.0 / most, &e);  // 32768 / most in [2^(e-1), 2^e)
  e -= 1;
  return ldexpf(1.0f, e > 60 ? 60 : e);
}

// Bounds of every step's singular values, from those of X_0 (at most 1, its
// Frobenius norm), and the scales that follow.  One part in 64 is left to the
// roundings of a step.
moe_status ortho_steps(const moe_ortho_args* a, moe::OrthoStep* out) {
  double m = 1.0;
  double gain[kMaxOrthoSteps];  // most that a step multiplies a singular value by
  for (int k = 0; k < a->steps; ++k) {
    const double ca = a->coeffs[3 * k], cb = a->coeffs[3 * k + 1], cc = a->coeffs[3 * k + 2];
    if (!isfinite(ca) || !isfinite(cb) || !isfinite(cc)) return MOE_ERR_INVALID_ARG;
    const double y = m * m;
    // |b t + c t^2| and |a + b t + c t^2| on [0, m^2], and |a s + b s^3 + c s^5| on [0, m]
    double q = fabs(cb * y + cc * y * y);
    gain[k] = fmax(fabs(ca), fabs(ca + cb * y + cc * y * y));
    if (cc != 0.0) {
      const double t = -cb / (2.0 * cc), v = cb * t + cc * t * t;
      if (t > 0.0 && t < y) {
        q = fmax(q, fabs(v));
        gain[k] = fmax(gain[k], fabs(ca + v));
      }
    }
    auto poly = [&](double s) { return fabs(s * (ca + s * s * (cb + cc * s * s))); };
    double p = poly(m);
    // 5 c t^2 + 3 b t + a = 0 for t = s^2
    double root[2];
    int n = 0;
    if (cc != 0.0) {
      const double d = 9.0 * cb * cb - 20.0 * ca * cc;
      if (d >= 0.0) {
        const double u = -0.5 * (3.0 * cb + (cb < 0.0 ? -sqrt(d) : sqrt(d)));
        root[n++] = u / (5.0 * cc);
        if (u != 0.0) root[n++] = ca / u;
      }
    } else if (cb != 0.0) {
      root[n++] = -ca / (3.0 * cb);
    }
    for (int i = 0; i < n; ++i)
      if (root[i] > 0.0 && root[i] < y && poly(sqrt(root[i])) > p) p = poly(sqrt(root[i]));
    const double slack = 1.0 + 1.0 / 64;
    out[k].a = (float)ca;
    out[k].b = (float)cb;
    out[k].c = (float)cc;
    out[k].sx = fp16_scale(m * slack);
    out[k].sa = fp16_scale(y * slack);
    out[k].sb = fp16_scale(q * slack);
    m = p * slack;
    if (!(m < kMaxSingular) || !(q < kMaxSingular * kMaxSingular)) return MOE_ERR_UNSUPPORTED;
  }
  // what a step leaves behind grows by the gains of those after it
  double later = 1.0;
  for (int k = a->steps - 1; k >= 0; --k) {
    out[k].low = later > 1.0 ? (float)(1.0 / later) : 1.0f;
    later = fmin(later * gain[k], 1e30);
  }
  return MOE_OK;
}

moe_status check_ortho(const moe_ortho_args* a, moe::OrthoStep* steps) {
  if (!a) return MOE_ERR_INVALID_ARG;
  if (a->batch < 0 || a->M < 0 || a->N < 0 || a->reserved != 0 || !valid_dtype(a->dtype) || !a->coeffs ||
      a->steps < 1 || a->steps > kMaxOrthoSteps || !(a->eps >= 0.0f) || !isfinite(a->eps) || !isfinite(a->scale))
    return MOE_ERR_INVALID_ARG;
  if (a->M > kMaxOrthoSide || a->N > kMaxOrthoSide || a->batch > kI32Max) return MOE_ERR_UNSUPPORTED;
  if (a->ldg < a->N || a->ldo < a->N) return MOE_ERR_INVALID_ARG;
  if (a->ldg > kMaxOrthoLd || a->ldo > kMaxOrthoLd) return MOE_ERR_UNSUPPORTED;
  if (a->batch > 1 && a->M > 0 &&
      (a->stride_g < (a->M - 1) * a->ldg + a->N || a->stride_o < (a->M - 1) * a->ldo + a->N ||
       a->stride_g > (int64_t(1) << 46) || a->stride_o > (int64_t(1) << 46)))
    return MOE_ERR_INVALID_ARG;
  if (!on_elem(a->g, a->dtype) || !aligned_to(a->out, 2)) return MOE_ERR_INVALID_ARG;
  return ortho_steps(a, steps);
}

int64_t align64(int64_t x) { return (x + 63) & ~int64_t(63); }

int64_t carve_ortho(const moe_ortho_args* a, void* ws, moe::Ortho* p, int64_t* group) {
  const int64_t m = a->M < a->N ? a->M : a->N, n = a->M < a->N ? a->N : a->M, mp = align64(m), np = align64(n);
  *group = moe::ortho_group(a->batch, m, n);
  const int64_t g = *group;
  Carver cv{static_cast<char*>(ws), 0};
  p->norm = static_cast<double*>(cv.take(g * moe::ortho_norm_chunks() * 8));
  p->x16[0] = static_cast<uint16_t*>(cv.take(g * m * np * 2));
  p->x16[1] = static_cast<uint16_t*>(cv.take(a->steps > 1 ? g * m * np * 2 : 0));
  p->lo16[0] = static_cast<uint16_t*>(cv.take(g * m * np * 2));
  p->lo16[1] = static_cast<uint16_t*>(cv.take(a->steps > 1 ? g * m * np * 2 : 0));
  p->a16 = static_cast<uint16_t*>(cv.take(g * m * mp * 2));
  p->b16 = static_cast<uint16_t*>(cv.take(g * m * mp * 2));
  p->da = static_cast<float*>(cv.take(g * m * 4));
  p->db = static_cast<float*>(cv.take(g * m * 4));
  p->m = (int)m;
  p->n = (int)n;
  p->mp = (int)mp;
  p->np = (int)np;
  return cv.used;
}

}  // namespace

MOE_API moe_status moe_orthogonalize_ws_bytes(const moe_ortho_args* args, size_t* bytes) {
  moe::OrthoStep steps[kMaxOrthoSteps];
  const moe_status st = check_ortho(args, steps);
  if (st != MOE_OK) return st;
  if (!bytes) return MOE_ERR_INVALID_ARG;
  *bytes = 0;
  if (args->batch == 0 || args->M == 0 || args->N == 0) return MOE_OK;
  moe::Ortho p{};
  int64_t group;
  *bytes = (size_t)carve_ortho(args, nullptr, &p, &group);
  return MOE_OK;
}

MOE_API moe_status moe_orthogonalize(const moe_ortho_args* args, void* ws, size_t ws_bytes, void* stream) {
  moe::OrthoStep steps[kMaxOrthoSteps];
  const moe_status st = check_ortho(args, steps);
  if (st != MOE_OK) return st;
  const moe_ortho_args& a = *args;
  if (a.batch == 0 || a.M == 0 || a.N == 0) return MOE_OK;
  if (!a.g || !a.out) return MOE_ERR_INVALID_ARG;
  moe::Ortho p{};
  int64_t group;
  const int64_t need = carve_ortho(args, nullptr, &p, &group);
  if (!ws || !aligned256(ws) || (int64_t)ws_bytes < need) return MOE_ERR_WORKSPACE;
  carve_ortho(args, ws, &p, &group);
  p.g = a.g;
  p.ldg = a.ldg;
  p.stride_g = a.stride_g;
  p.dt = a.dtype;
  p.M = (int)a.M;
  p.N = (int)a.N;
  p.out = static_cast<uint16_t*>(a.out);
  p.ldo = a.ldo;
  p.stride_o = a.stride_o;
  p.eps = a.eps;
  p.scale = a.scale;
  p.tall = a.M > a.N;
  const int64_t per = p.tall ? 4 : 8;
  p.vec_out = aligned_to(a.out, per * 2) && a.ldo % per == 0 && (a.batch == 1 || a.stride_o % per == 0);
  return hip_status(moe::launch_orthogonalize(p, steps, a.steps, a.batch, group, static_cast<hipStream_t>(stream)));
}

// ------------------------------------------------------------------ the branch for a few tokens
namespace {

constexpr int64_t kFewTokens = 16;

moe_status check_few(const moe_config* cfg) {
  moe_plan p;
  const moe_status st = check_dropless(cfg, &p);
  if (st != MOE_OK) return st;
  if (cfg->top_k > cfg->n_experts) return MOE_ERR_INVALID_ARG;
  return cfg->T > kFewTokens ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

int64_t carve_few(const moe_config* c, float* logits, int32_t* topk, float* gates, void* ws, moe::Few* f) {
  const int64_t T = c->T, L = c->d_latent, E = c->n_experts, k = c->top_k, F = c->d_ff, R = T * k;
  const int64_t W = c->n_shared > 0 ? (int64_t)c->n_shared * c->d_ff_shared : 0, most = R < E ? R : E;
  Carver cv{static_cast<char*>(ws), 0};
  auto pick = [&](void* given, int64_t bytes) {
    void* q = cv.take(bytes);
    return given ? given : q;
  };
  f->z = static_cast<uint16_t*>(cv.take(3 * T * L * 2));
  f->hs = static_cast<uint16_t*>(cv.take(2 * T * W * 2));
  f->logits = static_cast<float*>(pick(logits, T * E * 4));
  f->topk = static_cast<int32_t*>(pick(topk, R * 4));
  f->gates = static_cast<float*>(pick(gates, R * 4));
  f->n_act = static_cast<int32_t*>(cv.take(4));
  f->act = static_cast<int32_t*>(cv.take(most * 4));
  f->most = (int)most;
  f->rows = static_cast<int32_t*>(cv.take(most * 16 * 4));
  f->h = static_cast<uint16_t*>(cv.take(2 * R * F * 2));
  f->o = static_cast<float*>(cv.take(R * L * 4));
  f->ylat = static_cast<uint16_t*>(cv.take(2 * T * L * 2));
  f->ypart = static_cast<float*>(cv.take(W > 0 ? T * c->d_model * 4 : 0));
  f->counters = static_cast<int32_t*>(cv.take(moe::few_counter_ints((int)L) * 4));
  return cv.used;
}

}  // namespace

MOE_API moe_status moe_forward_few_ws_bytes(const moe_config* cfg, size_t* bytes) {
  const moe_status st = check_few(cfg);
  if (st != MOE_OK) return st;
  if (!bytes) return MOE_ERR_INVALID_ARG;
  moe::Few f{};
  *bytes = (size_t)carve_few(cfg, nullptr, nullptr, nullptr, nullptr, &f);
  return MOE_OK;
}

MOE_API moe_status moe_forward_few(const moe_config* cfg, const moe_weights* w, const void* x, const void* residual,
                                   void* y, float* logits, int32_t* topk_idx, float* gates, void* ws, size_t ws_bytes,
                                   void* stream) {
  const moe_status st = check_few(cfg);
  if (st != MOE_OK) return st;
  if (!w) return MOE_ERR_INVALID_ARG;
  for (const void* p : {w->w_latent, w->w_router, w->w_gate, w->w_up, w->w_down, w->w_up_proj})
    if (!p || !aligned16(p)) return MOE_ERR_INVALID_ARG;
  if (cfg->n_shared > 0)
    for (const void* p : {w->ws_gate, w->ws_up, w->ws_down})
      if (!p || !aligned16(p)) return MOE_ERR_INVALID_ARG;
  if (!aligned_to(w->router_bias, 4) || !aligned16(residual) || !aligned_to(logits, 4) || !aligned_to(topk_idx, 4) ||
      !aligned_to(gates, 4))
    return MOE_ERR_INVALID_ARG;
  if (cfg->T == 0) return MOE_OK;
  if (!x || !y || !aligned16(x) || !aligned16(y)) return MOE_ERR_INVALID_ARG;
  moe::Few f{};
  if (!ws || !aligned256(ws) || (int64_t)ws_bytes < carve_few(cfg, nullptr, nullptr, nullptr, nullptr, &f))
    return MOE_ERR_WORKSPACE;
  carve_few(cfg, logits, topk_idx, gates, ws, &f);
  auto bf16 = [](const void* p) { return static_cast<const uint16_t*>(p); };
  f.T = (int)cfg->T;
  f.D = cfg->d_model;
  f.L = cfg->d_latent;
  f.E = cfg->n_experts;
  f.k = cfg->top_k;
  f.F = cfg->d_ff;
  f.S = cfg->n_shared;
  f.Fs = cfg->n_shared > 0 ? cfg->d_ff_shared : 0;
  f.x = bf16(x);
  f.res = bf16(residual);
  f.y = static_cast<uint16_t*>(y);
  f.w_latent = bf16(w->w_latent);
  f.w_router = bf16(w->w_router);
  f.bias = w->router_bias;
  f.w_gate = bf16(w->w_gate);
  f.w_up = bf16(w->w_up);
  f.w_down = bf16(w->w_down);
  f.w_up_proj = bf16(w->w_up_proj);
  f.ws_gate = bf16(w->ws_gate);
  f.ws_up = bf16(w->ws_up);
  f.ws_down = bf16(w->ws_down);
  return hip_status(moe::launch_few(f, static_cast<hipStream_t>(stream)));
}

// ------------------------------------------------------------------ which kernels a call takes
// For tests (no part of moe.h): tests that are to reach a kernel ask here
// whether their sizes still do.  -1: refused.
//   linear    bits 0-2: 0 nothing, 1 + tile class, 5 straight from memory; 3: operands by way of registers; 4, 5: x, w
//             copied; 6: K shared
//   backward  bits 0-2: 1 + tile class; 3-5 likewise; 6, 7: K of dw, of dx shared; 8: d made
//   updates   of the first group: bits 0-2, 3-5: 1 + tile class of A and B, of X; 6: both fp16 numbers in the products
namespace {
void* const kAnyWs = reinterpret_cast<void*>(uintptr_t(256));
}
MOE_API int moe_linear_form(const moe_linear_args* args) {
  if (check_linear(args) != MOE_OK) return -1;
  if (args->M == 0 || args->N == 0) return 0;
  if (moe::linear_streams(args->M, args->N, args->K)) return 5;
  LinearWs w;
  carve_linear(args, kAnyWs, &w);
  return !w.fits ? -1
                 : (1 + w.plan.cls) | w.regs << 3 | (w.x != nullptr) << 4 | (w.w != nullptr) << 5 |
                       (w.plan.shares > 1) << 6;
}
MOE_API int moe_linear_backward_form(const moe_linear_grad* args) {
  if (check_linear_grad(args) != MOE_OK) return -1;
  LinearGradWs w;
  carve_linear_grad(args, kAnyWs, &w);
  return !w.fits ? -1
                 : (1 + w.dw.cls) | w.regs << 3 | (w.x != nullptr) << 4 | (w.w != nullptr) << 5 |
                       (w.part_dw != nullptr) << 6 | (w.part_dx != nullptr) << 7 | (w.d != nullptr) << 8;
}
MOE_API int moe_orthogonalize_form(const moe_ortho_args* args) {
  moe::OrthoStep steps[kMaxOrthoSteps];
  if (check_ortho(args, steps) != MOE_OK) return -1;
  if (args->batch == 0 || args->M == 0 || args->N == 0) return 0;
  moe::Ortho p{};
  int64_t group;
  carve_ortho(args, kAnyWs, &p, &group);
  const moe::OrthoForm f = moe::ortho_form(p, group);
  return (1 + f.gram) | (1 + f.update) << 3 | f.split << 6;
}
