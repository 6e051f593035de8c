// Host side of the feed-forward calls (include/svq_ffn.h): argument checks,
// workspace layout and dispatch.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstring>

#include "svq_ffn.h"

using namespace svq;

namespace svq {
size_t glu_fused_smem(int k, int units, int bd_gate, int bd_up, int R) {
  const size_t g = gf_lds(bd_gate, k, units, 1, R).total, u = gf_lds(bd_up, k, units, 1, R).total;
  return g <= (size_t)GLU_HALF && GLU_HALF + u <= GV_LDS_LIMIT ? GLU_HALF + u : 0;
}
}  // namespace svq

namespace {

bool valid_dt(svq_dtype t) { return t == SVQ_BF16 || t == SVQ_F32; }
bool valid_act(svq_act a) { return (int)a >= SVQ_ACT_NONE && (int)a <= SVQ_ACT_GELU_TANH; }
size_t size_of(svq_dtype t) { return t == SVQ_F32 ? 4 : 2; }
bool aligned(const void *p, int64_t row_elems, size_t esz, size_t to) {
  return (((uintptr_t)p) | ((uintptr_t)row_elems * esz)) % to == 0;
}
int64_t pad4(int64_t n) { return (n + 3) / 4 * 4; }
// Workspace regions start at multiples of 256 bytes from its base and are
// read in 16-byte pieces.
bool bad_workspace(const void *ws) { return ((uintptr_t)ws & 15) != 0; }

bool has_split(const svq_handle *w) {
  return w->xscale_log2 != SVQ_NO_EXACT_SPLIT && w->xscale_log2 >= -120 && w->xscale_log2 <= 120;
}

// Tiles of a job that one block sums whole, and the K ranges of the others.
struct TilePlan {
  int full, splits, ups;
};
// 64-row tiles: all in ranges, for about two blocks per compute unit.
// 256-row tiles, one block per compute unit: rounds of whole tiles, then the
// tiles that would fill only a part of the last round in K ranges; the number
// of rounds and ranges that takes the least time when a round of blocks costs
// UNIT a unit of 512 channels and EDGE for its start and its stores, and a
// reduce launch follows partial tiles.  (Either all tiles whole or all in
// ranges: gated pair 9728 x 2560 at 2048 rows 251 us against 239, at 1024 rows
// 160 against 142; one 9728 x 2560 matrix with a
// residual at 2048 rows 235 against 179, 158 since.)
TilePlan tile_plan(int tiles, int jobs, int units, int bm) {
  const int cus = compute_units();
  if (bm == 64) {
    const int all = tiles * jobs;
    const int64_t per = all >= 2 * cus ? units : ((int64_t)all * units + 2 * cus - 1) / (2 * cus);
    return {0, (int)((units + per - 1) / per), (int)per};
  }
  constexpr double UNIT = 13.5, EDGE = 8.0, REDUCE = 4.0, REDUCE_MB = 0.25, TILE_MB = 256 * 256 * 4e-6;  // us
  auto rounds = [&](int64_t blocks, int ups) { return (double)((blocks + cus - 1) / cus) * (ups * UNIT + EDGE); };
  TilePlan best = {tiles, 1, units};
  double t_best = rounds((int64_t)tiles * jobs, units);
  // the last few counts only: still fewer whole rounds just add partial tiles
  const int r_all = (int)((int64_t)tiles * jobs / cus);
  for (int r = r_all > 3 ? r_all - 3 : 0; r <= r_all; ++r) {
    const int full = (int)((int64_t)r * cus / jobs), tail = tiles - full;
    for (int s = 2; s <= units && s <= 16; ++s) {
      const int ups = (units + s - 1) / s;
      if ((units + ups - 1) / ups != s) continue;
      const double t = rounds((int64_t)full * jobs, units) + rounds((int64_t)tail * jobs * s, ups) + REDUCE +
                       REDUCE_MB * TILE_MB * tail * jobs * s;
      if (tail > 0 && t < t_best) {
        t_best = t;
        best = {full, s, ups};
      }
    }
  }
  return best;
}

// The calls beyond 16 rows: plan, workspace, launch (workspace null: only
// *bytes).
svq_status ffn_gemm(const svq_handle *const *w, int jobs, const void *x, int64_t m, int64_t ldx, const EpiArgs &epi,
                    const void *bias_g, void *y, int64_t ldy, svq_dtype ydt, void *workspace, size_t *bytes,
                    void *stream) {
  FfnGemmArgs a;
  std::memset(&a, 0, sizeof(a));
  // 64-row tiles up to two of them; padding to one 256-row tile costs less
  // from there on
  const int bm = m > 128 ? 256 : 64;
  a.jobs = jobs;
  a.m = (int)m;
  a.bm = bm;
  a.m_pad = (int)((m + bm - 1) / bm) * bm;
  a.tiles_m = a.m_pad / bm;
  a.tiles_n = prefill_tiles_n(w[0]->n_tiles);
  if ((int64_t)a.tiles_m * a.tiles_n > (1 << 28)) return SVQ_ERR_UNSUPPORTED;  // tile indexes are 32-bit
  const int units = w[0]->units, tiles = a.tiles_m * a.tiles_n;
  const TilePlan plan = tile_plan(tiles, jobs, units, bm);
  a.full = plan.full;
  a.splits = plan.splits;
  a.ups = plan.ups;
  const int tail = tiles - a.full;
  a.part_ld = (a.tiles_n - a.full / a.tiles_m) * PREFILL_BN;
  // prep: few rows per block (2 rows of 2560, 4096 and 9728 channels: 246, 77
  // and 136 us a call at 2048 rows; 4: 247, 78, 138; 8: 249, 80, -), chunk
  // ranges for about 512 blocks
  a.rpb = 8;
  while (a.rpb > 2 && prefill_prep_lds(a.rpb, w[0]->k) > 12 * 1024) a.rpb /= 2;
  if (prefill_prep_lds(a.rpb, w[0]->k) + 1024 > GV_LDS_LIMIT) a.rpb = 1;  // k beyond 40000
  const int rows = a.m_pad / a.rpb, nch = units * UNIT_SLOTS / 8;
  const int cs = (512 + rows - 1) / rows < nch / 64 ? (512 + rows - 1) / rows : nch / 64;
  a.csplit = cs < 1 ? 1 : cs;
  size_t off = 0;
  auto take = [&](size_t b) {
    const size_t at = off;
    off += align256(b);
    return at;
  };
  const size_t o_rs = take((size_t)a.m_pad * 4);
  size_t o_xb[2], o_part[2] = {0, 0}, o_swap = 0, o_cnt = 0;
  for (int j = 0; j < jobs; ++j) o_xb[j] = take((size_t)a.m_pad * units * UNIT_SLOTS * 2);
  if (tail > 0)
    for (int j = 0; j < jobs; ++j) o_part[j] = take((size_t)a.splits * a.m_pad * a.part_ld * 4);
  if (jobs == 2 && a.full > 0) {
    o_swap = take((size_t)a.full * 2 * 256 * 256 * 4);
    o_cnt = take((size_t)a.full * 4);
    a.n_cnt = a.full;
  }
  if (!workspace) {
    *bytes = off;
    return SVQ_OK;
  }
  if (!x || !y) return SVQ_ERR_INVALID_ARG;
  if (*bytes < off) return SVQ_ERR_BUFFER_TOO_SMALL;
  uint8_t *ws = (uint8_t *)workspace;
  for (int j = 0; j < jobs; ++j) {
    a.job[j].w = matrix_view(w[j]);
    a.job[j].xb = (uint16_t *)(ws + o_xb[j]);
    a.job[j].part = tail > 0 ? (float *)(ws + o_part[j]) : nullptr;
    a.job[j].xexp = -w[j]->xscale_log2;
  }
  a.rs = (int32_t *)(ws + o_rs);
  if (a.n_cnt) {
    a.swap = (float *)(ws + o_swap);
    a.cnt = (int32_t *)(ws + o_cnt);
  }
  a.x = (const uint16_t *)x;
  a.ldx = ldx;
  a.ydt = (int32_t)ydt;
  a.yvec = aligned(y, ldy, size_of(ydt), 16);
  a.y = y;
  a.ldy = ldy;
  a.epi = epi;
  a.bias_g = bias_g;
  return launch_ffn_gemm(a, aligned(x, ldx, 2, 16), (hipStream_t)stream) == hipSuccess ? SVQ_OK : SVQ_ERR_HIP;
}

// A gated pair of 2..16 rows: the gather or prep launch of svq_linear_batched
// over both matrices, then one launch whose blocks take the same row tiles of
// both (with K ranges, 5..16 rows of more than 4096 channels: a block per
// matrix and range, joined by whichever ends last).
svq_status pair_small(const svq_handle *gate, const svq_handle *up, const void *x, int64_t m, int64_t ldx,
                      PairArgs pa, void *y, int64_t ldy, svq_dtype ydt, void *workspace, size_t *bytes,
                      void *stream) {
  const svq_handle *const w[2] = {gate, up};
  const int U = gate->units, nt = gate->n_tiles;
  const bool exact = m <= EXACT_MAX_M;
  size_t off = 0;
  auto take = [&](size_t b) {
    const size_t at = off;
    off += align256(b);
    return at;
  };
  size_t o_x[2], o_s[2], o_part = 0, o_cnt = 0;
  SbPlan pl = {};
  int R = 1;
  if (exact) {
    // row tiles of both matrices per block: one round of blocks, one per
    // compute unit, while the tiles allow it
    R = (nt + compute_units() - 1) / compute_units();
    R = R < 1 ? 1 : (R > GV_MAX_R ? GV_MAX_R : R);
    for (int j = 0; j < 2; ++j) {
      o_x[j] = take((size_t)m * U * GV_XG_UNIT_BYTES);
      o_s[j] = take((size_t)U * 16);
    }
  } else {
    pl = sb_plan(nt, U, sb_block_items(2 * (int64_t)nt * U, compute_units()));
    for (int j = 0; j < 2; ++j) {
      o_x[j] = take((size_t)U * SB_XA_UNIT_BYTES);
      o_s[j] = take((size_t)U * 16 * 4);
    }
    if (pl.splits > 1) {  // K ranges meet through memory
      o_part = take((size_t)pl.groups * pl.tiles * 2 * pl.splits * 1024);
      o_cnt = take((size_t)pl.groups * 4);
      pa.n_cnt = pl.groups;
    }
  }
  if (!workspace) {
    *bytes = off;
    return SVQ_OK;
  }
  if (!x || !y) return SVQ_ERR_INVALID_ARG;
  if (*bytes < off) return SVQ_ERR_BUFFER_TOO_SMALL;
  uint8_t *ws = (uint8_t *)workspace;
  if (pa.n_cnt) {
    pa.part = (float *)(ws + o_part);
    pa.cnt = (int32_t *)(ws + o_cnt);
  }
  hipError_t e;
  if (exact) {
    GemvBatch b;
    std::memset(&b, 0, sizeof(b));
    b.count = 2;
    b.m = (int)m;
    b.ydt = (int)ydt;
    b.xvec = aligned(x, ldx, 2, 16);
    b.pair = &pa;
    const int blocks = (nt + R - 1) / R, gather = (int)m * ((U + 3) / 4);
    for (int j = 0; j < 2; ++j) {
      GemvJob &J = b.job[j];
      J.w = matrix_view(w[j]);
      J.x = (const uint16_t *)x;
      J.ldx = ldx;
      J.xg = ws + o_x[j];
      J.xs = (float *)(ws + o_s[j]);
      J.y = y;
      J.ldy = ldy;
      J.R = R;
      J.block_begin = b.starts.first[j] = j * blocks;
      b.gather_starts.first[j] = j * gather;
    }
    b.touch_begin = (2 * gather + 7) / 8 * 8;
    const int bd = gate->bd > up->bd ? gate->bd : up->bd;
    b.red_off = (int32_t)gemv_smem_bytes((int)m, bd, 0);
    e = launch_gemv_batched(b, b.touch_begin + 16, gate->k, 2 * blocks, gemv_smem_bytes((int)m, bd, R),
                            (hipStream_t)stream);
  } else {
    SbBatch b;
    std::memset(&b, 0, sizeof(b));
    b.count = 2;
    b.m = (int)m;
    b.ydt = (int)ydt;
    b.pair = &pa;
    for (int j = 0; j < 2; ++j) {
      SbJob &J = b.job[j];
      J.w = matrix_view(w[j]);
      J.x = (const uint16_t *)x;
      J.ldx = ldx;
      J.y = y;
      J.ldy = ldy;
      J.tiles = pl.tiles;
      J.upr = pl.upr;
      J.groups = pl.groups;
      J.splits = pl.splits;
      J.xa = ws + o_x[j];
      J.xs = (float *)(ws + o_s[j]);
      J.xinv = std::ldexp(1.0f, -w[j]->xscale_log2);
      J.part = pa.part;  // the pair's ranges share one exchange and its arrivals,
      J.cnt = pa.cnt;    // which either prep form clears
      J.block_begin = b.starts.first[j] = j * pl.groups * pl.splits;
      J.prep_begin = b.prep_starts.first[j] = j * U;
    }
    e = launch_sb(b, 2 * U, 2 * pl.groups * pl.splits, (hipStream_t)stream);
  }
  return e == hipSuccess ? SVQ_OK : SVQ_ERR_HIP;
}

}  // namespace

extern "C" {

svq_status svq_linear_epilogue(const svq_handle *w, const void *x, int64_t m, int64_t ldx,
                               const svq_epilogue *ep, void *y, int64_t ldy, svq_dtype ydt,
                               void *workspace, size_t *workspace_bytes, void *stream) {
  if (!w || !ep || !workspace_bytes || bad_workspace(workspace)) return SVQ_ERR_INVALID_ARG;
  const svq_status st = check_handle(w);
  if (st != SVQ_OK) return st;
  if (!valid_act(ep->act) || (ep->bias && !valid_dt(ep->bias_dt))) return SVQ_ERR_INVALID_ARG;
  if (ep->residual && (!valid_dt(ep->residual_dt) || ep->ldr < w->n)) return SVQ_ERR_INVALID_ARG;
  EpiArgs e;
  std::memset(&e, 0, sizeof(e));
  e.act = (int32_t)ep->act;
  e.bias = ep->bias;
  e.bias_f32 = ep->bias_dt == SVQ_F32;
  e.bias_vec = aligned(ep->bias, 0, 1, 4 * size_of(ep->bias_dt));
  if (ep->residual) {
    e.res = ep->residual;
    e.ldr = ep->ldr;
    e.res_f32 = ep->residual_dt == SVQ_F32;
    e.res_vec = aligned(ep->residual, ep->ldr, size_of(ep->residual_dt), 4 * size_of(ep->residual_dt));
    if (ep->residual == y && (ep->ldr != ldy || ep->residual_dt != ydt)) return SVQ_ERR_INVALID_ARG;
  }
  if (m > SB_MAX_M && m <= (1 << 24) && has_split(w)) {
    if (!valid_dt(ydt) || ldx < w->k || ldy < w->n) return SVQ_ERR_INVALID_ARG;
    return ffn_gemm(&w, 1, x, m, ldx, e, nullptr, y, ldy, ydt, workspace, workspace_bytes, stream);
  }
  return linear_epi(w, 1, workspace ? &x : nullptr, &ldx, m, workspace ? &y : nullptr, &ldy, ydt, &e, workspace,
                    workspace_bytes, stream);
}

svq_status svq_linear_glu(const svq_handle *gate, const svq_handle *up, const void *x, int64_t m,
                          int64_t ldx, svq_act act, const void *bias_gate, const void *bias_up,
                          svq_dtype bias_dt, void *y, int64_t ldy, svq_dtype ydt,
                          void *workspace, size_t *workspace_bytes, void *stream) {
  if (!gate || !up || !workspace_bytes || bad_workspace(workspace)) return SVQ_ERR_INVALID_ARG;
  svq_status st = check_handle(gate);
  if (st == SVQ_OK) st = check_handle(up);
  if (st != SVQ_OK) return st;
  if (gate->n != up->n || gate->k != up->k) return SVQ_ERR_INVALID_ARG;
  if (!valid_act(act) || !valid_dt(ydt)) return SVQ_ERR_INVALID_ARG;
  if ((bias_gate || bias_up) && !valid_dt(bias_dt)) return SVQ_ERR_INVALID_ARG;
  if (m < 1 || m > (1 << 24) || ldx < gate->k || ldy < gate->n) return SVQ_ERR_INVALID_ARG;
  if (m == 1) {
    // one launch while both halves of a block fit in LDS; row tiles per block
    // so that one round of blocks, one per compute unit, covers the matrices
    int R = (gate->n_tiles + compute_units() - 1) / compute_units();
    R = R > GF_MAX_R ? GF_MAX_R : R;
    while (R > 1 && !glu_fused_smem(gate->k, gate->units, gate->bd, up->bd, R)) --R;
    if (glu_fused_smem(gate->k, gate->units, gate->bd, up->bd, R)) {
      const size_t need = 256;  // unused: everything stays in LDS
      if (!workspace) {
        *workspace_bytes = need;
        return SVQ_OK;
      }
      if (!x || !y) return SVQ_ERR_INVALID_ARG;
      if (*workspace_bytes < need) return SVQ_ERR_BUFFER_TOO_SMALL;
      GluFusedArgs a;
      std::memset(&a, 0, sizeof(a));
      a.gate = matrix_view(gate);
      a.up = matrix_view(up);
      a.x = (const uint16_t *)x;
      a.bias_g = bias_gate;
      a.bias_u = bias_up;
      a.bias_f32 = bias_dt == SVQ_F32;
      a.act = (int32_t)act;
      a.y = y;
      a.ydt = (int32_t)ydt;
      a.R = R;
      return launch_glu_fused(a, (hipStream_t)stream) == hipSuccess ? SVQ_OK : SVQ_ERR_HIP;
    }
  }
  if (m > SB_MAX_M && has_split(gate) && has_split(up)) {
    EpiArgs e;
    std::memset(&e, 0, sizeof(e));
    e.act = (int32_t)act;
    e.bias = bias_up;
    e.bias_f32 = bias_dt == SVQ_F32;
    const svq_handle *const pair[2] = {gate, up};
    return ffn_gemm(pair, 2, x, m, ldx, e, bias_gate, y, ldy, ydt, workspace, workspace_bytes, stream);
  }
  if (m > 1 && m <= SB_MAX_M && (m <= EXACT_MAX_M || (has_split(gate) && has_split(up)))) {
    PairArgs pa;
    std::memset(&pa, 0, sizeof(pa));
    pa.bias_g = bias_gate;
    pa.bias_u = bias_up;
    pa.bias_f32 = bias_dt == SVQ_F32;
    pa.act = (int32_t)act;
    return pair_small(gate, up, x, m, ldx, pa, y, ldy, ydt, workspace, workspace_bytes, stream);
  }
  const int64_t ldp = pad4(gate->n);
  const svq_handle w[2] = {*gate, *up};
  const int64_t lx[2] = {ldx, ldx}, ly[2] = {ldp, ldp};
  size_t inner = 0;
  st = linear_epi(w, 2, nullptr, lx, m, nullptr, ly, SVQ_F32, nullptr, nullptr, &inner, stream);
  if (st != SVQ_OK) return st;
  const size_t part = align256((size_t)m * ldp * 4), need = 2 * part + inner;
  if (!workspace) {
    *workspace_bytes = need;
    return SVQ_OK;
  }
  if (!x || !y) return SVQ_ERR_INVALID_ARG;
  if (*workspace_bytes < need) return SVQ_ERR_BUFFER_TOO_SMALL;
  uint8_t *ws = (uint8_t *)workspace;
  const void *xs[2] = {x, x};
  void *ys[2] = {ws, ws + part};
  st = linear_epi(w, 2, xs, lx, m, ys, ly, SVQ_F32, nullptr, ws + 2 * part, &inner, stream);
  if (st != SVQ_OK) return st;
  GluArgs a;
  std::memset(&a, 0, sizeof(a));
  a.g = (const float *)ws;
  a.u = (const float *)(ws + part);
  a.rows = m;
  a.ldp = ldp;
  a.bias_g = bias_gate;
  a.bias_u = bias_up;
  a.bias_f32 = bias_dt == SVQ_F32;
  a.act = (int32_t)act;
  a.y = y;
  a.ldy = ldy;
  a.n = gate->n;
  a.ydt = (int32_t)ydt;
  return launch_glu(a, (hipStream_t)stream) == hipSuccess ? SVQ_OK : SVQ_ERR_HIP;
}

svq_status svq_moe_route(const void *x, int64_t m, int64_t ldx, const void *w, svq_dtype wdt,
                         int32_t num_experts, int32_t k, int64_t ldw, const float *select_bias,
                         svq_route_score score, int32_t renormalize, float scale, int32_t topk,
                         int32_t *ids, float *weights, void *workspace, size_t *workspace_bytes,
                         void *stream) {
  if (!workspace_bytes || bad_workspace(workspace)) return SVQ_ERR_INVALID_ARG;
  if (num_experts < 1 || num_experts > MAX_EXPERTS) return SVQ_ERR_UNSUPPORTED;
  if (topk < 1 || topk > num_experts) return SVQ_ERR_INVALID_ARG;
  if (topk > ROUTE_MAX_TOPK) return SVQ_ERR_UNSUPPORTED;
  if (m < 1 || m > (1 << 20) || k < 1 || ldx < k || ldw < k) return SVQ_ERR_INVALID_ARG;
  if (k > SVQ_MAX_K) return SVQ_ERR_UNSUPPORTED;
  if (!valid_dt(wdt) || (renormalize != 0 && renormalize != 1)) return SVQ_ERR_INVALID_ARG;
  if (score != SVQ_ROUTE_SOFTMAX && score != SVQ_ROUTE_SIGMOID) return SVQ_ERR_INVALID_ARG;
  if (!std::isfinite(scale)) return SVQ_ERR_INVALID_ARG;
  const size_t need = align256((size_t)m * num_experts * 8);  // the logits
  if (!workspace) {
    *workspace_bytes = need;
    return SVQ_OK;
  }
  if (!x || !w || !ids || !weights) return SVQ_ERR_INVALID_ARG;
  if (*workspace_bytes < need) return SVQ_ERR_BUFFER_TOO_SMALL;
  RouteArgs a;
  std::memset(&a, 0, sizeof(a));
  a.x = (const uint16_t *)x;
  a.m = m;
  a.ldx = ldx;
  a.w = w;
  a.ldw = ldw;
  a.select_bias = select_bias;
  a.k = k;
  a.num_experts = num_experts;
  a.topk = topk;
  a.score = (int32_t)score;
  a.renormalize = renormalize;
  a.w_f32 = wdt == SVQ_F32;
  a.vec = k % 8 == 0 && aligned(x, ldx, 2, 16) && aligned(w, ldw, size_of(wdt), 16);
  a.scale = scale;
  a.ids = ids;
  a.weights = weights;
  a.logits = (double *)workspace;
  return launch_route(a, compute_units(), (hipStream_t)stream) == hipSuccess ? SVQ_OK : SVQ_ERR_HIP;
}

svq_status svq_moe_ffn(const svq_handle *gate, const svq_handle *up, const svq_handle *down,
                       int32_t num_experts, const void *x, int64_t ldx, const int32_t *expert_ids,
                       const float *weights, int64_t m, int32_t topk, svq_act act,
                       const void *residual, int64_t ldr, svq_dtype residual_dt, void *y,
                       int64_t ldy, svq_dtype ydt, void *workspace, size_t *workspace_bytes,
                       void *stream) {
  if (!gate || !up || !down || !workspace_bytes || bad_workspace(workspace)) return SVQ_ERR_INVALID_ARG;
  if (num_experts < 1 || num_experts > MAX_EXPERTS) return SVQ_ERR_UNSUPPORTED;
  if (topk < 1 || topk > num_experts || m < 1 || m > (1 << 20)) return SVQ_ERR_INVALID_ARG;
  if (!valid_act(act) || !valid_dt(ydt)) return SVQ_ERR_INVALID_ARG;
  const svq_handle *const sets[3] = {gate, up, down};
  for (int c = 0; c < 3; ++c)
    for (int32_t e = 0; e < num_experts; ++e) {
      const svq_status st = check_handle(&sets[c][e]);
      if (st != SVQ_OK) return st;
      if (sets[c][e].n != sets[c][0].n || sets[c][e].k != sets[c][0].k) return SVQ_ERR_INVALID_ARG;
    }
  if (gate->n != up->n || gate->k != up->k || down->k != gate->n) return SVQ_ERR_INVALID_ARG;
  if (ldx < gate->k || ldy < down->n) return SVQ_ERR_INVALID_ARG;
  if (residual && (!valid_dt(residual_dt) || ldr < down->n)) return SVQ_ERR_INVALID_ARG;
  const int64_t S = m * topk;
  const bool few = moe_ffn_few_fits(gate, up, down, num_experts, S);
  bool split = true;
  for (int c = 0; c < 3 && !few; ++c)
    for (int32_t e = 0; e < num_experts; ++e) split = split && has_split(&sets[c][e]);
  // up to 64 slots the inner width has its documented limit
  const bool grouped = split && (S > 64 || down->k <= MOE_FEW_MAX_INNER);
  // what is left runs as separate products, which need more slots than the
  // per-slot launch takes
  if (!few && !grouped && S <= 64) return SVQ_ERR_UNSUPPORTED;
  if (few || grouped) {
    MoeFfnArgs fa;
    std::memset(&fa, 0, sizeof(fa));
    fa.gate = gate;
    fa.up = up;
    fa.down = down;
    fa.num_experts = num_experts;
    fa.x = x;
    fa.ldx = ldx;
    fa.ids = expert_ids;
    fa.weights = weights;
    fa.m = m;
    fa.topk = topk;
    fa.act = (int32_t)act;
    fa.res = residual;
    fa.ldr = ldr;
    fa.res_f32 = residual_dt == SVQ_F32;
    fa.y = y;
    fa.ldy = ldy;
    fa.ydt = (int32_t)ydt;
    size_t need = 0;
    const auto launch = few ? launch_moe_ffn_few : launch_moe_ffn_grouped;
    if (launch(fa, nullptr, &need, nullptr) != hipSuccess) return SVQ_ERR_HIP;
    if (!workspace) {
      *workspace_bytes = need;
      return SVQ_OK;
    }
    if (!x || !expert_ids || !weights || !y) return SVQ_ERR_INVALID_ARG;
    if (residual == y && (ldr != ldy || residual_dt != ydt)) return SVQ_ERR_INVALID_ARG;
    if (*workspace_bytes < need) return SVQ_ERR_BUFFER_TOO_SMALL;
    return launch(fa, workspace, &need, (hipStream_t)stream) == hipSuccess ? SVQ_OK : SVQ_ERR_HIP;
  }
  const int32_t f = gate->n, n = down->n;
  const int64_t ldf = pad4(f), ldh = (f + 7) / 8 * 8, ldd = pad4(n);
  // workspace: gate and up sums, the inner activation, the slots' outputs,
  // then the products' own workspace (used in turn)
  size_t inner = 0, ws1 = 0, ws2 = 0;
  svq_status st = svq_moe_linear(gate, num_experts, nullptr, ldx, 0, nullptr, m, topk, nullptr, ldf, SVQ_F32,
                                 nullptr, &ws1, stream);
  if (st == SVQ_OK)
    st = svq_moe_linear(down, num_experts, nullptr, ldh, 1, nullptr, m, topk, nullptr, ldd, SVQ_F32, nullptr,
                        &ws2, stream);
  if (st != SVQ_OK) return st;
  inner = ws1 > ws2 ? ws1 : ws2;
  const size_t b_g = align256((size_t)S * ldf * 4), b_h = align256((size_t)S * ldh * 2),
               b_d = align256((size_t)S * ldd * 4);
  const size_t need = 2 * b_g + b_h + b_d + inner;
  if (!workspace) {
    *workspace_bytes = need;
    return SVQ_OK;
  }
  if (!x || !expert_ids || !weights || !y) return SVQ_ERR_INVALID_ARG;
  if (residual == y && (ldr != ldy || residual_dt != ydt)) return SVQ_ERR_INVALID_ARG;
  if (*workspace_bytes < need) return SVQ_ERR_BUFFER_TOO_SMALL;
  uint8_t *ws = (uint8_t *)workspace;
  float *g = (float *)ws, *u = (float *)(ws + b_g);
  uint8_t *h = ws + 2 * b_g;
  float *d = (float *)(ws + 2 * b_g + b_h);
  uint8_t *iw = ws + 2 * b_g + b_h + b_d;
  size_t cap = inner;
  st = svq_moe_linear(gate, num_experts, x, ldx, 0, expert_ids, m, topk, g, ldf, SVQ_F32, iw, &cap, stream);
  if (st == SVQ_OK)
    st = svq_moe_linear(up, num_experts, x, ldx, 0, expert_ids, m, topk, u, ldf, SVQ_F32, iw, &cap, stream);
  if (st != SVQ_OK) return st;
  GluArgs ga;
  std::memset(&ga, 0, sizeof(ga));
  ga.g = g;
  ga.u = u;
  ga.rows = S;
  ga.ldp = ldf;
  ga.act = (int32_t)act;
  ga.y = h;
  ga.ldy = ldh;
  ga.n = f;
  ga.ydt = SVQ_BF16;
  if (launch_glu(ga, (hipStream_t)stream) != hipSuccess) return SVQ_ERR_HIP;
  st = svq_moe_linear(down, num_experts, h, ldh, 1, expert_ids, m, topk, d, ldd, SVQ_F32, iw, &cap, stream);
  if (st != SVQ_OK) return st;
  CombineArgs ca;
  std::memset(&ca, 0, sizeof(ca));
  ca.d = d;
  ca.ldd = ldd;
  ca.ids = expert_ids;
  ca.weights = weights;
  ca.m = m;
  ca.topk = topk;
  ca.num_experts = num_experts;
  ca.res = residual;
  ca.ldr = ldr;
  ca.res_f32 = residual_dt == SVQ_F32;
  ca.y = y;
  ca.ldy = ldy;
  ca.n = n;
  ca.ydt = (int32_t)ydt;
  return launch_combine(ca, (hipStream_t)stream) == hipSuccess ? SVQ_OK : SVQ_ERR_HIP;
}

}  // extern "C"
