// Launch interfaces of the feed-forward calls (not part of the public ABI).
#pragma once
#include "svq_internal.h"

#include "../../include/svq_ffn.h"

namespace svq {

// ---- host code shared with svq_host.cpp ------------------------------------
svq_status linear_epi(const svq_handle *w, int32_t count, const void *const *x, const int64_t *ldx, int64_t m,
                      void *const *y, const int64_t *ldy, svq_dtype ydt, const EpiArgs *epi,
                      void *workspace, size_t *workspace_bytes, void *stream);
svq_status check_handle(const svq_handle *w);
MatView matrix_view(const svq_handle *w);
int compute_units();  // of the current device

// ---- elementwise steps -------------------------------------------------------
struct GluArgs {
  const float *g, *u;  // [rows][ldp]
  int64_t rows, ldp;
  const void *bias_g, *bias_u;  // [n] or null
  int32_t bias_f32, act;
  void *y;
  int64_t ldy;
  int32_t n, ydt;
};
hipError_t launch_glu(const GluArgs &a, hipStream_t s);

// One row through both matrices in one launch (R row tiles per block).
constexpr int GLU_HALF = 65536;  // LDS offset of the second matrix's half of a block
struct GluFusedArgs {
  MatView gate, up;
  const uint16_t *x;
  const void *bias_g, *bias_u;
  int32_t bias_f32, act;
  void *y;
  int32_t ydt, R;
};
size_t glu_fused_smem(int k, int units, int bd_gate, int bd_up, int R);  // LDS, or 0: does not fit
hipError_t launch_glu_fused(const GluFusedArgs &a, hipStream_t s);

struct CombineArgs {
  const float *d;  // [m * topk][ldd]
  int64_t ldd;
  const int32_t *ids;
  const float *weights;
  int64_t m;
  int32_t topk, num_experts;
  const void *res;
  int64_t ldr;
  int32_t res_f32;
  void *y;
  int64_t ldy;
  int32_t n, ydt;
};
hipError_t launch_combine(const CombineArgs &a, hipStream_t s);

// ---- beyond 16 rows --------------------------------------------------------
// One matrix with its epilogue, or a gated pair (job 0 the gate), on the
// 256 x 256 tile (bm 256) or the 64 x 256 tile.
struct FfnGemmJob {
  MatView w;
  uint16_t *xb;  // fp16 activations in fragment order (workspace)
  float *part;   // fp32 sums of the K ranges [splits][m_pad][part_ld], columns from the first
                 // n-tile that has any (workspace)
  int32_t xexp;  // -xscale_log2 of the matrix's exact split
};
struct FfnGemmArgs {
  FfnGemmJob job[2];
  int32_t jobs, m, bm, m_pad, tiles_m, tiles_n;
  // tiles 0 .. full - 1 of each job are summed by one block; the rest by
  // `splits` blocks of `ups` units, whose partial tiles the reduce launch joins
  int32_t full, splits, ups, part_ld;
  int32_t rpb, csplit;  // prep: rows per block, chunk ranges
  const uint16_t *x;
  int64_t ldx;
  int32_t *rs;    // exponents of the inverse row scales [m_pad] (workspace)
  float *swap;    // gated pair, whole tiles: [full][2] tiles of 256 x 256 sums
  int32_t *cnt;   // and their arrivals
  int32_t n_cnt;
  int32_t ydt, yvec;
  void *y;
  int64_t ldy;
  EpiArgs epi;         // gated pair: act, and the up matrix's bias
  const void *bias_g;  // the gate's bias
};
hipError_t launch_ffn_gemm(const FfnGemmArgs &a, bool xvec, hipStream_t s);

// ---- expert layer ---------------------------------------------------------
struct MoeFfnArgs {
  const svq_handle *gate, *up, *down;  // host arrays of num_experts
  int32_t num_experts;
  const void *x;
  int64_t ldx;
  const int32_t *ids;
  const float *weights;
  int64_t m;
  int32_t topk, act;
  const void *res;
  int64_t ldr;
  int32_t res_f32, ydt;
  void *y;
  int64_t ldy;
};
// The per-slot form: few slots (see there) whose rows fit a block's LDS.
bool moe_ffn_few_fits(const svq_handle *gate, const svq_handle *up, const svq_handle *down, int32_t num_experts,
                      int64_t slots);
// ws null: only *need.
hipError_t launch_moe_ffn_few(const MoeFfnArgs &f, void *ws, size_t *need, hipStream_t s);
// The grouped form; every matrix has an exact split (its rows are staged in
// LDS as fp16, one at a time if need be, so any width up to SVQ_MAX_K fits).
// MOE_FEW_MAX_INNER: the widest inner row that svq_moe_ffn takes for up to 64
// slots (a documented refusal, which callers may rely on).
constexpr int MOE_FEW_MAX_INNER = 36 * 1024;
hipError_t launch_moe_ffn_grouped(const MoeFfnArgs &f, void *ws, size_t *need, hipStream_t s);

// ---- router --------------------------------------------------------------------
constexpr int ROUTE_MAX_TOPK = 32;
// Tokens summed on the vector units, at most (32 tokens: 10.3 us a call
// against 13.7 on the matrix cores; 64: 13.3 and 13.9; 128: 16.1 and 14.0).
constexpr int ROUTE_FEW = 64;
struct RouteArgs {
  const uint16_t *x;
  int64_t m, ldx;
  const void *w;  // [num_experts][ldw], bf16 or fp32 (w_f32)
  int64_t ldw;
  const float *select_bias;
  int32_t k, num_experts, topk, score, renormalize, w_f32;
  int32_t vec;  // k a multiple of 8, every row 16-byte aligned
  float scale;
  int32_t *ids;
  float *weights;
  double *logits;  // [m][num_experts] (workspace)
};
hipError_t launch_route(const RouteArgs &a, int cus, hipStream_t s);

}  // namespace svq
