// Stand-ins for the feed-forward launchers (see launch_checks.cpp for those
// of the products): every workspace region a launch is handed lies inside the
// queried workspace, regions do not overlap, and every tile's units lie inside
// its matrix.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <utility>
#include <vector>

#include "../../bit_spherical_vector_amd/csrc/svq_ffn.h"

namespace check {
extern const uint8_t *ws_base;
extern size_t ws_bytes;
extern long launches, loads_checked;
void check_ws(const void *p, size_t bytes, const char *what);
void check_code_load(const svq::MatView &w, size_t off, const char *what);
}  // namespace check

#define CHECK(cond, ...)                                                                      \
  do {                                                                                        \
    if (!(cond)) {                                                                            \
      std::fprintf(stderr, "launch check failed (%s:%d): %s: ", __FILE__, __LINE__, #cond);   \
      std::fprintf(stderr, __VA_ARGS__);                                                      \
      std::fprintf(stderr, "\n");                                                             \
      std::abort();                                                                           \
    }                                                                                         \
  } while (0)

namespace {
struct Regions {
  std::vector<std::pair<const uint8_t *, size_t>> r;
  void add(const void *p, size_t bytes, const char *what) {
    check::check_ws(p, bytes, what);
    r.emplace_back((const uint8_t *)p, bytes);
  }
  ~Regions() {
    std::sort(r.begin(), r.end());
    for (size_t i = 1; i < r.size(); ++i)
      CHECK(r[i - 1].first + r[i - 1].second <= r[i].first, "regions %zu and %zu overlap", i - 1, i);
  }
};
}  // namespace

namespace check {
long mixed = 0;  // launches of whole tiles and K ranges
}
namespace svq {

hipError_t launch_ffn_gemm(const FfnGemmArgs &a, bool, hipStream_t) {
  ++check::launches;
  Regions R;
  CHECK(a.bm == 64 || a.bm == 256, "bm %d", a.bm);
  CHECK(a.m_pad >= a.m && a.m_pad % a.bm == 0 && a.tiles_m * a.bm == a.m_pad, "rows");
  CHECK(a.rpb >= 1 && a.rpb <= 8 && 32 % a.rpb == 0, "rows per prep block %d", a.rpb);
  CHECK(prefill_prep_lds(a.rpb, a.job[0].w.k) + 64 <= GV_LDS_LIMIT, "prep LDS");
  R.add(a.rs, (size_t)a.m_pad * 4, "row scales");
  const int tail = a.tiles_m * a.tiles_n - a.full;  // tiles in K ranges
  CHECK(a.full >= 0 && tail >= 0 && (a.bm == 256 || a.full == 0), "whole tiles %d, others %d", a.full, tail);
  for (int j = 0; j < a.jobs; ++j) {
    const MatView &w = a.job[j].w;
    CHECK(a.tiles_n * 256 >= w.n, "columns");
    CHECK(a.full / a.tiles_m * 256 + a.part_ld == a.tiles_n * 256, "columns of the K ranges");
    R.add(a.job[j].xb, (size_t)a.m_pad * w.units * UNIT_SLOTS * 2, "activations");
    CHECK((a.job[j].part != nullptr) == (tail > 0), "partial tiles");
    if (tail > 0) R.add(a.job[j].part, (size_t)a.splits * a.m_pad * a.part_ld * 4, "partial tiles");
    CHECK(a.splits >= 1 && a.splits * a.ups >= w.units && (a.splits - 1) * a.ups < w.units, "K ranges");
    for (int s = 0; s < a.splits; ++s)
      for (int u = s * a.ups; u < std::min(w.units, (s + 1) * a.ups); ++u)
        for (int rt : {0, w.n_tiles - 1})
          check::check_code_load(w, w.off_codes + ((size_t)rt * w.units + u) * UNIT_BYTES, "ffn gemm");
  }
  if (a.full > 0 && a.jobs == 2) {
    R.add(a.swap, (size_t)a.full * 2 * 65536 * 4, "exchange tiles");
    R.add(a.cnt, (size_t)a.full * 4, "arrivals");
    CHECK(a.n_cnt == a.full, "arrivals cleared");
  } else {
    CHECK(a.n_cnt == 0, "no arrivals");
  }
  check::mixed += a.full > 0 && tail > 0;
  return hipSuccess;
}

hipError_t launch_glu_fused(const GluFusedArgs &a, hipStream_t) {
  ++check::launches;
  const size_t smem = glu_fused_smem(a.gate.k, a.gate.units, a.gate.bd, a.up.bd, a.R);
  CHECK(smem > 0 && smem <= GV_LDS_LIMIT && a.R >= 1 && a.R <= GF_MAX_R, "R %d LDS %zu", a.R, smem);
  return hipSuccess;
}
hipError_t launch_glu(const GluArgs &a, hipStream_t) {
  ++check::launches;
  CHECK(a.ldp >= a.n && a.ldp % 4 == 0, "ldp");
  Regions R;
  R.add(a.g, (size_t)a.rows * a.ldp * 4, "gate sums");
  R.add(a.u, (size_t)a.rows * a.ldp * 4, "up sums");
  return hipSuccess;
}
hipError_t launch_combine(const CombineArgs &a, hipStream_t) {
  ++check::launches;
  CHECK(a.ldd >= a.n && a.ldd % 4 == 0, "ldd");
  check::check_ws(a.d, (size_t)a.m * a.topk * a.ldd * 4, "slot outputs");
  return hipSuccess;
}
hipError_t launch_route(const RouteArgs &a, int cus, hipStream_t) {
  ++check::launches;
  CHECK(cus > 0, "compute units");
  check::check_ws(a.logits, (size_t)a.m * a.num_experts * 8, "logits");
  return hipSuccess;
}
// the expert layer's own plans live beside its kernels
bool moe_ffn_few_fits(const svq_handle *, const svq_handle *, const svq_handle *, int32_t, int64_t slots) {
  return slots <= 64;
}
hipError_t launch_moe_ffn_few(const MoeFfnArgs &, void *, size_t *need, hipStream_t) {
  *need = 256;
  return hipSuccess;
}
hipError_t launch_moe_ffn_grouped(const MoeFfnArgs &, void *, size_t *need, hipStream_t) {
  *need = 256;
  return hipSuccess;
}

}  // namespace svq
