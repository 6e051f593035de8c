// Drives the feed-forward calls' host code on the CPU (see ffn_checks.cpp):
// every call twice, the workspace query and the call itself on a workspace of
// exactly that size, over ragged shapes and row counts from one to thousands.
// Built with AddressSanitizer and UndefinedBehaviorSanitizer by
// tests/test_ffn_host.py.
#include <cstdio>
#include <cstdlib>
#include <functional>
#include <random>
#include <vector>

#include "../../include/svq_ffn.h"

namespace check {
extern const uint8_t *ws_base;
extern size_t ws_bytes;
extern long launches, loads_checked, mixed;
}

static int fails = 0;
#define EXPECT(cond, ...)                           \
  do {                                              \
    if (!(cond)) {                                  \
      std::fprintf(stderr, "harness: %s: ", #cond); \
      std::fprintf(stderr, __VA_ARGS__);            \
      std::fprintf(stderr, "\n");                   \
      ++fails;                                      \
    }                                               \
  } while (0)

static std::vector<void *> owned;

static svq_handle packed(int n, int k, int bd, unsigned seed, bool split = true) {
  std::mt19937 g(seed);
  std::vector<uint8_t> codes(((size_t)n * (k / 8) * 18 + 7) / 8);
  for (auto &b : codes) b = (uint8_t)g();
  std::vector<uint16_t> cb((size_t)8 << bd), rad((size_t)1 << (10 - bd));
  for (auto &v : cb) v = (uint16_t)(0x3000 + (g() & 0x7FF));
  for (size_t r = 0; r < rad.size(); ++r) rad[r] = (uint16_t)(0x2C00 + 0x40 * r);
  if (!split) {
    rad[0] = 0x3C01;
    rad[1] = 0x7B53;
    for (int l = 0; l < 8; ++l) cb[l] = 1;
  }
  std::vector<int32_t> perm(k);
  for (int p = 0; p < k; ++p) perm[p] = k - 1 - p;
  const svq_matrix_desc d{n, k, bd, 10 - bd, codes.data(), cb.data(), rad.data(), perm.data()};
  size_t bytes = 0;
  EXPECT(svq_pack(&d, nullptr, &bytes, nullptr, nullptr) == SVQ_OK, "size %dx%d", n, k);
  void *buf = std::malloc(bytes);
  owned.push_back(buf);
  svq_handle h{};
  EXPECT(svq_pack(&d, buf, &bytes, &h, nullptr) == SVQ_OK, "pack %dx%d", n, k);
  EXPECT((h.xscale_log2 != SVQ_NO_EXACT_SPLIT) == split, "split of %dx%d", n, k);
  return h;
}

// f(workspace, &bytes): queried, run at exactly that size, refused one short
// and at a misaligned address.
static void run(const char *what, const std::function<svq_status(void *, size_t *)> &f) {
  size_t need = 0;
  svq_status st = f(nullptr, &need);
  EXPECT(st == SVQ_OK && need > 0, "%s: query %d", what, (int)st);
  if (st != SVQ_OK) return;
  uint8_t *ws = (uint8_t *)std::aligned_alloc(256, (need + 255) / 256 * 256);
  check::ws_base = ws;
  check::ws_bytes = need;
  size_t cap = need;
  const long before = check::launches;
  st = f(ws, &cap);
  EXPECT(st == SVQ_OK, "%s: call %d", what, (int)st);
  const long after = check::launches;
  cap = need - 1;
  EXPECT(f(ws, &cap) == SVQ_ERR_BUFFER_TOO_SMALL, "%s: one byte short", what);
  cap = need;
  EXPECT(f(ws + 8, &cap) == SVQ_ERR_INVALID_ARG, "%s: misaligned", what);
  EXPECT(check::launches == after && after >= before, "%s: a refused call launched", what);
  std::free(ws);
  check::ws_base = nullptr;
}

int main() {
  const void *x = (const void *)0x100000;  // never dereferenced on the host
  void *y = (void *)0x200000;
  const int ms[] = {1, 2, 4, 5, 16, 17, 63, 64, 65, 128, 129, 255, 256, 257, 300, 515, 2048, 4100};
  const int shapes[][3] = {{1, 8, 7},       {37, 104, 6},    {512, 1024, 8}, {1021, 2560, 6}, {9728, 2560, 7},
                           {2560, 9728, 7}, {64, 20000, 8}, {300, 4608, 6}, {16, 512, 7},    {40, 65536, 6}};
  unsigned seed = 1;
  char what[128];
  for (auto &s : shapes)
    for (bool split : {true, false}) {
      if (!split && s[0] != 37 && s[0] != 300) continue;
      const int n = s[0], k = s[1];
      const svq_handle a = packed(n, k, s[2], seed++, split), b = packed(n, k, 6 + seed % 3, seed, split);
      ++seed;
      for (int m : ms) {
        if ((size_t)m * k > ((size_t)1 << 26)) continue;  // keep the host run short
        for (int variant = 0; variant < 2; ++variant) {
          const svq_dtype out = variant ? SVQ_F32 : SVQ_BF16;
          svq_epilogue ep{};
          if (variant) {
            ep.bias = x;
            ep.bias_dt = SVQ_F32;
            ep.act = SVQ_ACT_SILU;
            ep.residual = y;  // in place
            ep.ldr = n + 3;
            ep.residual_dt = out;
          }
          std::snprintf(what, sizeof(what), "epilogue %dx%d m=%d %d", n, k, m, variant);
          run(what, [&](void *ws, size_t *bytes) {
            return svq_linear_epilogue(&a, x, m, k + 8 * variant, &ep, y, n + 3, out, ws, bytes, nullptr);
          });
          std::snprintf(what, sizeof(what), "glu %dx%d m=%d %d", n, k, m, variant);
          run(what, [&](void *ws, size_t *bytes) {
            return svq_linear_glu(&a, &b, x, m, k, SVQ_ACT_GELU, variant ? x : nullptr, nullptr, SVQ_BF16, y, n, out,
                                  ws, bytes, nullptr);
          });
        }
      }
    }
  for (int m : ms)
    for (int e : {1, 8, 129, 256}) {
      std::snprintf(what, sizeof(what), "route m=%d e=%d", m, e);
      run(what, [&](void *ws, size_t *bytes) {
        return svq_moe_route(x, m, 72, x, SVQ_BF16, e, 72, 72, nullptr, SVQ_ROUTE_SOFTMAX, 1, 1.f, e < 8 ? e : 8,
                             (int32_t *)y, (float *)y, ws, bytes, nullptr);
      });
    }
  for (bool split : {true, false}) {
    std::vector<svq_handle> g, u, d;
    for (int e = 0; e < 4; ++e) {
      g.push_back(packed(72, 40, 7, seed++, split || e != 2));
      u.push_back(packed(72, 40, 7, seed++));
      d.push_back(packed(40, 72, 7, seed++));
    }
    for (int m : {1, 30, 33, 600}) {
      std::snprintf(what, sizeof(what), "moe m=%d split=%d", m, (int)split);
      run(what, [&](void *ws, size_t *bytes) {
        return svq_moe_ffn(g.data(), u.data(), d.data(), 4, x, 40, (const int32_t *)x, (const float *)x, m, 2,
                           SVQ_ACT_SILU, y, 40, SVQ_BF16, y, 40, SVQ_BF16, ws, bytes, nullptr);
      });
    }
  }
  EXPECT(check::mixed > 0, "no plan with a last round in K ranges%s", "");
  for (void *p : owned) std::free(p);
  std::printf("host harness: %ld launches checked, %ld code loads, %d failures\n", check::launches,
              check::loads_checked, fails);
  return fails ? 1 : 0;
}
