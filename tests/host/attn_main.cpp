// Drives the attention calls' host code on the CPU against stand-ins for the
// launchers: every call twice, the workspace query and the call on a workspace
// of exactly that size, over ragged shapes; what the kernels derive from a plan
// (ranges of keys, tiles of rows, bytes of the cache) is checked against plain
// arithmetic.  Built with AddressSanitizer and UndefinedBehaviorSanitizer by
// tests/test_attn_host.py.
#include <algorithm>
#include <cstdio>
#include <cstring>
#include <random>
#include <vector>

#include "../../bit_spherical_vector_amd/csrc/svq_attn.h"

static int fails = 0;
static long launches = 0, checks = 0;
#define EXPECT(cond, ...)                           \
  do {                                              \
    ++checks;                                       \
    if (!(cond)) {                                  \
      std::fprintf(stderr, "harness: %s: ", #cond); \
      std::fprintf(stderr, __VA_ARGS__);            \
      std::fprintf(stderr, "\n");                   \
      ++fails;                                      \
    }                                               \
  } while (0)

static const uint8_t *ws_base;
static size_t ws_bytes;
static std::mt19937 rng(7);
static int64_t pick(int64_t lo, int64_t hi) { return lo + (int64_t)(rng() % (uint64_t)(hi - lo + 1)); }

namespace svq {
int compute_units() { return 256; }

// Every byte of a page block belongs to one slot, side and group.
static void check_layout(const KvView &c) {
  const int ps = 1 << c.page_shift;
  std::vector<uint8_t> used(c.block, 0);
  auto take = [&](int at, int n) {
    for (int i = 0; i < n; ++i) {
      EXPECT(at + i >= 0 && at + i < c.block, "byte %d of %d", at + i, c.block);
      if (at + i < c.block) ++used[at + i];
    }
  };
  for (int s = 0; s < ps; ++s) {
    for (int n = 0; n < c.dim / 8; ++n) take(kv_key_word(c, s, n), 4);
    for (int r = 0; r < 16; ++r) take(kv_value_run(c, s, r), c.dim / 32);
    for (int side = 0; side < 2; ++side)
      for (int g = 0; g < c.groups; ++g) take(kv_param(c, side, s, g), 4);
  }
  for (int i = 0; i < c.block; ++i) EXPECT(used[i] == 1, "byte %d taken %d times", i, used[i]);
  unsigned nibbles = 0;
  for (int j = 0; j < 8; ++j) nibbles |= 1u << kv_nibble(j);
  EXPECT(nibbles == 0xFF, "nibbles %x", nibbles);
}

hipError_t launch_kv_write(const KvWriteArgs &a, hipStream_t) {
  ++launches;
  EXPECT(a.tokens > 0 && a.slots && a.k && a.v, "write");
  return hipSuccess;
}
hipError_t launch_kv_read(const KvReadArgs &a, hipStream_t) {
  ++launches;
  EXPECT(a.tokens > 0 && a.slots && a.k && a.v, "read");
  return hipSuccess;
}

hipError_t launch_attn_prompt(const AttnPromptArgs &a, hipStream_t) {
  ++launches;
  const PromptPlan p = prompt_plan(a.tokens, a.sequences, a.heads, a.kv_heads, 4, compute_units());
  EXPECT(p.tokens >= 1 && p.tokens * p.G <= 128, "tile of %d tokens of %d heads", p.tokens, p.G);
  for (int x = 0; x < 128; ++x) EXPECT(quotient16(x, p.g_mul) == x / p.G, "%d / %d", x, p.G);
  for (int i = 0; i < 64; ++i) {
    const int n = (int)pick(0, (1 << 24) + 127);
    EXPECT(quotient(n, p.tokens_mul) == n / p.tokens, "%d / %d", n, p.tokens);
  }
  // any split of the tokens into the sequences fits the tiles
  int64_t left = a.tokens, tiles = 0;
  for (int s = 0; s < a.sequences; ++s) {
    const int64_t n = s + 1 == a.sequences ? left : pick(0, left / 2 + 1 > left ? left : left / 2 + 1);
    tiles += (n + p.tokens - 1) / p.tokens;
    left -= n;
  }
  EXPECT(tiles <= p.tiles, "%ld tiles of %d", (long)tiles, p.tiles);
  EXPECT((int64_t)p.tiles * a.kv_heads <= 1 << 24, "%d tiles of %d heads", p.tiles, a.kv_heads);
  EXPECT(a.splits >= 1 && a.splits <= 16, "%d ranges", a.splits);
  if (a.splits > 1) {
    EXPECT((int64_t)p.tiles * a.kv_heads * a.splits <= 1024, "%d ranges of %d tiles", a.splits, p.tiles);
    const size_t rows = (size_t)a.tokens * a.heads * a.splits;
    const uint8_t *part = (const uint8_t *)a.part, *sums = (const uint8_t *)a.sums;
    EXPECT(part >= ws_base && part + rows * a.dim * 4 <= sums, "numerators");
    EXPECT(sums + rows * 16 <= ws_base + ws_bytes, "sums");
    // the ranges of a tile's keys, as the kernel derives them
    for (int i = 0; i < 16; ++i) {
      const int t0 = (int)pick(0, 40), t1 = t0 + (int)pick(-3, 300), n = std::max(t1 - t0, 0), per = (n + a.splits - 1) / a.splits;
      int at = t0;
      for (int sp = 0; sp < a.splits; ++sp) {
        const int from = t0 + sp * per, to = std::min(t1, from + per);
        if (from >= to) continue;
        EXPECT(from == at, "range %d from %d after %d", sp, from, at);
        at = to;
      }
      EXPECT(at == std::max(t0, t1), "ranges end at %d of %d", at, t1);
    }
  }
  if (p.tiles < 20000) {
    // every tile has its turn, over all launches of 65535 turns
    std::vector<int> seen(p.tiles, 0);
    for (int t = 0; t < p.tiles; ++t) ++seen[prompt_tile(p, t)];
    for (int t = 0; t < p.tiles; ++t) EXPECT(seen[t] == 1, "tile %d has %d turns", t, seen[t]);
  } else {
    EXPECT(p.half == p.tiles, "several rounds in two directions");
  }
  return hipSuccess;
}

hipError_t launch_attn_cache(const AttnCacheArgs &a, hipStream_t) {
  ++launches;
  const int R = a.heads / a.c.heads * a.q_len;
  EXPECT(a.row_tiles == (R + 15) / 16 && a.splits >= 1, "%d rows in %d tiles, %d ranges", R, a.row_tiles, a.splits);
  EXPECT((int64_t)a.row_tiles * a.splits <= 65535 && a.batch <= 65535, "grid %d x %d x %d", a.c.heads,
         a.row_tiles * a.splits, a.batch);
  EXPECT((int64_t)a.batch * a.c.heads * a.row_tiles * a.splits <= std::max<int64_t>(16 * 512, (int64_t)a.batch * a.c.heads * a.row_tiles),
         "%d ranges of many blocks", a.splits);
  if (a.splits > 1) {
    const size_t rows = (size_t)a.batch * a.heads * a.q_len * a.splits;
    const uint8_t *part = (const uint8_t *)a.part, *sums = (const uint8_t *)a.sums;
    EXPECT(part >= ws_base && part + rows * a.c.dim * 4 <= sums, "numerators");
    EXPECT(sums + rows * 8 <= ws_base + ws_bytes, "sums");
  }
  // the ranges of a tile's chunks, as the kernel derives them
  for (int i = 0; i < 16; ++i) {
    const int len = (int)pick(0, a.max_len), rt = (int)pick(0, a.row_tiles - 1), shared = a.heads / a.c.heads;
    const int first = len - a.q_len + 1;
    auto hi_of = [&](int token) { return std::max(first + token, 0); };
    auto lo_of = [&](int token) { return a.window > 0 ? std::max(0, first + token - a.window) : 0; };
    const int t_first = rt * 16 / shared, t_last = (std::min(rt * 16 + 16, R) - 1) / shared;
    const int lo = lo_of(t_first), hi = hi_of(t_last);
    const int c_first = lo / 32, chunks = std::max((hi + 31) / 32 - c_first, 0);
    const int per = a.splits > 1 ? (chunks + a.splits - 1) / a.splits : chunks;
    int at = c_first;
    for (int sp = 0; sp < a.splits; ++sp) {
      const int c0 = c_first + std::min(sp * per, chunks), c1 = c_first + std::min(sp * per + per, chunks);
      EXPECT(c0 == at && c1 >= c0, "range %d: %d .. %d after %d", sp, c0, c1, at);
      at = c1;
    }
    EXPECT(at == c_first + chunks, "ranges end at %d of %d", at, c_first + chunks);
    EXPECT(hi <= len && (hi == 0 || (hi - 1) >> a.c.page_shift < a.ld_table), "key %d, table of %ld", hi, (long)a.ld_table);
  }
  return hipSuccess;
}
}  // namespace svq

using namespace svq;

template <typename F>
static void run(const char *what, F f) {
  size_t need = 0;
  svq_status st = f(nullptr, &need);
  EXPECT(st == SVQ_OK && need > 0, "%s: query %d", what, (int)st);
  if (st != SVQ_OK || need > (size_t)1 << 33) return;
  uint8_t *const ws = (uint8_t *)0x100000;  // never touched: the stand-ins look at addresses only
  ws_base = ws;
  ws_bytes = need;
  size_t cap = need;
  const long before = launches;
  st = f(ws, &cap);
  EXPECT(st == SVQ_OK && launches == before + 1, "%s: call %d", what, (int)st);
  cap = need - 1;
  EXPECT(f(ws, &cap) == SVQ_ERR_BUFFER_TOO_SMALL, "%s: one byte short", what);
  cap = need;
  EXPECT(f(ws + 8, &cap) == SVQ_ERR_INVALID_ARG, "%s: misaligned", what);
  EXPECT(launches == before + 1, "%s: a refused call launched", what);
}

int main() {
  void *const P = (void *)0x200000;
  const int dims[] = {64, 128, 256}, groups[] = {32, 64, 128}, pages[] = {16, 32, 64, 128, 256};
  for (int dim : dims)
    for (int group : groups)
      for (int ps : pages) {
        if (group > dim) continue;
        svq_kv_cache c{P, 7, ps, 3, dim, group};
        size_t bytes = 0;
        EXPECT(svq_kv_bytes(&c, &bytes) == SVQ_OK, "bytes");
        KvView v;
        std::memset(&v, 0, sizeof(v));
        v.pages = 7;
        v.heads = 3;
        v.dim = dim;
        v.groups = dim / group;
        for (v.page_shift = 0; 1 << v.page_shift < ps; ++v.page_shift) {
        }
        for (v.group_shift = 0; 1 << v.group_shift < group; ++v.group_shift) {
        }
        v.off_v = ps * dim / 2;
        v.off_kp = 2 * v.off_v;
        v.off_vp = v.off_kp + ps * v.groups * 4;
        v.block = v.off_vp + ps * v.groups * 4;
        EXPECT(bytes == (size_t)v.block * 21, "%zu bytes, blocks of %d", bytes, v.block);
        check_layout(v);
        EXPECT(svq_kv_write(&c, P, 3 * dim, P, 3 * dim, 5, (const int32_t *)P, nullptr) == SVQ_OK, "write");
        EXPECT(svq_kv_read(&c, (const int32_t *)P, 5, P, 3 * dim, P, 3 * dim, SVQ_F32, nullptr) == SVQ_OK, "read");
      }
  const int kvs[] = {1, 2, 3, 8, 16, 71}, shareds[] = {1, 2, 4, 5, 7, 8, 16, 17, 64};
  for (int kv : kvs)
    for (int sh : shareds)
      for (int i = 0; i < 12; ++i) {
        const int dim = dims[rng() % 3], heads = kv * sh;
        const int64_t ld = (int64_t)heads * dim, ldk = (int64_t)kv * dim;
        const int64_t most = std::min<int64_t>((1 << 29) / heads, 1 << 24);
        const int64_t tokens = pick(1, i < 6 ? std::min<int64_t>(5000, most) : most), seqs = pick(1, i % 2 ? 300 : 3);
        const int span = i % 3 ? 0 : (int)pick(1, 3000);
        run("prompt", [&](void *ws, size_t *n) {
          return svq_attn_prompt(P, ld, P, ldk, P, ldk, heads, kv, dim, (const int32_t *)P, nullptr, seqs, tokens, tokens, 1,
                                 span, 0.1f, P, ld, ws, n, nullptr);
        });
        const int ps = pages[rng() % 5], group = std::min(groups[rng() % 3], dim);
        svq_kv_cache c{P, 1000, ps, kv, dim, group};
        const int64_t batch = pick(1, i % 3 ? 100 : 3), q_len = pick(1, i % 4 ? 8 : 300);
        const int64_t len = pick(1, i < 6 ? 3000 : 1 << 20), table = (len + ps - 1) / ps + pick(0, 3);
        const int window = i % 2 ? (int)pick(1, 2000) : 0;
        run("cache", [&](void *ws, size_t *n) {
          return svq_attn_cache(&c, P, ld, heads, (const int32_t *)P, table, (const int32_t *)P, batch, (int)q_len, len, window,
                                0.1f, P, ld, ws, n, nullptr);
        });
      }
  std::printf("%ld launches, %ld checks, %d failures\n", launches, checks, fails);
  return fails != 0;
}
