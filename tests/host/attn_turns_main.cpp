// The turns of a prompt's tiles over all launches of a call, on the CPU: every
// tile has one, in whatever number of launches; and the scores up to which a row
// keeps its maximum, for scales and maxima of every size.  Built with AddressSanitizer and
// UndefinedBehaviorSanitizer by tests/test_attn_turns_host.py.
#include <cmath>
#include <cstdio>
#include <cstring>
#include <random>
#include <vector>

#include "../../bit_spherical_vector_amd/csrc/svq_attn.h"

using namespace svq;

static int fails = 0;
static long plans = 0, several = 0, both_ways = 0;

static void check(int tokens, int sequences, int heads, int kv_heads, int units) {
  const PromptPlan plan = prompt_plan(tokens, sequences, heads, kv_heads, PROMPT_WAVES, units);
  std::vector<int> seen(plan.tiles, 0);
  int launches = 0;
  prompt_launches(plan, [&](const PromptPlan &p, int n) {
    ++launches;
    if (n < 1 || n > 65535) ++fails;
    for (int block = 0; block < n; ++block) {
      const int tile = prompt_tile(p, block);
      if (tile < 0 || tile >= plan.tiles) {
        ++fails;
        continue;
      }
      ++seen[tile];
    }
  });
  int without = 0, twice = 0;
  for (int n : seen) {
    without += n == 0;
    twice += n > 1;
  }
  if (without || twice) {
    std::fprintf(stderr, "%d tokens, %d sequences, %d heads over %d, %d units: of %d tiles %d without a turn, %d with several\n",
                 tokens, sequences, heads, kv_heads, units, plan.tiles, without, twice);
    ++fails;
  }
  ++plans;
  several += launches > 1;
  both_ways += launches > 1 && plan.half < plan.tiles;
}

int main() {
  std::mt19937 rng(3);
  auto pick = [&](int lo, int hi) { return lo + (int)(rng() % (unsigned)(hi - lo + 1)); };
  check(65535, 65535, 1, 1, 256);
  check(65536, 65535, 1, 1, 256);
  check(65000, 65279, 1, 1, 256);
  check(1 << 24, 65535, 16, 1, 256);
  check(1 << 23, 1, 64, 1, 256);
  const int kvs[] = {1, 2, 3, 8, 16, 32}, shareds[] = {1, 2, 3, 5, 8, 64}, units[] = {256, 304, 64, 1};
  for (int kv : kvs)
    for (int sh : shareds)
      for (int u : units)
        for (int i = 0; i < 8; ++i) {
          const int sequences = i % 2 ? pick(1, 65535) : pick(65000, 65535);
          const int tokens = i < 4 ? pick(1, 70000) : pick(1, 1 << 20);
          check(tokens, sequences, kv * sh, kv, u);
        }
  // raised_by: not below the maximum, not more than asked for above it, and not
  // the maximum itself where fp32 has scores between
  for (int i = 0; i < 200000; ++i) {
    auto any = [&](int lo, int hi) { return std::ldexp(1.f + (float)(rng() & 0x7FFFFF) * 0x1p-23f, pick(lo, hi)); };
    const float scale = i % 97 == 0 ? 0.f : any(-149, 127), sc = exponent_scale(i % 2 ? scale : -scale);
    if (!(sc > 0.f) || !std::isfinite(sc)) ++fails;
    const float m = i % 11 == 0 ? 0.f : (i % 2 ? 1.f : -1.f) * any(-149, 126), by = i % 3 ? 8.f : 6.f;
    const float to = raised_by(m, by, sc);
    const float room = (std::nextafterf(m, INFINITY) - m) * sc;
    if (!(to >= m) || !((to - m) * sc <= by) || (room < 0.25f && std::isfinite(m + by / sc) && !((to - m) * sc > by - 0.75f) && sc > 1e-37f && sc < 1e37f)) {
      std::fprintf(stderr, "raised_by(%g, %g, %g) = %g\n", m, by, sc, to);
      ++fails;
    }
  }
  if (raised_by(-3.40282347e38f, 8.f, 0.1f) != -3.40282347e38f) ++fails;  // no maximum yet
  std::printf("%ld plans, %ld of several launches, %ld of them in two directions, %d failures\n", plans, several, both_ways, fails);
  return fails != 0 || several == 0 || both_ways == 0;
}
