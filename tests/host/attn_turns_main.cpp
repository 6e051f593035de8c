// The turns of a prompt's tiles over all launches of a call, on the CPU: every
// tile has one, in whatever number of launches.  Built with AddressSanitizer and
// UndefinedBehaviorSanitizer by tests/test_attn_turns_host.py.
#include <cstdio>
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
  std::printf("%ld plans, %ld of several launches, %ld of them in two directions, %d failures\n", plans, several, both_ways, fails);
  return fails != 0 || several == 0 || both_ways == 0;
}
