// Launch interfaces of the attention calls (include/svq_attn.h) and the
// layout of the 4-bit cache.
#pragma once
#include "svq_internal.h"

#include "../../include/svq_attn.h"

namespace svq {

int compute_units();  // of the current device

// The cache is [pages][kv_heads] blocks; a block holds its page's key codes,
// value codes, key parameters and value parameters of one head.  A parameter
// is one dword: scale (bf16) in the low half, minimum (bf16) in the high one.
//
// Both code layouts give a lane of v_mfma_f32_16x16x32_f16 its operand with
// wide loads and no exchange between lanes:
//   keys    [slot/16][h][slot%16][word c]: word c of D/32 holds channels
//           32c + 8h .. 32c + 8h + 7, so lane 16h + r reads slot r's words of
//           all steps c of 32 channels in one piece, and a wave one stretch;
//   values  [slot/4][r][slot%4]: 16 runs a slot, run r = channels r, 16 + r,
//           32 + r ... (D/16 of them, D/32 bytes): lane 16h + r reads channel
//           16t + r of four slots for every 16-channel tile t in one piece,
//           and a token's bytes are its own;
//   parameters [slot/4][group][slot%4]: a lane reads four slots of a group at
//           once.
// Nibble order.  Nibbles come out as fp16 subnormals in pairs 4 nibbles apart,
// each pair by a mask and (but for nibbles 1 and 5) a shift.  Key words hold
// channel j of their eight at nibble kv_nibble(j), so that the pairs are
// consecutive channels; value runs hold tile t at nibble t.
struct KvView {
  uint8_t *base;
  int64_t pages;
  int32_t page_shift, heads, dim, groups, group_shift;  // page_size = 1 << page_shift
  int32_t off_v, off_kp, off_vp, block;                 // bytes within a block, its size
};

__host__ __device__ inline int kv_nibble(int j) { return (j >> 1) | ((j & 1) << 2); }

// Bytes of a view's block at which a slot's data lie.
// (key word: channels 8n .. 8n + 7)
__host__ __device__ inline int kv_key_word(const KvView &c, int place, int n) {
  return (((place >> 4) * 64 + (n & 3) * 16 + (place & 15)) * (c.dim / 32) + (n >> 2)) * 4;
}
__host__ __device__ inline int kv_value_run(const KvView &c, int place, int r) {
  return c.off_v + ((place >> 2) * 64 + r * 4 + (place & 3)) * (c.dim / 32);
}
__host__ __device__ inline int kv_param(const KvView &c, int side, int place, int g) {
  return (side ? c.off_vp : c.off_kp) + (((place >> 2) * c.groups + g) * 4 + (place & 3)) * 4;
}
__host__ __device__ inline uint8_t *kv_block(const KvView &c, int64_t page, int head) {
  return c.base + (page * c.heads + head) * (int64_t)c.block;
}

struct KvWriteArgs {
  KvView c;
  const uint16_t *k, *v;
  int64_t ldk, ldv, tokens;
  const int32_t *slots;
};
struct KvReadArgs {
  KvView c;
  const int32_t *slots;
  void *k, *v;
  int64_t ldk, ldv, tokens;
  int32_t f32;
};
hipError_t launch_kv_write(const KvWriteArgs &a, hipStream_t s);
hipError_t launch_kv_read(const KvReadArgs &a, hipStream_t s);

// Exponents are base 2.  A scale of zero stays a number that keeps hidden scores
// at -infinity and takes any score to nothing, the largest one that keeps equal
// scores equal.
__host__ __device__ inline float exponent_scale(float scale) {
  return fminf(fmaxf(fabsf(scale) * 1.44269504088896f, 0x1p-149f), 3.40282347e38f);
}

// The score that lies `by` exponents (less a quarter, for the roundings) above a
// maximum m, or m itself where fp32 has none so near; a row without a maximum
// takes any score.
__host__ __device__ inline float raised_by(float m, float by, float sc) {
  const float to = m + (by - 0.25f) / sc;
  return m > -3.40282347e38f && (to - m) * sc <= by ? to : m;
}

struct AttnPromptArgs {
  const uint16_t *q, *k, *v;
  uint16_t *y;
  int64_t ldq, ldk, ldv, ldy;
  const int32_t *starts, *starts_k;  // starts_k null: as starts
  int32_t sequences, tokens, tokens_k;
  int32_t heads, kv_heads, dim;
  int32_t causal, window;
  float scale;
  int32_t splits;      // ranges of keys
  float *part, *sums;  // splits > 1, [token][head][split] numerators [dim] and (maximum, how far it lies above the reference, sum, no keys: -1)
};

constexpr int PROMPT_WAVES = 4;  // of a block
hipError_t launch_attn_prompt(const AttnPromptArgs &a, hipStream_t s);

// Divisions by launch constants d, with multipliers 2^32 / d + 1 and
// 2^16 / d + 1: exact where n * d < 2^32 and 2^16.
__host__ __device__ inline int quotient(int n, uint32_t mul) { return (int)((uint64_t)(uint32_t)n * mul >> 32); }
__host__ __device__ inline int quotient16(int n, uint32_t mul) { return (int)((uint32_t)n * mul >> 16); }

// A block's tile of rows: `tokens` tokens of a sequence, each with the G query
// heads that share a key head, in 32 rows a wave.
struct PromptPlan {
  int32_t tiles, half;         // see prompt_tile
  int32_t first;               // turn of a launch's first block
  int32_t tokens, G;           // tokens = 32 * waves / G
  uint32_t tokens_mul, g_mul;  // for quotient, quotient16
};
inline PromptPlan prompt_plan(int tokens, int sequences, int heads, int kv_heads, int waves, int units) {
  PromptPlan p;
  p.G = heads / kv_heads;
  p.tokens = 32 * waves / p.G;
  p.tokens_mul = (uint32_t)((1ull << 32) / (uint32_t)p.tokens) + 1;
  p.g_mul = 65536u / (uint32_t)p.G + 1;
  // a sequence adds a tile at most to what its tokens fill; most of these are
  // not there when the tiles are counted into rounds
  p.tiles = tokens / p.tokens + sequences;
  const int round = units / kv_heads;
  p.half = round > 0 && p.tiles > round && p.tiles - sequences <= 2 * round ? round : p.tiles;
  p.first = 0;
  return p;
}
// The tile of a launch's block, by its turn.  The last tiles come first: under a causal
// mask they have the most keys.  Where one round of blocks, two a compute unit,
// covers all, the second on each unit takes the tiles from the front on, which
// leaves every unit about as many keys (2048 tokens 51 -> 47 us).
__host__ __device__ inline int prompt_tile(const PromptPlan &p, int block) {
  const int turn = p.first + block;
  return turn < p.half ? p.tiles - 1 - turn : turn - p.half;
}
// Calls launch(plan, blocks) for all turns, at most 65535 at a time (the end of
// the grid's second dimension).
template <typename F>
inline void prompt_launches(PromptPlan p, F launch) {
  while (p.first < p.tiles) {
    const int n = p.tiles - p.first < 65535 ? p.tiles - p.first : 65535;
    launch(p, n);
    p.first += n;
  }
}

// Ranges of keys a tile.  Few tiles (one key head of a long prompt, say) leave
// units idle while each goes through all its keys.  A range more takes time off
// the longest tile's `keys` / 64 steps (~1.3 us each at 128 channels) and adds
// the writing and reading of every row's sums (~0.35 ns a row): the least is
// near n = sqrt(keys / 64 * 4000 / rows).  No ranges under 1024 keys, where the
// second launch takes what they give (512 keys, 4 heads: 13.8 us in two ranges,
// 13.0 without).
inline int prompt_splits(const PromptPlan &p, int64_t rows, int sequences, int tokens_k, int kv_heads, int dim, int window, int units) {
  const int64_t blocks = (int64_t)p.tiles * kv_heads, round = dim == 256 ? units : 2 * units;
  int64_t keys = tokens_k / sequences;
  if (window > 0 && (int64_t)window + p.tokens < keys) keys = (int64_t)window + p.tokens;
  if (keys < 1024) return 1;
  int64_t most = 2 * round / blocks;  // no more than two rounds of blocks
  if (most > 16) most = 16;
  if (most > keys / 256) most = keys / 256;
  int n = 1;
  while (n < most && (n + 1) * (n + 1) * rows <= keys / 64 * 4000) ++n;
  return n;
}

struct AttnCacheArgs {
  KvView c;
  const uint16_t *q;
  uint16_t *y;
  int64_t ldq, ldy, ld_table;
  const int32_t *table, *lens;
  int32_t batch, q_len, heads, max_len, window;
  float scale;
  int32_t row_tiles, splits;  // tiles of 16 rows, ranges of keys
  float *part, *sums;         // splits > 1: [batch][kv head][row][split] results [dim] and (maximum, sum of weights)
};
// rows of a tile, keys of a block's step, steps of a block at most
constexpr int CACHE_ROWS = 16, CACHE_BLOCK_KEYS = 128, CACHE_MAX_STEPS = 16;
hipError_t launch_attn_cache(const AttnCacheArgs &a, hipStream_t s);

}  // namespace svq
