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
// Nibble order.  Nibbles 2i and 2i+1 of a byte come out of one shift as two
// fp16 subnormals (c * 2^-24 and c * 16 * 2^-24), in pairs 4 nibbles apart.
// Key words hold channel j of their eight at nibble KV_NIBBLE(j), so that the
// pairs are consecutive channels; value runs hold tile t at nibble t.
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

struct AttnPromptArgs {
  const uint16_t *q, *k, *v;
  uint16_t *y;
  int64_t ldq, ldk, ldv, ldy;
  const int32_t *starts, *starts_k;  // starts_k null: as starts
  int32_t sequences, tokens, tokens_k;
  int32_t heads, kv_heads, dim;
  int32_t causal, window;
  float scale;
};
hipError_t launch_attn_prompt(const AttnPromptArgs &a, hipStream_t s);

struct AttnCacheArgs {
  KvView c;
  const uint16_t *q;
  uint16_t *y;
  int64_t ldq, ldy, ld_table;
  const int32_t *table, *lens;
  int32_t batch, q_len, heads, max_len, window;
  float scale;
  int32_t row_tiles, splits, per;  // tiles of 16 rows; ranges of keys, each of `per` chunks of 32
  float *part, *sums;         // splits > 1: [batch][kv head][row][split] numerators [dim] and (reference, sum)
};
// rows of a tile, keys of a block's step, steps of a block at most
constexpr int CACHE_ROWS = 16, CACHE_BLOCK_KEYS = 128, CACHE_MAX_STEPS = 16;
hipError_t launch_attn_cache(const AttnCacheArgs &a, hipStream_t s);

}  // namespace svq
