/*
 * libsvq, attention: what stands between the q/k/v products of a decoder
 * layer and its output projection.  A whole prompt's attention, a paged cache
 * of keys and values held in 4 bits, and the attention of new tokens over
 * that cache.  Same library, same rules as svq.h (ownership, errors, streams,
 * workspaces: a call with workspace == NULL only reports the bytes needed and
 * validates what it is given; a workspace starts on 16 bytes; calls that share
 * a workspace must be ordered on one stream; nothing is kept from one call for
 * the next).
 *
 * Rows.  Queries, keys, values and outputs are rows of heads side by side, as
 * svq_linear writes them: row t holds head h at columns [h*head_dim,
 * (h+1)*head_dim), rows lie ld elements apart and start on 16 bytes (a base
 * or an ld that does not is refused with SVQ_ERR_UNSUPPORTED), so q, k and v
 * may be columns of one wider buffer.  Query head h attends over key head
 * h / (q_heads / kv_heads).  q_heads (at most 16384) is a multiple of kv_heads
 * (at most 1024), at most 64 query heads share a key head, and head_dim is 64,
 * 128 or 256.
 *
 * Numerics.  Inputs and outputs of the attention calls are bf16.  Scores are
 * products of the bf16 inputs (of the stored values, for the cache) summed in
 * fp32; the softmax's maximum, exponentials and sum are fp32; each output is
 * rounded once, to nearest even.
 *   Over a prompt a weight (at most 2^0.5, a row's greatest at least 2^-9) meets
 * its value rounded to bf16, and the products' sums are fp32: values from 2^127
 * over the number of keys on may give infinities, results below 2^-122 lose bits.
 *   Over the cache, where codes are multiplied as they are, a query's channel
 * meets the codes with all its bits down to 2^-28 of the greatest magnitude in
 * its group of channels, and within 2^-35 of that magnitude below; the product of
 * a weight and a scale is held in 22 bits, down to 2^-32 of the greatest scale or
 * minimum that the row sees; and of 32 products of codes that are added at once
 * each is kept within 2^-22 of the greatest that any code (15) would give.
 *   Weights below 2^-117 of a row's greatest are zero.  A query that sees no key,
 * or only keys whose scores are minus infinity, gives a row of zeros.  A key that
 * a query does not see has no influence on it, whatever it, its value or its
 * stored scales hold (infinities and NaN included): not a bit of its row changes.
 */
#ifndef SVQ_ATTN_H
#define SVQ_ATTN_H

#include "svq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* svq_attn_prompt: attention of whole sequences, packed one behind another.
 *   Sequence i has the queries starts[i] .. starts[i+1]-1 and, with starts_k,
 *   the keys starts_k[i] .. starts_k[i+1]-1 (a prefix in front of the new
 *   tokens); starts_k NULL: keys as queries.  Its query t of n sits at
 *   position p = keys - n + t and sees the keys j of its sequence with
 *     causal 0:            all;
 *     causal 1:            j <= p;
 *     causal 1, window w:  p - w < j <= p      (window 0: no window).
 *   y = sum_j softmax_j(scale * q . k_j) v_j.
 *   q:        device bf16 [tokens][ldq]; y: device bf16 [tokens][ldy], out; it
 *             must not overlap q, k or v.
 *   k, v:     device bf16 [tokens_k][ldk], [tokens_k][ldv].
 *   starts, starts_k: device int32 [sequences + 1], not decreasing, within
 *             [0, tokens] and [0, tokens_k] (values beyond are taken as the
 *             nearest that is not).  Rows of y before starts[0] and from
 *             starts[sequences] on are left as they were.
 *   tokens, tokens_k: 1 .. 2^24; sequences: 1 .. 65535; scale: finite.
 * SVQ_ERR_UNSUPPORTED: ldk or ldv beyond 2^24, tokens * q_heads beyond 2^29,
 * sequences * kv_heads beyond 2^21. */
svq_status svq_attn_prompt(const void *q, int64_t ldq, const void *k, int64_t ldk, const void *v, int64_t ldv,
                           int32_t q_heads, int32_t kv_heads, int32_t head_dim, const int32_t *starts,
                           const int32_t *starts_k, int64_t sequences, int64_t tokens, int64_t tokens_k,
                           int32_t causal, int32_t window, float scale, void *y, int64_t ldy, void *workspace,
                           size_t *workspace_bytes, void *stream);

/* A paged cache: pages of page_size token slots, caller-owned device memory
 * of svq_kv_bytes bytes.  Slot s is place s % page_size of page s / page_size
 * and holds one token's keys and values of every head.
 *
 * A group of `group` consecutive channels of a slot, head and side (key or
 * value) is held as 4-bit codes c, a scale s and a minimum m, both bf16, and
 * stands for the values m + c * s:
 *   m = the group's least value;
 *   s = (greatest - least) / 15, rounded to fp32 and then to bf16;
 *   c = (x - m) / s rounded to the nearest whole number (ties to even),
 *       at most 15; 0 where s is 0.
 * A group that holds an infinity or NaN stands for NaN throughout. */
typedef struct {
  void *dev;         /* device memory, on 16 bytes                       */
  int64_t pages;     /* 1 .. (2^31 - 1) / page_size                      */
  int32_t page_size; /* 16, 32, 64, 128 or 256                           */
  int32_t kv_heads;  /* 1 .. 1024                                        */
  int32_t head_dim;  /* 64, 128 or 256                                   */
  int32_t group;     /* 32, 64 or 128, at most head_dim                  */
} svq_kv_cache;

/* svq_kv_bytes: the size of a cache (cache->dev is not read). */
svq_status svq_kv_bytes(const svq_kv_cache *cache, size_t *bytes);

/* svq_kv_write: quantises the keys and values of `tokens` tokens into the
 * slots named; a slot outside [0, pages * page_size) is skipped.  The slots
 * of a call are distinct (of several tokens for one slot, each head's keys and
 * values are those of one of them or a mixture).
 *   k, v:   device bf16 [tokens][ldk], [tokens][ldv], kv_heads heads a row.
 *   slots:  device int32 [tokens].  tokens: 1 .. 2^24. */
svq_status svq_kv_write(const svq_kv_cache *cache, const void *k, int64_t ldk, const void *v, int64_t ldv,
                        int64_t tokens, const int32_t *slots, void *stream);

/* svq_kv_read: the values that the slots stand for, m + c * s in fp32,
 * rounded to bf16 or as they are; a slot outside [0, pages * page_size) gives
 * zeros.
 *   k, v:   device, out, [tokens][ldk], [tokens][ldv] of type dt; apart from
 *           each other and from the cache. */
svq_status svq_kv_read(const svq_kv_cache *cache, const int32_t *slots, int64_t tokens, void *k, int64_t ldk,
                       void *v, int64_t ldv, svq_dtype dt, void *stream);

/* svq_attn_cache: attention of the newest q_len tokens of each sequence over
 * its cached keys and values, which hold these tokens too.
 *   Token j of sequence b is place j % page_size of page
 *   table[b * ld_table + j / page_size]; a page outside [0, pages) holds
 *   nothing that is seen.  Query t of q_len of a sequence of lens[b] tokens
 *   sits at p = lens[b] - q_len + t and sees the tokens j <= p, with window
 *   w > 0 those of them with j > p - w.
 *   q:        device bf16 [batch * q_len][ldq], row b * q_len + t.
 *   table:    device int32 [batch][ld_table].
 *   lens:     device int32 [batch], within [0, max_len] (values beyond are
 *             taken as the nearest that is not).
 *   max_len:  1 .. ld_table * page_size, at most 2^30: what the launch is
 *             planned for.
 *   batch:    1 .. 65535; q_len: 1 .. 1024; scale: finite.
 *   y:        device bf16 [batch * q_len][ldy], out; must not overlap q or the
 *             cache. */
svq_status svq_attn_cache(const svq_kv_cache *cache, const void *q, int64_t ldq, int32_t q_heads,
                          const int32_t *table, int64_t ld_table, const int32_t *lens, int64_t batch,
                          int32_t q_len, int64_t max_len, int32_t window, float scale, void *y, int64_t ldy,
                          void *workspace, size_t *workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SVQ_ATTN_H */
