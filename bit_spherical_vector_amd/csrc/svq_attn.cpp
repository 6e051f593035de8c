// Host side of the attention calls (include/svq_attn.h): argument checks,
// workspace layout and dispatch.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstring>

#include "svq_attn.h"

using namespace svq;

namespace {

constexpr int64_t MAX_TOKENS = 1 << 24, MAX_LD = 1 << 24, MAX_SEQUENCES = 65535;
constexpr int MAX_HEADS = 1024, MAX_Q_HEADS = 16384, MAX_SHARED = 64, MAX_Q_LEN = 1024;

bool bad_workspace(const void *ws) { return ((uintptr_t)ws & 15) != 0; }
bool on_16(const void *p, int64_t ld, size_t esz) { return (((uintptr_t)p) | ((uintptr_t)ld * esz)) % 16 == 0; }

svq_status check_heads(int32_t q_heads, int32_t kv_heads, int32_t dim) {
  if (q_heads < 1 || kv_heads < 1 || q_heads % kv_heads != 0) return SVQ_ERR_INVALID_ARG;
  if (dim != 64 && dim != 128 && dim != 256) return SVQ_ERR_UNSUPPORTED;
  if (kv_heads > MAX_HEADS || q_heads > MAX_Q_HEADS || q_heads / kv_heads > MAX_SHARED) return SVQ_ERR_UNSUPPORTED;
  return SVQ_OK;
}

int log2_of(int v) {
  int s = 0;
  while ((1 << s) < v) ++s;
  return s;
}

svq_status check_cache(const svq_kv_cache *c, KvView *out) {
  if (!c) return SVQ_ERR_INVALID_ARG;
  const int ps = c->page_size;
  if (ps != 16 && ps != 32 && ps != 64 && ps != 128 && ps != 256) return SVQ_ERR_UNSUPPORTED;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return SVQ_ERR_UNSUPPORTED;
  if ((c->group != 32 && c->group != 64 && c->group != 128) || c->group > c->head_dim) return SVQ_ERR_UNSUPPORTED;
  if (c->kv_heads < 1 || c->pages < 1) return SVQ_ERR_INVALID_ARG;
  if (c->kv_heads > MAX_HEADS || c->pages > INT32_MAX / ps) return SVQ_ERR_UNSUPPORTED;
  KvView v;
  v.base = (uint8_t *)c->dev;
  v.pages = c->pages;
  v.page_shift = log2_of(ps);
  v.heads = c->kv_heads;
  v.dim = c->head_dim;
  v.groups = c->head_dim / c->group;
  v.group_shift = log2_of(c->group);
  v.off_v = ps * v.dim / 2;
  v.off_kp = 2 * v.off_v;
  v.off_vp = v.off_kp + ps * v.groups * 4;
  v.block = v.off_vp + ps * v.groups * 4;
  *out = v;
  return SVQ_OK;
}

svq_status check_cache_dev(const svq_kv_cache *c, KvView *out) {
  const svq_status st = check_cache(c, out);
  if (st != SVQ_OK) return st;
  if (!c->dev || ((uintptr_t)c->dev & 15)) return SVQ_ERR_INVALID_ARG;
  return SVQ_OK;
}

svq_status of(hipError_t e) { return e == hipSuccess ? SVQ_OK : SVQ_ERR_HIP; }

}  // namespace

extern "C" {

svq_status svq_kv_bytes(const svq_kv_cache *cache, size_t *bytes) {
  if (!bytes) return SVQ_ERR_INVALID_ARG;
  KvView c;
  const svq_status st = check_cache(cache, &c);
  if (st != SVQ_OK) return st;
  *bytes = (size_t)c.pages * c.heads * c.block;
  return SVQ_OK;
}

svq_status svq_kv_write(const svq_kv_cache *cache, const void *k, int64_t ldk, const void *v, int64_t ldv,
                        int64_t tokens, const int32_t *slots, void *stream) {
  KvWriteArgs a;
  const svq_status st = check_cache_dev(cache, &a.c);
  if (st != SVQ_OK) return st;
  const int64_t cols = (int64_t)a.c.heads * a.c.dim;
  if (!k || !v || !slots || tokens < 1 || tokens > MAX_TOKENS || ldk < cols || ldv < cols) return SVQ_ERR_INVALID_ARG;
  if (!on_16(k, ldk, 2) || !on_16(v, ldv, 2)) return SVQ_ERR_UNSUPPORTED;
  a.k = (const uint16_t *)k;
  a.v = (const uint16_t *)v;
  a.ldk = ldk;
  a.ldv = ldv;
  a.tokens = tokens;
  a.slots = slots;
  return of(launch_kv_write(a, (hipStream_t)stream));
}

svq_status svq_kv_read(const svq_kv_cache *cache, const int32_t *slots, int64_t tokens, void *k, int64_t ldk,
                       void *v, int64_t ldv, svq_dtype dt, void *stream) {
  KvReadArgs a;
  const svq_status st = check_cache_dev(cache, &a.c);
  if (st != SVQ_OK) return st;
  const int64_t cols = (int64_t)a.c.heads * a.c.dim;
  if (dt != SVQ_BF16 && dt != SVQ_F32) return SVQ_ERR_INVALID_ARG;
  if (!k || !v || !slots || tokens < 1 || tokens > MAX_TOKENS || ldk < cols || ldv < cols) return SVQ_ERR_INVALID_ARG;
  const size_t esz = dt == SVQ_F32 ? 4 : 2;
  if (!on_16(k, ldk, esz) || !on_16(v, ldv, esz)) return SVQ_ERR_UNSUPPORTED;
  a.slots = slots;
  a.k = k;
  a.v = v;
  a.ldk = ldk;
  a.ldv = ldv;
  a.tokens = tokens;
  a.f32 = dt == SVQ_F32;
  return of(launch_kv_read(a, (hipStream_t)stream));
}

svq_status svq_attn_prompt(const void *q, int64_t ldq, const void *k, int64_t ldk, const void *v, int64_t ldv,
                           int32_t q_heads, int32_t kv_heads, int32_t head_dim, const int32_t *starts,
                           const int32_t *starts_k, int64_t sequences, int64_t tokens, int64_t tokens_k,
                           int32_t causal, int32_t window, float scale, void *y, int64_t ldy, void *workspace,
                           size_t *workspace_bytes, void *stream) {
  if (!workspace_bytes || bad_workspace(workspace)) return SVQ_ERR_INVALID_ARG;
  const svq_status st = check_heads(q_heads, kv_heads, head_dim);
  if (st != SVQ_OK) return st;
  const int64_t cols = (int64_t)q_heads * head_dim, cols_k = (int64_t)kv_heads * head_dim;
  if (tokens < 1 || tokens > MAX_TOKENS || tokens_k < 1 || tokens_k > MAX_TOKENS) return SVQ_ERR_INVALID_ARG;
  if (sequences < 1 || sequences > MAX_SEQUENCES) return SVQ_ERR_INVALID_ARG;
  if (ldq < cols || ldy < cols || ldk < cols_k || ldv < cols_k) return SVQ_ERR_INVALID_ARG;
  if ((causal != 0 && causal != 1) || window < 0 || (window > 0 && !causal)) return SVQ_ERR_INVALID_ARG;
  if (!std::isfinite(scale)) return SVQ_ERR_INVALID_ARG;
  if (!on_16(q, ldq, 2) || !on_16(k, ldk, 2) || !on_16(v, ldv, 2) || !on_16(y, ldy, 2)) return SVQ_ERR_UNSUPPORTED;
  if (ldk > MAX_LD || ldv > MAX_LD) return SVQ_ERR_UNSUPPORTED;  // bytes within a tile of 64 keys are 32-bit
  // a grid of at most 2^23 blocks
  if (tokens * q_heads > (int64_t)1 << 29 || sequences * kv_heads > 1 << 21) return SVQ_ERR_UNSUPPORTED;
  window = window < tokens_k ? window : 0;  // none hides a key; positions less the window stay 32-bit numbers
  const PromptPlan plan = prompt_plan((int)tokens, (int)sequences, q_heads, kv_heads, PROMPT_WAVES, compute_units());
  const int splits = prompt_splits(plan, tokens * q_heads, (int)sequences, (int)tokens_k, kv_heads, head_dim, window, compute_units());
  const size_t rows = (size_t)tokens * q_heads * splits;  // of partial sums
  const size_t part = splits > 1 ? align256(rows * head_dim * 4) : 0;
  const size_t need = splits > 1 ? part + align256(rows * 16) : 256;
  if (!workspace) {
    *workspace_bytes = need;
    return SVQ_OK;
  }
  if (!q || !k || !v || !y || !starts) return SVQ_ERR_INVALID_ARG;
  if (*workspace_bytes < need) return SVQ_ERR_BUFFER_TOO_SMALL;
  AttnPromptArgs a;
  std::memset(&a, 0, sizeof(a));
  a.q = (const uint16_t *)q;
  a.k = (const uint16_t *)k;
  a.v = (const uint16_t *)v;
  a.y = (uint16_t *)y;
  a.ldq = ldq;
  a.ldk = ldk;
  a.ldv = ldv;
  a.ldy = ldy;
  a.starts = starts;
  a.starts_k = starts_k ? starts_k : starts;
  a.sequences = (int32_t)sequences;
  a.tokens = (int32_t)tokens;
  a.tokens_k = (int32_t)tokens_k;
  a.heads = q_heads;
  a.kv_heads = kv_heads;
  a.dim = head_dim;
  a.causal = causal;
  a.window = window;
  a.scale = scale;
  a.splits = splits;
  if (splits > 1) {
    a.part = (float *)workspace;
    a.sums = (float *)((uint8_t *)workspace + part);
  }
  return of(launch_attn_prompt(a, (hipStream_t)stream));
}

svq_status svq_attn_cache(const svq_kv_cache *cache, const void *q, int64_t ldq, int32_t q_heads,
                          const int32_t *table, int64_t ld_table, const int32_t *lens, int64_t batch,
                          int32_t q_len, int64_t max_len, int32_t window, float scale, void *y, int64_t ldy,
                          void *workspace, size_t *workspace_bytes, void *stream) {
  if (!workspace_bytes || bad_workspace(workspace)) return SVQ_ERR_INVALID_ARG;
  AttnCacheArgs a;
  std::memset(&a, 0, sizeof(a));
  svq_status st = check_cache_dev(cache, &a.c);
  if (st == SVQ_OK) st = check_heads(q_heads, a.c.heads, a.c.dim);
  if (st != SVQ_OK) return st;
  const int64_t cols = (int64_t)q_heads * a.c.dim;
  if (batch < 1 || batch > MAX_SEQUENCES || q_len < 1 || q_len > MAX_Q_LEN || batch * q_len > MAX_TOKENS)
    return SVQ_ERR_INVALID_ARG;
  if (ld_table < 1 || max_len < 1 || max_len > (1 << 30) || (max_len + cache->page_size - 1) / cache->page_size > ld_table)
    return SVQ_ERR_INVALID_ARG;
  if (ldq < cols || ldy < cols || window < 0 || !std::isfinite(scale)) return SVQ_ERR_INVALID_ARG;
  if (!on_16(q, ldq, 2) || !on_16(y, ldy, 2)) return SVQ_ERR_UNSUPPORTED;
  if (window >= max_len) window = 0;  // hides no key; positions less the window stay 32-bit numbers
  const int R = q_heads / a.c.heads * q_len;
  a.row_tiles = (R + CACHE_ROWS - 1) / CACHE_ROWS;
  // Ranges of keys: for one round of blocks, two a compute unit (one sequence of
  // 32768 tokens 18.6 us for one, 16.7 for two, 19.6 for three).  Sequences of
  // different lengths share the units evenly if no block is long: at most
  // CACHE_MAX_STEPS steps a block (64 sequences of up to 8192 tokens: 101 us for
  // 8 steps, 77 for 16, 75 for 32), in at most sixteen rounds, which bounds the
  // workspace (many rows need no ranges).
  const int64_t blocks = batch * a.c.heads * a.row_tiles;
  const int64_t spread = (int64_t)window + q_len + 31;  // a window and the chunk that it starts in
  const int64_t keys = window > 0 && spread < max_len ? spread : max_len;
  const int64_t steps = (keys + CACHE_BLOCK_KEYS - 1) / CACHE_BLOCK_KEYS;
  const int64_t slots = 2 * compute_units();
  int64_t splits = blocks < slots ? slots / blocks : 1;
  if (batch > 1) {
    const int64_t even = (steps + CACHE_MAX_STEPS - 1) / CACHE_MAX_STEPS, most = 16 * slots / blocks;
    const int64_t want = even < most ? even : most;
    splits = want > splits ? want : splits;
  }
  a.splits = (int32_t)(splits < steps ? splits : steps);
  const size_t part = a.splits > 1 ? align256((size_t)batch * q_heads * q_len * a.splits * a.c.dim * 4) : 0;
  const size_t need = a.splits > 1 ? part + align256((size_t)batch * q_heads * q_len * a.splits * 8) : 256;
  if (!workspace) {
    *workspace_bytes = need;
    return SVQ_OK;
  }
  if (!q || !y || !table || !lens) return SVQ_ERR_INVALID_ARG;
  if (*workspace_bytes < need) return SVQ_ERR_BUFFER_TOO_SMALL;
  a.q = (const uint16_t *)q;
  a.y = (uint16_t *)y;
  a.ldq = ldq;
  a.ldy = ldy;
  a.table = table;
  a.ld_table = ld_table;
  a.lens = lens;
  a.batch = (int32_t)batch;
  a.q_len = q_len;
  a.heads = q_heads;
  a.max_len = (int32_t)max_len;
  a.window = window;
  a.scale = scale;
  if (a.splits > 1) {
    a.part = (float *)workspace;
    a.sums = (float *)((uint8_t *)workspace + part);
  }
  return of(launch_attn_cache(a, (hipStream_t)stream));
}

}  // extern "C"
