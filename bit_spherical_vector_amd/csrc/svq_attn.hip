// Attention over whole prompts (include/svq_attn.h).
//
// One pass over the keys with a running maximum and sum.  A block takes a tile
// of tokens of one key head, row r being query head r % G of the G that share
// it and token r / G of the tile, so the heads that share keys share their
// reads and a block's rows span few positions under a causal mask.  A wave owns 32
// rows and forms everything transposed:
//
//   S^T = K Q^T     32 keys x 32 rows (v_mfma_f32_32x32x16_bf16, A = keys)
//   O^T += V^T P^T  32 channels x 32 rows per step of 16 keys
//
// so a lane holds scores of one row only: the maximum, the exponentials and
// their sum stay in the lane, but for one exchange between the wave's halves,
// and P^T leaves the scores' registers in the layout that the second product
// reads, when the keys of a step are taken in the order of those registers
// (keys 16t + 4h + 0..3 and 16t + 8 + 4h + 0..3 in half h).  V is read
// transposed out of LDS (ds_read_b64_tr_b16: four keys of one channel a lane).
//
// Tiles of 64 keys: two of K and two of V in LDS (64 KB at 128 channels, two
// blocks a compute unit), copied by buffer loads while earlier ones are worked
// on.  The next tile's score products are issued between this tile's weights,
// so that the matrix unit runs while the vector unit takes exponentials.  More
// rows a block (8 waves) halve the copies but leave one block a unit, which
// waits for itself at every barrier: 2048 tokens 62 us against 51 of the same
// kernel with 4.  Two teams of 4 waves on the same rows, every second tile
// each, are no gain either (49 against 47): a tile takes 1800 cycles instead of
// 2650, but a block's first loads and its end (18000 cycles) no longer overlap
// another's tiles.
//
// What bounds it: over long prompts the matrix unit with the clock that the
// power allows (65 % of the cycles busy; 16384 tokens, 32 heads of 128 channels,
// causal: 1920-2040 us from box to box, 1.08-1.14 PFLOP/s, where a library product
// of 8192^3 reaches 1.36); at 2048 tokens (44.8 us, 770 TFLOP/s) the block with the most keys,
// alone on its unit for most of the time at 2650 cycles a tile, 1024 of them the
// matrix unit's; for short sequences the first loads (5000 to 8000 cycles).
#include "svq_attn.h"
#include "svq_device.h"

namespace svq {
namespace {

constexpr int KT = 64;       // keys of a tile
constexpr float GROW = 8.f;  // by how much (base 2) a row's maximum grows before its reference follows

typedef __attribute__((address_space(3))) uint8_t lds_t;
typedef short s4v __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s4v lds_s4v;
typedef __attribute__((address_space(3))) u4 lds_u4;

// A buffer from `base` on: reads beyond its bytes (element 2) give zeros.
__device__ __forceinline__ u4 buffer_at(const uint8_t *base) {
  const uint64_t at = (uint64_t)base;
  return (u4){(uint32_t)__builtin_amdgcn_readfirstlane((int)at), (uint32_t)__builtin_amdgcn_readfirstlane((int)(at >> 32)) & 0xFFFFu, 0u, 0x00020000u};
}
// The compiler does not look into the copies below, so the wait states between
// the vector unit's writes of these scalars and their first use there stand here
// (and between M0 and its use, there); nothing but scalar instructions touches
// them after.
__device__ __forceinline__ void settle(u4 &a, u4 &b) { asm volatile("s_nop 4" : "+s"(a), "+s"(b)); }
// 16 bytes a lane from byte off + first of the buffer to LDS bytes dst + 16 *
// lane, waited for by vmcnt.  (The builtin makes every LDS read behind it wait
// for the copy.)
__device__ __forceinline__ void copy_to_lds(const u4 &buffer, uint32_t off, uint32_t first, uint32_t dst) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(dst), "v"(off), "s"(buffer), "s"(first) : "memory", "m0");
}

// Rows of a staged tile are D bf16 values, 16-byte chunk c at place
// c ^ swizzle(key): 16 consecutive keys' equal chunks (a fragment of K) and
// four consecutive keys' 64-byte pieces (a transposed fragment of V) fill all
// 64 banks.
template <int D>
__device__ __forceinline__ int swizzle(int key) {
  return D == 64 ? ((key >> 1 & 1) << 2) | (key >> 2 & 3) : ((key & 3) << 2) | (key >> 2 & 3);
}

// v of the lane's place in the lower half and in the upper half.
__device__ __forceinline__ float2 both_halves(float v) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v);
  const auto r = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  const uint32_t lower = r[0], upper = r[1];
  return make_float2(__builtin_bit_cast(float, lower), __builtin_bit_cast(float, upper));
}
__device__ __forceinline__ float max_halves(float v) {
  const float2 r = both_halves(v);
  return fmaxf(r.x, r.y);
}
// The greater value, NaN if one is (one instruction for three; fmaxf takes one
// more for each value that a matrix product has left).
__device__ __forceinline__ float max_nan(float a, float b) { return __builtin_elementwise_maximum(a, b); }
__device__ __forceinline__ float sum_halves(float v) {
  const float2 r = both_halves(v);
  return r.x + r.y;
}

typedef __bf16 b2 __attribute__((ext_vector_type(2)));
typedef float f2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pk_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2){a, b}, b2));
}
// c plus both halves of a.
__device__ __forceinline__ float add_bf16(uint32_t a, float c) {
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(b2, a), (b2){(__bf16)1.f, (__bf16)1.f}, c, false);
}
__device__ __forceinline__ f16x mfma_bf16(const u4 &a, const u4 &b, const f16x &c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(b8, a), __builtin_bit_cast(b8, b), c, 0, 0, 0);
}

// The sum of v over the lanes up to the lane's own: within rows of 16 lanes,
// then the last lane of a row to the next row and of the lower half to the upper.
template <int CTRL, int ROWS>
__device__ __forceinline__ int add_dpp(int v) {
  return v + __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ int sum_below(int v) {
  v = add_dpp<0x111, 0xF>(v);  // row_shr:1
  v = add_dpp<0x112, 0xF>(v);
  v = add_dpp<0x114, 0xF>(v);
  v = add_dpp<0x118, 0xF>(v);
  v = add_dpp<0x142, 0xA>(v);  // row_bcast:15
  return add_dpp<0x143, 0xC>(v);  // row_bcast:31
}

// The sequence and tile of number `u` of the tiles of all sequences in order;
// false beyond the last.  Every wave looks for itself, 64 sequences at a time,
// in one trip to memory.
struct TileOf {
  int q_at, n, k_at, keys, tile;
};
__device__ __forceinline__ bool find_tile(const AttnPromptArgs &a, const PromptPlan &plan, int u, TileOf &o) {
  const int lane = threadIdx.x & 63;
  int before = 0;
  for (int s0 = 0; s0 < a.sequences; s0 += 64) {
    const int s = s0 + lane;
    int b = 0, e = 0, kb = 0, ke = 0;
    if (s < a.sequences) {
      b = a.starts[s];
      e = a.starts[s + 1];
      kb = a.starts_k[s];
      ke = a.starts_k[s + 1];
    }
    b = min(max(b, 0), a.tokens);
    e = min(max(e, b), a.tokens);
    kb = min(max(kb, 0), a.tokens_k);
    ke = min(max(ke, kb), a.tokens_k);
    const int tiles = quotient(e - b + plan.tokens - 1, plan.tokens_mul);
    const int sum = sum_below(tiles);
    const uint64_t past = __ballot(before + sum > u);
    if (past) {
      const int at = __builtin_ctzll(past);
      o.q_at = __builtin_amdgcn_readlane(b, at);
      o.n = __builtin_amdgcn_readlane(e, at) - o.q_at;
      o.tile = u - before - (__builtin_amdgcn_readlane(sum, at) - __builtin_amdgcn_readlane(tiles, at));
      o.k_at = __builtin_amdgcn_readlane(kb, at);
      o.keys = __builtin_amdgcn_readlane(ke, at) - o.k_at;
      return true;
    }
    before += __builtin_amdgcn_readlane(sum, 63);
  }
  return false;
}

__device__ __forceinline__ uint32_t finite_or_zero(uint32_t x) {
  const uint32_t lo = x & 0xFFFFu, hi = x & 0xFFFF0000u;
  return ((lo & 0x7F80u) == 0x7F80u ? 0u : lo) | ((hi & 0x7F800000u) == 0x7F800000u ? 0u : hi);
}

// LDS bytes of the tiles: K and V of two each, and (64 channels) 4 KB a wave
// from the last one on.
template <int D, int NW>
constexpr int prompt_tiles() {
  constexpr int SIDE = KT * 2 * D;
  return 4 * SIDE > 3 * SIDE + NW * 4096 ? 4 * SIDE : 3 * SIDE + NW * 4096;
}

template <int D, int NW>
__global__ __launch_bounds__(64 * NW, D == 256 ? 1 : 2) void attn_prompt_kernel(AttnPromptArgs a, PromptPlan plan) {
  constexpr int ROW = 2 * D, CH = D / 8, SIDE = KT * ROW;  // bytes of a row, its chunks, bytes of a tile
  constexpr int NB = D / 32, NS = D / 16;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];  // K and V of two tiles each, from LDS byte 0 on
  int(*odd)[NW] = (int(*)[NW])(smem + prompt_tiles<D, NW>());  // which waves have met values that are not finite
  const int tid = threadIdx.x, lane = tid & 63, col = lane & 31, h = lane >> 5;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int kvh = blockIdx.x, G = plan.G;
  TileOf T;
  if (!find_tile(a, plan, prompt_tile(plan, blockIdx.y), T)) return;
  const int t_first = T.tile * plan.tokens, rows = min(plan.tokens, T.n - t_first) * G;
  const int shift = T.keys - T.n + t_first;  // position of the tile's first token

  // what a row sees, by its token: keys [lo, hi)
  auto hi_of = [&](int token) { return a.causal ? min(max(shift + token + 1, 0), T.keys) : T.keys; };
  auto lo_of = [&](int token) { return a.window > 0 ? max(0, shift + token + 1 - a.window) : 0; };
  const int last = min(plan.tokens, T.n - t_first) - 1;
  int t0 = lo_of(0) / KT, t1 = (hi_of(last) + KT - 1) / KT;
  const int b_lo1 = lo_of(last), b_hi0 = hi_of(0);
  if (a.splits > 1) {
    const int per = (max(t1 - t0, 0) + a.splits - 1) / a.splits;
    t0 += blockIdx.z * per;
    t1 = min(t1, t0 + per);
  }
  const bool mine = 32 * wv < rows;  // the wave has rows
  const int w_hi0 = hi_of(quotient16(min(32 * wv, rows - 1), plan.g_mul));
  const int w_lo1 = lo_of(quotient16(min(32 * wv + 31, rows - 1), plan.g_mul));
  const int r = min(32 * wv + col, rows - 1), token = quotient16(r, plan.g_mul);
  const int lo = lo_of(token), hi = hi_of(token);
  const int64_t row_off = (int64_t)(T.q_at + t_first + token);
  const int head = kvh * G + r - token * G;

  // staging: pieces of 1 KB (1024 / ROW keys), piece i * NW + wv by wave wv; a
  // lane's place in a piece is the same for every i (i & 1 with 256 channels
  // and four waves)
  const uint8_t *kg = (const uint8_t *)(a.k + (int64_t)T.k_at * a.ldk + kvh * D);
  const uint8_t *vg = (const uint8_t *)(a.v + (int64_t)T.k_at * a.ldv + kvh * D);
  constexpr int PER = SIDE / 1024 / NW, KEYS = 1024 / ROW, KINDS = D == 256 && NW == 4 ? 2 : 1;
  const uint32_t ldk = (uint32_t)a.ldk * 2, ldv = (uint32_t)a.ldv * 2;
  uint32_t off_k[KINDS], off_v[KINDS];
#pragma unroll
  for (int i = 0; i < KINDS; ++i) {
    const int key = (i * NW + wv) * KEYS + lane / CH, chunk = ((lane % CH) ^ swizzle<D>(key)) * 16;
    off_k[i] = key * ldk + chunk;
    off_v[i] = key * ldv + chunk;
  }
  const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_t *)smem;  // two places of K, two of V, taken in turn from tile t0 on
  // tile t of the keys (values) as a buffer that ends with the sequence: rows
  // behind it become zeros, a tile behind it is not read
  auto ends = [&](u4 &buffer, uint32_t ld, int t) {
    const int left = T.keys - t * KT;
    buffer[2] = left > 0 ? (uint32_t)(min(left, KT) - 1) * ld + ROW : 0u;
  };
  auto advance = [&](u4 &buffer, uint32_t ld, int t) {
    const uint64_t at = ((uint64_t)buffer[1] << 32 | buffer[0]) + (uint64_t)(KT * ld);
    buffer[0] = (uint32_t)at;
    buffer[1] = (uint32_t)(at >> 32);
    ends(buffer, ld, t);
  };
  auto copy_k = [&](const u4 &buffer, int place, int i) {
    copy_to_lds(buffer, off_k[i % KINDS], i / KINDS * KINDS * NW * KEYS * ldk, lds0 + place * SIDE + (i * NW + wv) * 1024);
  };
  auto copy_v = [&](const u4 &buffer, int place, int i) {
    copy_to_lds(buffer, off_v[i % KINDS], i / KINDS * KINDS * NW * KEYS * ldv, lds0 + (2 + place) * SIDE + (i * NW + wv) * 1024);
  };

  // fragment addresses, a chunk's place an exclusive or: K chunk 2s + h of key
  // col (32 kb more: 32 rows on); V^T keys 8jj + 4h + r4 (16t more: 16 rows
  // on), channels 32db + 16g + 4c
  const uint32_t ka = lds0 + col * ROW + ((h ^ swizzle<D>(col)) << 4);
  uint32_t va[2];
#pragma unroll
  for (int jj = 0; jj < 2; ++jj) {
    const int g = lane >> 4 & 1, c = lane & 3, key = 8 * jj + 4 * h + (lane >> 2 & 3);
    va[jj] = lds0 + 2 * SIDE + key * ROW + (((2 * g + (c >> 1)) ^ swizzle<D>(key)) << 4) + 8 * (c & 1);
  }

  // the first tiles are on their way before the queries are asked for
  u4 buf_k = buffer_at(kg + (int64_t)t0 * KT * ldk), buf_v = buffer_at(vg + (int64_t)t0 * KT * ldv);
  ends(buf_k, ldk, t0);
  ends(buf_v, ldv, t0);
  settle(buf_k, buf_v);
  if (t0 < t1) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      copy_k(buf_k, 0, i);
      copy_v(buf_v, 0, i);
    }
    advance(buf_k, ldk, t0 + 1);
    settle(buf_k, buf_v);
#pragma unroll
    for (int i = 0; i < PER; ++i) copy_k(buf_k, 1, i);
  }
  // Queries come as whole lines, eight lanes 64 channels of a row, and pass
  // through LDS (the second place of V, 4 KB a wave) to the lanes of their rows.
  u4 qf[NS];
  {
    const uint32_t flip = a.scale < 0.f ? 0x80008000u : 0u, to = lds0 + 3 * SIDE + wv * 4096;
    u4 raw[D / 64][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = min(32 * wv + 8 * i + (lane >> 3), rows - 1), token = quotient16(r, plan.g_mul);
      const uint16_t *q = a.q + (int64_t)(T.q_at + t_first + token) * a.ldq + (kvh * G + r - token * G) * D + 8 * (lane & 7);
#pragma unroll
      for (int p = 0; p < D / 64; ++p) raw[p][i] = *(const u4 *)(q + 64 * p);
    }
#pragma unroll
    for (int p = 0; p < D / 64; ++p) {
      // chunk c of row n at place c ^ (n / 2 % 8)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *(lds_u4 *)(lds_t *)(uintptr_t)(to + i * 1024 + (lane >> 3) * 128 + (((lane & 7) ^ ((4 * i + (lane >> 4)) & 7)) << 4)) = raw[p][i] ^ flip;
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
      for (int s = 0; s < 4; ++s) qf[4 * p + s] = *(const lds_u4 *)(lds_t *)(uintptr_t)(to + col * 128 + (((2 * s + h) ^ (col >> 1 & 7)) << 4));
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
  }
  const float sc = exponent_scale(a.scale);

  f16x O[NB];
#pragma unroll
  for (int db = 0; db < NB; ++db) O[db] = (f16x){};
  float m = -__FLT_MAX__, mref = 0.f, most = m, l = 0.f;  // most: the greatest score without a new reference
  bool dirty = false, far_any = false;

  u4 kf[2][2];
  auto load_k = [&](int place, int s) {
    const uint32_t at = (ka + place * SIDE) ^ (s << 5);
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) kf[s & 1][kb] = *(const lds_u4 *)(lds_t *)(uintptr_t)(at + kb * 32 * ROW);
  };

  // The reference lies GROW above the maximum, so that weights are at most 1
  // until the next one.  One beyond 2^24 is rounded by more than one: such a row's
  // weights are taken from the maximum, the scores' differences formed before the
  // scale.
  auto far = [&]() { return fabsf(mref) > 16777216.f; };
  // How far the scaled maximum lies above the reference that weights are taken
  // from (-GROW, and up to a half off it near 2^24).
  auto above = [&]() { return far() || m == -__FLT_MAX__ ? -GROW : fmaf(m, sc, -mref); };

  // Tile t, its V in `place`: S holds its scores and N takes the next tile's.
  float top = 0.f;
  auto maximum = [&](const f16x (&S)[2]) {
    top = max_nan(S[0][0], S[1][0]);
#pragma unroll
    for (int i = 1; i < 16; ++i) top = max_nan(max_nan(top, S[0][i]), S[1][i]);
  };
  auto step = [&](int t, int turn, f16x (&S)[2], f16x (&N)[2]) {
    // A constant saves address arithmetic.  At 256 channels, whose registers are
    // all taken, the second set of addresses would be spilled (8192 tokens, 16
    // heads: 629 us against 611).
    int place = turn;
    if constexpr (D == 256) asm volatile("" : "+s"(place));
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    const int k0 = t * KT;
    const bool edge = k0 < b_lo1 || k0 + KT > b_hi0;  // some row of the block does not see all keys
    if (edge) {
      // P^T is zero for a hidden key, but zero times infinity is not.  A wave
      // looks at the values that it has copied itself.
      uint32_t mag = 0;
      const uint32_t at = lds0 + (2 + place) * SIDE + wv * 1024 + lane * 16;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const u4 x = *(const lds_u4 *)(lds_t *)(uintptr_t)(at + i * NW * 1024);
#pragma unroll
        for (int w = 0; w < 4; ++w) mag = pk_max_mag(mag, x[w]);
      }
      odd[place][wv] = __any((mag & 0xFFFF) >= 0x7F80 || mag >= 0x7F800000u);
    }
    __syncthreads();  // V of t and K of t + 1 are there; nobody reads V of t - 1 and K of t
    advance(buf_k, ldk, t + 2);
    advance(buf_v, ldv, t + 1);
    settle(buf_k, buf_v);
    if (edge) {
      int any = 0;
#pragma unroll
      for (int w = 0; w < NW; ++w) any |= odd[place][w];
      if (__builtin_expect(__builtin_amdgcn_readfirstlane(any), 0)) {
        // values that are not finite become zero, and the rows that do see
        // them get them at the end
        dirty = true;
        for (int i = wv; i < SIDE / 1024; i += NW) {
          lds_u4 *x = (lds_u4 *)(lds_t *)(uintptr_t)(lds0 + (2 + place) * SIDE + i * 1024 + lane * 16);
          u4 v = *x;
#pragma unroll
          for (int w = 0; w < 4; ++w) v[w] = finite_or_zero(v[w]);
          *x = v;
        }
        __syncthreads();
      }
    }
    if (!mine) {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        copy_k(buf_k, place, i);
        copy_v(buf_v, place ^ 1, i);
      }
      return;
    }
    if (k0 < w_lo1 || k0 + KT > w_hi0) {
      // register i of half h is key 32 kb + 8 (i / 4) + 4 h + i % 4 of the tile
      const int first = lo - k0 - 4 * h, end = hi - k0 - 4 * h;
      if (k0 + KT > w_hi0) {
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
          for (int i = 0; i < 16; ++i) S[kb][i] = 32 * kb + 8 * (i >> 2) + (i & 3) < end ? S[kb][i] : -__builtin_inff();
      }
      if (k0 < w_lo1) {
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
          for (int i = 0; i < 16; ++i) S[kb][i] = 32 * kb + 8 * (i >> 2) + (i & 3) >= first ? S[kb][i] : -__builtin_inff();
      }
      maximum(S);
    }
    // a new reference only once the maximum has grown by 2^GROW: weights down
    // from 2^-GROW are as exact as weights from 1 (the growth formed before the
    // scale: beyond 2^27 a scaled maximum and the reference are 16 and more apart)
    if (__any(top > most)) {
      const float old_m = m, old_above = above();
      const bool first = m == -__FLT_MAX__;
      // of the rows that need one: the others keep theirs, and with it every bit
      // of their weights, whatever the wave's other rows see
      const float row = max_halves(top);
      if (row > most) m = row;
      most = raised_by(m, GROW, sc);
      mref = m == -__FLT_MAX__ ? 0.f : fmaf(m, sc, GROW);
      far_any = __any(far());
      const float alpha = first ? 0.f : __builtin_amdgcn_exp2f((old_m - m) * sc + (above() - old_above));
      l *= alpha;
#pragma unroll
      for (int db = 0; db < NB; ++db)
#pragma unroll
        for (int i = 0; i < 16; ++i) O[db][i] *= alpha;
    }
    float less = mref;
    if (__builtin_expect(far_any, 0)) {
      less = far() ? GROW : mref;
      const float before = far() ? m : 0.f;
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int i = 0; i < 16; ++i) S[kb][i] -= before;
    }
    // The weights, between the next tile's score products: one product, then
    // the exponentials of EACH scores and the rounding of the EACH before them,
    // which keeps the vector unit busy for as long as the product runs.
    u4 pf[4];
    constexpr int EACH = NS < 8 ? 4 : 2, EVERY = NS > 8 ? 2 : 1;  // scores; after every product or every second one
    float x[EACH], y[EACH];
    auto exps = [&](int n) {
#pragma unroll
      for (int e = 0; e < EACH; ++e) x[e] = __builtin_amdgcn_exp2f(fmaf(S[(EACH * n + e) >> 4][(EACH * n + e) & 15], sc, -less));
    };
    auto round = [&](int n) {
#pragma unroll
      for (int e = 0; e < EACH; e += 2) {
        const int at = EACH * n + e;
        const uint32_t p = pk_bf16(y[e], y[e + 1]);
        l = add_bf16(p, l);
        pf[at >> 3][(at & 7) >> 1] = p;
      }
    };
    load_k(place ^ 1, 0);
    N[0] = N[1] = (f16x){};
#pragma unroll
    for (int n = 0; n < 2 * NS; ++n) {
      const int s = n >> 1, kb = n & 1;
      if (kb == 0 && s + 1 < NS) load_k(place ^ 1, s + 1);
      N[kb] = mfma_bf16(kf[s & 1][kb], qf[s], N[kb]);
      // copies one by one: all at once they hold the wave until the last is taken
      if (n % 4 == 0 && n / 4 < PER) copy_k(buf_k, place, n / 4);
      if (n % 4 == 2 && n / 4 < PER) copy_v(buf_v, place ^ 1, n / 4);
      if (n % EVERY == 0) {
        exps(n / EVERY);
        if (n > 0) round(n / EVERY - 1);
#pragma unroll
        for (int e = 0; e < EACH; ++e) y[e] = x[e];
      }
    }
    round(32 / EACH - 1);
    u4 vf[2][NB];
    auto load_v = [&](int n) {
#pragma unroll
      for (int db = 0; db < NB; ++db) {
        u2 x[2];
#pragma unroll
        for (int jj = 0; jj < 2; ++jj) {
          const uint32_t at = ((va[jj] + place * SIDE) ^ (db << 6)) + n * 16 * ROW;
          x[jj] = __builtin_bit_cast(u2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4v *)(lds_t *)(uintptr_t)at));
        }
        vf[n & 1][db] = (u4){x[0][0], x[0][1], x[1][0], x[1][1]};
      }
    };
    load_v(0);
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      if (n + 1 < 4) load_v(n + 1);
#pragma unroll
      for (int db = 0; db < NB; ++db) O[db] = mfma_bf16(vf[n & 1][db], pf[n], O[db]);
      // the next tile's maximum, a third at a time
      if (n == 1) top = max_nan(N[0][0], N[1][0]);
      if (n > 0) {
#pragma unroll
        for (int i = 5 * n - 4; i <= 5 * n; ++i) top = max_nan(max_nan(top, N[0][i]), N[1][i]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  if (t0 < t1) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    f16x A[2] = {(f16x){}, (f16x){}}, B[2];
    load_k(0, 0);
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      if (s + 1 < NS) load_k(0, s + 1);
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) A[kb] = mfma_bf16(kf[s & 1][kb], qf[s], A[kb]);
    }
    maximum(A);
#pragma unroll 1
    for (int t = t0; t < t1; t += 2) {
      step(t, 0, A, B);
      if (t + 1 < t1) step(t + 1, 1, B, A);
    }
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no copy outlives the block
  if (32 * wv + col >= rows) return;
  if (dirty)
    for (int t = t0; t < t1; ++t) {
      const int k0 = t * KT;
      if (k0 >= b_lo1 && k0 + KT <= b_hi0) continue;
      for (int key = max(k0, lo); key < min(k0 + KT, hi); ++key) {
        const uint16_t *v = (const uint16_t *)(vg + (int64_t)key * ldv) + 4 * h;
#pragma unroll
        for (int db = 0; db < NB; ++db)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const uint32_t x = v[32 * db + 8 * (i >> 2) + (i & 3)];
            O[db][i] += (x & 0x7F80u) == 0x7F80u ? bf16_bits_to_f32(x) : 0.f;
          }
      }
    }
  // the lane's half of the row's sum is added to its partner's, which is in
  // the same state
  l = sum_halves(l);
  if (a.splits > 1) {
    const int64_t at = (row_off * a.heads + head) * a.splits + blockIdx.z;
    if (h == 0) *(f4 *)(a.sums + 4 * at) = (f4){m, above(), l, t0 >= t1 ? -1.f : 0.f};
    if (t0 >= t1) return;  // no keys: its numerators are not read
    float *part = a.part + at * D + 4 * h;
#pragma unroll
    for (int db = 0; db < NB; ++db)
#pragma unroll
      for (int i = 0; i < 16; i += 4) *(f4 *)(part + 32 * db + 2 * i) = (f4){O[db][i], O[db][i + 1], O[db][i + 2], O[db][i + 3]};
    return;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint16_t *y = a.y + row_off * a.ldy + head * D;
#pragma unroll
  for (int db = 0; db < NB; ++db)
#pragma unroll
    for (int i = 0; i < 16; i += 4)
      *(u2 *)(y + 32 * db + 2 * i + 4 * h) = (u2){pk_bf16(O[db][i] * inv, O[db][i + 1] * inv),
                                                 pk_bf16(O[db][i + 2] * inv, O[db][i + 3] * inv)};
}

// Joins the key ranges of a row, each under its own reference: D / 4 threads a
// row, four channels a thread.  Rows that no sequence has are left alone.  A
// numerator that is not finite (of a value that is not) stays what it is under
// any weight.  Latency and reads: 4000 rows of 128 channels in 7 ranges, 14.5 MB, take
// 6 of the call's 23.5 us.
template <int D>
__global__ __launch_bounds__(256) void prompt_join_kernel(AttnPromptArgs a) {
  constexpr int T = D / 4;
  const int64_t row = (int64_t)blockIdx.x * (256 / T) + threadIdx.x / T;
  const int part = threadIdx.x % T, token = (int)(row / a.heads), head = (int)(row - (int64_t)token * a.heads);
  if (token < max(a.starts[0], 0) || token >= min(a.starts[a.sequences], a.tokens)) return;
  const f4 *sums = (const f4 *)a.sums + row * a.splits;
  const float sc = exponent_scale(a.scale);
  float m = -__FLT_MAX__;
#pragma unroll 4
  for (int s = 0; s < a.splits; ++s) m = fmaxf(m, sums[s][0]);
  f4 o = {};
  float sum = 0.f;
  const f4 *num = (const f4 *)(a.part + row * a.splits * D) + part;
#pragma unroll 4
  for (int s = 0; s < a.splits; ++s) {
    const f4 x = sums[s], v = num[(int64_t)s * T];
    // a range in which the row sees nothing has zeros, one without keys has
    // left what was there
    const float f = x[0] == -__FLT_MAX__ && x[2] == 0.f ? 0.f : __builtin_amdgcn_exp2f((x[0] - m) * sc - (x[1] + GROW));
    sum += x[2] * f;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] += x[3] < 0.f ? 0.f : fabsf(v[e]) < __builtin_inff() ? v[e] * f : v[e];
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  *(u2 *)(a.y + token * a.ldy + head * D + 4 * part) = (u2){pk_bf16(o[0] * inv, o[1] * inv), pk_bf16(o[2] * inv, o[3] * inv)};
}

template <int D>
hipError_t launch(const AttnPromptArgs &a, hipStream_t s) {
  constexpr int NW = PROMPT_WAVES;
  constexpr size_t lds = prompt_tiles<D, NW>() + 2 * NW * sizeof(int);
  const hipError_t e = allow_smem(attn_prompt_kernel<D, NW>, lds);
  if (e != hipSuccess) return e;
  const PromptPlan plan = prompt_plan(a.tokens, a.sequences, a.heads, a.kv_heads, NW, compute_units());
  prompt_launches(plan, [&](const PromptPlan &p, int n) {
    attn_prompt_kernel<D, NW><<<dim3(a.kv_heads, n, a.splits), 64 * NW, lds, s>>>(a, p);
  });
  if (a.splits > 1) {
    const int64_t rows = (int64_t)a.tokens * a.heads, per = 256 / (D / 4);
    prompt_join_kernel<D><<<dim3((unsigned)((rows + per - 1) / per)), 256, 0, s>>>(a);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_prompt(const AttnPromptArgs &a, hipStream_t s) {
  switch (a.dim) {
    case 64: return launch<64>(a, s);
    case 128: return launch<128>(a, s);
    default: return launch<256>(a, s);
  }
}

}  // namespace svq
