// The 4-bit cache of keys and values (include/svq_attn.h): quantising tokens
// into it, reading them back, attention over it.
#include "svq_attn.h"
#include "svq_device.h"

#include <type_traits>

namespace svq {
namespace {

// Maximum over groups of 2, 4, 8 or 16 consecutive lanes.
template <int CTRL>
__device__ __forceinline__ float dpp_max(float v) {
  const int o = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, false);
  return fmaxf(v, __builtin_bit_cast(float, o));
}
__device__ __forceinline__ float lanes_max(float v, int lanes) {
  if (lanes > 1) v = dpp_max<0xB1>(v);   // quad_perm [1,0,3,2]
  if (lanes > 2) v = dpp_max<0x4E>(v);   // quad_perm [2,3,0,1]
  if (lanes > 4) v = dpp_max<0x141>(v);  // row_half_mirror
  if (lanes > 8) v = dpp_max<0x140>(v);  // row_mirror
  return v;
}

struct KvScale {
  float s, m, r;  // scale, minimum, 1 / scale
  uint32_t bits;  // as stored
};
// The parameters of a group of greatest value hi and least value -nlo.  A NaN
// among its values has made hi infinite.
__device__ __forceinline__ KvScale kv_scale(float hi, float nlo) {
  KvScale p;
  if (!(hi < __builtin_inff()) || !(nlo < __builtin_inff())) {
    p.s = p.m = p.r = 0.f;
    p.bits = 0x7FC07FC0u;
    return p;
  }
  p.m = -nlo;
  const uint32_t sb = f32_to_bf16_bits((float)(((double)hi - (double)p.m) / 15.0));
  p.s = bf16_bits_to_f32(sb);
  p.r = 1.f / p.s;
  p.bits = sb | (__builtin_bit_cast(uint32_t, p.m) & 0xFFFF0000u);
  return p;
}
// Nearest whole number to (x - m) / s.  The fp32 quotient is off by less than
// 3e-6, so only one that near to a border (or not finite) asks for 64 bits,
// where the difference of two bf16 values 2^45 apart and less is exact.
__device__ __forceinline__ uint32_t kv_code(float x, const KvScale &p) {
  if (p.s == 0.f) return 0;
  const float t = (x - p.m) * p.r;
  float q = rintf(t);
  if (!(fabsf(fabsf(t - q) - 0.5f) > 1e-4f)) q = (float)rint(((double)x - (double)p.m) / (double)p.s);
  return (uint32_t)fminf(q, 15.f);
}

// 16 lanes a (token, head), four tokens a wave, so that the value runs of
// four neighbouring slots (one 256-byte piece at 128 channels) leave in one
// store.  A lane holds D/16 channels: consecutive ones of the keys, 16t + r of
// the values.
template <int D, int SIDE>
__global__ __launch_bounds__(256) void kv_write_kernel(KvWriteArgs a) {
  constexpr int N = D / 16;
  const int lane = threadIdx.x & 63, r = lane & 15;
  const int head = blockIdx.y;
  const int64_t t = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
  const int32_t slot = t < a.tokens ? a.slots[t] : -1;
  const bool in = slot >= 0 && slot < a.c.pages << a.c.page_shift;  // uniform over the 16 lanes
  const uint16_t *src = SIDE ? a.v + (in ? t : 0) * a.ldv : a.k + (in ? t : 0) * a.ldk;
  src += head * D;
  float x[N], hi[N], nlo[N];
  if constexpr (SIDE == 0) {
    uint16_t raw[N];
    __builtin_memcpy(raw, src + r * N, sizeof(raw));
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = bf16_bits_to_f32(raw[i]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = bf16_bits_to_f32(src[16 * i + r]);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const bool nan = x[i] != x[i];
    hi[i] = nan ? __builtin_inff() : x[i];
    nlo[i] = nan ? __builtin_inff() : -x[i];
  }
  uint8_t *blk = kv_block(a.c, slot >> a.c.page_shift, head);
  const int place = slot & ((1 << a.c.page_shift) - 1);
  uint32_t word[(N + 7) / 8] = {};
  if constexpr (SIDE == 0) {
#pragma unroll
    for (int i = 1; i < N; ++i) {
      hi[0] = fmaxf(hi[0], hi[i]);
      nlo[0] = fmaxf(nlo[0], nlo[i]);
    }
    const int lanes = (1 << a.c.group_shift) / N;  // lanes of a group
    const KvScale p = kv_scale(lanes_max(hi[0], lanes), lanes_max(nlo[0], lanes));
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int j = N == 4 ? 4 * (r & 1) + i : i & 7;
      word[i >> 3] |= kv_code(x[i], p) << 4 * kv_nibble(j);
    }
    if constexpr (N == 4) word[0] |= __builtin_amdgcn_update_dpp(0, word[0], 0xB1, 0xF, 0xF, false);
    if (!in) return;
#pragma unroll
    for (int w = 0; w < (N + 7) / 8; ++w) {
      const int n = N == 4 ? r >> 1 : r * (N / 8) + w;  // channels 8n ..
      if (N > 4 || !(r & 1)) *(uint32_t *)(blk + kv_key_word(a.c, place, n)) = word[w];
    }
    if (r % lanes == 0) *(uint32_t *)(blk + kv_param(a.c, 0, place, r / lanes)) = p.bits;
  } else {
    const int tiles = 1 << (a.c.group_shift - 4);  // 2, 4 or 8 of a group
#pragma unroll
    for (int g0 = 0; g0 < N; g0 += 2) {
      if (g0 & (tiles - 1)) continue;
      float h = -__builtin_inff(), l = -__builtin_inff();
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < tiles && g0 + i < N) {
          h = fmaxf(h, hi[g0 + i < N ? g0 + i : 0]);
          l = fmaxf(l, nlo[g0 + i < N ? g0 + i : 0]);
        }
      const KvScale p = kv_scale(lanes_max(h, 16), lanes_max(l, 16));
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < tiles && g0 + i < N) word[(g0 + i) >> 3] |= kv_code(x[g0 + i < N ? g0 + i : 0], p) << 4 * ((g0 + i) & 7);
      if (in && r == 0) *(uint32_t *)(blk + kv_param(a.c, 1, place, g0 / tiles)) = p.bits;
    }
    if (!in) return;
    __builtin_memcpy(blk + kv_value_run(a.c, place, r), word, N / 2);
  }
}

template <int D, int SIDE>
__global__ __launch_bounds__(256) void kv_read_kernel(KvReadArgs a) {
  constexpr int N = D / 16;
  const int lane = threadIdx.x & 63, r = lane & 15;
  const int head = blockIdx.y;
  const int64_t t = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
  if (t >= a.tokens) return;
  const int32_t slot = a.slots[t];
  const bool in = slot >= 0 && slot < a.c.pages << a.c.page_shift;
  const uint8_t *blk = kv_block(a.c, in ? slot >> a.c.page_shift : 0, head);
  const int place = in ? slot & ((1 << a.c.page_shift) - 1) : 0;
  float x[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int d = SIDE ? 16 * i + r : r * N + i;
    const uint32_t p = *(const uint32_t *)(blk + kv_param(a.c, SIDE, place, d >> a.c.group_shift));
    uint32_t code;
    if constexpr (SIDE == 0) {
      const int n = d >> 3;
      const uint32_t w = *(const uint32_t *)(blk + kv_key_word(a.c, place, n));
      code = (w >> 4 * kv_nibble(d & 7)) & 15;
    } else {
      code = (blk[kv_value_run(a.c, place, r) + (i >> 1)] >> 4 * (i & 1)) & 15;
    }
    const float v = fmaf((float)code, bf16_bits_to_f32(p & 0xFFFFu), __builtin_bit_cast(float, p & 0xFFFF0000u));
    x[i] = in ? v : 0.f;
  }
  const int64_t row = t * (SIDE ? a.ldv : a.ldk) + head * D;
#pragma unroll
  for (int i = 0; i < N; ++i) store_out(SIDE ? a.v : a.k, row + (SIDE ? 16 * i + r : r * N + i), x[i], a.f32);
}

// ---- attention over the cache -------------------------------------------
//
// A block takes 16 rows (query token t of q_len, query head g of the G that
// share a key head: row t * G + g) of one sequence and key head, and one of
// `splits` ranges of its keys; a wave every fourth chunk of 32 keys in it.
// Codes enter the matrix cores as they are: a nibble left in place by a mask
// is a subnormal fp16 number, c * 2^-24 or c * 16 * 2^-24, which
// v_mfma_f32_16x16x32_f16 multiplies exactly.  So, transposed (a lane holds
// one row, and four keys of each 16):
//
//   A_g[key][row] = sum over the group's channels of c * q     (q in fp16
//        under a power-of-two scale per row, a sixteenth of it where the
//        nibble stands for 16 c)
//   score         = sum over groups of s_g A_g + m_g sum q     (fp32)
//   O_t[channel][row] += sum over keys of c * (p s_g)          (p s_g in units
//        of 2^(E - 8) as the sum of two fp16 numbers, 22 bits: the minimum's
//        term below cancels much of this one, and with 11 bits a value near
//        zero would carry the rounding of its whole range)
//   M_g[row]          += sum over keys of p m_g                (fp32)
//
// and the row is (2^24 O + M) / sum p.  The weight p is exp2(score - ref), ref
// = m + E - 8: m a running maximum, raised once a score exceeds it by 6, E an
// exponent that is raised once a p s_g overflows fp16 (it starts so low that
// the first chunk raises it to the exponent of that chunk's greatest scale or
// minimum).
constexpr int CACHE_WAVES = 4, CACHE_STAGES = 3, CHUNK = 32, ROWS = 16;

typedef __attribute__((address_space(3))) uint8_t lds_t;
__device__ __forceinline__ uint32_t lds_u32(uint32_t at) {
  return *(const __attribute__((address_space(3))) uint32_t *)(lds_t *)(uintptr_t)at;
}
__device__ __forceinline__ u4 lds_u128(uint32_t at) {
  return *(const __attribute__((address_space(3))) u4 *)(lds_t *)(uintptr_t)at;
}
// 16 bytes a lane from base + off to LDS bytes dst + 16 * lane, waited for by
// vmcnt.  (The builtin makes every LDS read behind it wait for the copy.)  The
// wait states stand between the scalar values' writers and their use as M0 and
// as a base: the compiler does not look into the block.
__device__ __forceinline__ void copy_to_lds(const uint8_t *base, uint32_t off, uint32_t dst) {
  const uint32_t d = __builtin_amdgcn_readfirstlane(dst);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(d), "v"(off), "s"(base) : "memory", "m0");
}
template <int N>
__device__ __forceinline__ void wait_copies() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"i"(N) : "memory");
}

__device__ __forceinline__ float lo_bf16(uint32_t p) { return bf16_bits_to_f32(p & 0xFFFFu); }
__device__ __forceinline__ float hi_bf16(uint32_t p) { return __builtin_bit_cast(float, p & 0xFFFF0000u); }

// Over the four lanes that hold a row (lane % 16): maximum, sum.
__device__ __forceinline__ float2 swap32(float v) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v);
  const auto r = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  const uint32_t x = r[0], y = r[1];
  return make_float2(__builtin_bit_cast(float, x), __builtin_bit_cast(float, y));
}
__device__ __forceinline__ float2 swap16(float v) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v);
  const auto r = __builtin_amdgcn_permlane16_swap(b, b, false, false);
  const uint32_t x = r[0], y = r[1];
  return make_float2(__builtin_bit_cast(float, x), __builtin_bit_cast(float, y));
}
__device__ __forceinline__ float row_max(float v) {
  const float2 a = swap32(v);
  const float2 b = swap16(fmaxf(a.x, a.y));
  return fmaxf(b.x, b.y);
}
__device__ __forceinline__ float row_sum(float v) {
  const float2 a = swap32(v);
  const float2 b = swap16(a.x + a.y);
  return b.x + b.y;
}

// Four key words' steps of 8 channels as fp16 pairs (see kv_nibble).
__device__ __forceinline__ u4 nibbles(uint32_t w) {
  const uint32_t x = w >> 8;
  return (u4){w & 0x000F000Fu, w & 0x00F000F0u, x & 0x000F000Fu, x & 0x00F000F0u};
}

__device__ __forceinline__ f4 mfma_f16(const u4 &a, const u4 &b, const f4 &c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, a), __builtin_bit_cast(h8, b), c, 0, 0, 0);
}
__device__ __forceinline__ uint32_t pk_f16(_Float16 a, _Float16 b) {
  return (uint32_t)__builtin_bit_cast(uint16_t, a) | (uint32_t)__builtin_bit_cast(uint16_t, b) << 16;
}

template <int D, int GROUP>
__global__ __launch_bounds__(64 * CACHE_WAVES, 2) void attn_cache_kernel(AttnCacheArgs a) {
  constexpr int G = D / GROUP, NS = D / 32, NT = D / 16, TPG = GROUP / 16, SPG = GROUP / 32;
  const KvView &c = a.c;
  const int tid = threadIdx.x, lane = tid & 63, col = lane & 15, h = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  int id = blockIdx.x;
  const int kvh = id % c.heads;
  id /= c.heads;
  const int sp = id % a.splits;
  id /= a.splits;
  const int rt = id % a.row_tiles, b = id / a.row_tiles;
  const int shared = a.heads / c.heads, R = shared * a.q_len;
  const int len = __builtin_amdgcn_readfirstlane(min(max(a.lens[b], 0), a.max_len));
  const int r = min(rt * ROWS + col, R - 1);

  // what a row sees: keys [lo, hi)
  auto hi_of = [&](int row) { return max(len - a.q_len + row / shared + 1, 0); };
  auto lo_of = [&](int row) { return a.window > 0 ? max(0, len - a.q_len + row / shared + 1 - a.window) : 0; };
  const int r_first = rt * ROWS, r_last = min(rt * ROWS + ROWS, R) - 1;
  const int lo_min = lo_of(r_first), lo_max = lo_of(r_last), hi_min = hi_of(r_first), hi_max = hi_of(r_last);
  const int lo = lo_of(r), hi = hi_of(r);
  const int c_first = lo_min / CHUNK, chunks = max((hi_max + CHUNK - 1) / CHUNK - c_first, 0);
  const int per = (chunks + a.splits - 1) / a.splits;
  const int c0 = c_first + min(sp * per, chunks) + wv, c1 = c_first + min(sp * per + per, chunks);
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];

  // queries: step s takes channels 32s + 8h + j, a sixteenth of them where the
  // nibble pair is 16 times its code (j = 2, 3, 6, 7)
  const int token = b * a.q_len + r / shared, head = kvh * shared + r % shared;
  h8 qf[NS];
  float qsum[G];
  int qe;
  {
    const uint16_t *q = a.q + (int64_t)token * a.ldq + head * D + 8 * h;
    u4 raw[NS];
    uint32_t mx = 0;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      raw[s] = *(const u4 *)(q + 32 * s);
#pragma unroll
      for (int w = 0; w < 4; ++w) mx = pk_max_finite(mx, raw[s][w]);
    }
    const float top = row_max(fmaxf(lo_bf16(mx), hi_bf16(mx)));
    qe = top > 0.f ? 15 - __builtin_amdgcn_frexp_expf(top) : 0;
#pragma unroll
    for (int g = 0; g < G; ++g) qsum[g] = 0.f;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float x = ldexpf(lo_bf16(raw[s][w]), qe), y = ldexpf(hi_bf16(raw[s][w]), qe);
        qsum[s / SPG] += x + y;
        const float f = w & 1 ? 0.0625f : 1.f;
        qf[s][2 * w] = (_Float16)(x * f);
        qf[s][2 * w + 1] = (_Float16)(y * f);
      }
    }
#pragma unroll
    for (int g = 0; g < G; ++g) qsum[g] = row_sum(qsum[g]) * 0x1p-24f;
  }
  const float sc = a.scale * 1.44269504088896f;
  const int se = 24 - qe;

  f4 O[NT];
  float M[G], l = 0.f, m = -__FLT_MAX__;
  int E = -80;
#pragma unroll
  for (int t = 0; t < NT; ++t) O[t] = (f4){};
#pragma unroll
  for (int g = 0; g < G; ++g) M[g] = 0.f;

  // pages of 32 chunks of the wave at a time: lane 2i + j holds that of run j
  // of chunk i
  const int32_t *table = a.table + b * a.ld_table;
  int32_t pages = -1;
  auto load_pages = [&](int at) {
    const int ch = at + (lane >> 1) * CACHE_WAVES, key = ch * CHUNK + 16 * (lane & 1);
    pages = ch < c1 && key < hi_max ? table[key >> c.page_shift] : -1;
    asm volatile("" : "+v"(pages));  // waited for here, not at every use among the copies
  };
  // A wave copies its chunks into its own part of LDS, STAGES of them in
  // flight: per run of 16 keys the key words, the value runs and the
  // parameters of both, each one stretch of the page.
  constexpr int KB = 8 * D, PB = 64 * G, RUN = 2 * KB + 2 * PB;
  constexpr int COPIES = 2 * (2 * KB / 1024 + (2 * PB + 1023) / 1024);  // copies a chunk
  const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_t *)smem + wv * CACHE_STAGES * 2 * RUN;
  // the chunk in place i of the 32; bit j of the result: run j's page exists
  auto load = [&](int ch, int i, int stage) {
    int ok = 0;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int32_t page = __builtin_amdgcn_readlane(pages, 2 * i + j);
      const bool in = page >= 0 && page < c.pages;
      ok |= in ? 1 << j : 0;
      const int place = (ch * CHUNK + 16 * j) & ((1 << c.page_shift) - 1);
      const uint8_t *blk = kv_block(c, in ? page : 0, kvh);
      const uint32_t dst = lds0 + (stage * 2 + j) * RUN;
      const uint8_t *codes = blk + place * (D / 2), *par = blk + c.off_kp + place * (G * 4);
      if constexpr (D == 64) {
        copy_to_lds(codes, lane < 32 ? lane * 16 : c.off_v + (lane - 32) * 16, dst);
      } else {
#pragma unroll
        for (int n = 0; n < KB / 1024; ++n) {
          copy_to_lds(codes + n * 1024, lane * 16, dst + n * 1024);
          copy_to_lds(codes + c.off_v + n * 1024, lane * 16, dst + KB + n * 1024);
        }
      }
      if (lane < 2 * PB / 16)
        copy_to_lds(par, lane < PB / 16 ? lane * 16 : c.off_vp - c.off_kp + (lane - PB / 16) * 16, dst + 2 * KB);
    }
    return ok;
  };

  auto work = [&](uint32_t src, int k0, int ok, auto partial) {
    float t[2][4];
    bool seen[2][4];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      f4 A[G];
      uint32_t kw[NS];
#pragma unroll
      for (int s = 0; s < NS; ++s) kw[s] = lds_u32(src + j * RUN + lane * (4 * NS) + 4 * s);
#pragma unroll
      for (int g = 0; g < G; ++g) {
        A[g] = (f4){};
#pragma unroll
        for (int s = 0; s < SPG; ++s)
          A[g] = mfma_f16(nibbles(kw[g * SPG + s]), __builtin_bit_cast(u4, qf[g * SPG + s]), A[g]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) t[j][i] = 0.f;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const u4 kp = lds_u128(src + j * RUN + 2 * KB + (h * G + g) * 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) t[j][i] = fmaf(lo_bf16(kp[i]), A[g][i], fmaf(hi_bf16(kp[i]), qsum[g], t[j][i]));
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        t[j][i] = ldexpf(t[j][i] * sc, se);
        if constexpr (partial) {
          const int key = k0 + 16 * j + 4 * h + i;
          seen[j][i] = key >= lo && key < hi && (ok >> j & 1);
          t[j][i] = seen[j][i] ? t[j][i] : -__builtin_inff();
        } else {
          seen[j][i] = true;
        }
      }
    }
    auto rescale = [&](float f) {
      l *= f;
#pragma unroll
      for (int g = 0; g < G; ++g) M[g] *= f;
#pragma unroll
      for (int n = 0; n < NT; ++n) O[n] *= f;
    };
    float top = t[0][0];
#pragma unroll
    for (int i = 1; i < 8; ++i) top = fmaxf(top, t[i >> 2][i & 3]);
    if (__any(top > m + 6.f)) {
      const float now = fmaxf(m, row_max(top));
      rescale(__builtin_amdgcn_exp2f(m - now));
      m = now;
    }
    u4 vp[2][G];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int g = 0; g < G; ++g) {
        vp[j][g] = lds_u128(src + j * RUN + 2 * KB + PB + (h * G + g) * 16);
        if constexpr (partial) {
#pragma unroll
          for (int i = 0; i < 4; ++i) vp[j][g][i] = seen[j][i] ? vp[j][g][i] : 0u;
        }
      }
    float p[2][4], pm[G];
    u4 w[G], rest[G];
    auto weigh = [&]() {
      const float ref = m + (float)(E - 8);
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) p[j][i] = __builtin_amdgcn_exp2f(t[j][i] - ref);
      uint32_t most = 0;
      float far = 0.f;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        pm[g] = 0.f;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < 4; i += 2) {
            const uint32_t a0 = vp[j][g][i], a1 = vp[j][g][i + 1];
            const float w0 = p[j][i] * lo_bf16(a0), w1 = p[j][i + 1] * lo_bf16(a1);
            pm[g] = fmaf(p[j][i], hi_bf16(a0), pm[g]);
            pm[g] = fmaf(p[j][i + 1], hi_bf16(a1), pm[g]);
            const _Float16 h0 = (_Float16)w0, h1 = (_Float16)w1;
            const uint32_t hh = pk_f16(h0, h1);
            w[g][2 * j + (i >> 1)] = hh;
            rest[g][2 * j + (i >> 1)] = pk_f16((_Float16)(w0 - (float)h0), (_Float16)(w1 - (float)h1));
            most = pk_max_mag(most, hh);
          }
        far = fmaxf(far, fabsf(pm[g]));
      }
      return (most & 0xFFFF) >= 0x7C00 || most >= 0x7C000000u || far > 0x1p100f;
    };
    if (__any(weigh())) {
      // E from the greatest finite scale or minimum that a row sees here
      float big = 0.f;
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            big = fmaxf(big, fmaxf(finite_mag(lo_bf16(vp[j][g][i])), finite_mag(hi_bf16(vp[j][g][i]))));
      for (int d = 32; d; d >>= 1) big = fmaxf(big, __shfl_xor(big, d));
      const int now = __builtin_amdgcn_readfirstlane(big > 0.f ? __builtin_amdgcn_frexp_expf(big) : E);
      if (now > E) {
        rescale(ldexpf(1.f, E - now));
        E = now;
        weigh();
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) l += p[i >> 2][i & 3];
#pragma unroll
    for (int g = 0; g < G; ++g) M[g] += pm[g];
    uint32_t vw[2][NS];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int s = 0; s < NS; ++s) vw[j][s] = lds_u32(src + j * RUN + KB + lane * (4 * NS) + 4 * s);
    // value runs: dword w of a key holds tiles 8w .. 8w + 7 (at 64 channels
    // a half dword, two keys a dword)
#pragma unroll
    for (int n4 = 0; n4 < NT / 4; ++n4) {
      u4 v4;  // tiles 4 n4 .. 4 n4 + 3, key pairs of both runs
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if constexpr (D == 64) {
            v4[2 * j + e] = vw[j][e];
          } else {
            constexpr int W = D / 128;  // dwords of a key's run
            const uint32_t x0 = vw[j][2 * e * W + (n4 >> 1)], x1 = vw[j][(2 * e + 1) * W + (n4 >> 1)];
            v4[2 * j + e] = __builtin_amdgcn_perm(x1, x0, n4 & 1 ? 0x07060302u : 0x05040100u);
          }
        }
      const u4 v8 = v4 >> 8;
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const u4 f = (n & 2 ? v8 : v4) & (n & 1 ? 0x00F000F0u : 0x000F000Fu);
        const int g = (4 * n4 + n) / TPG;
        O[4 * n4 + n] = mfma_f16(f, w[g], O[4 * n4 + n]);
        O[4 * n4 + n] = mfma_f16(f, rest[g], O[4 * n4 + n]);
      }
    }
  };

  if (c0 < c1) {
    const int count = (c1 - c0 + CACHE_WAVES - 1) / CACHE_WAVES;
    load_pages(c0);
    int oks = 0;  // two bits a stage
    auto fetch = [&](int n) {
      if (n % 32 == 0 && n > 0) load_pages(c0 + n * CACHE_WAVES);
      const int stage = n % CACHE_STAGES;
      oks = (oks & ~(3 << 2 * stage)) | load(c0 + n * CACHE_WAVES, n % 32, stage) << 2 * stage;
    };
    for (int n = 0; n < CACHE_STAGES - 1 && n < count; ++n) fetch(n);
    for (int n = 0; n < count; ++n) {
      // the chunk's reads are over before its place is written again
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      if (n + CACHE_STAGES - 1 < count) {
        fetch(n + CACHE_STAGES - 1);
        wait_copies<(CACHE_STAGES - 1) * COPIES>();
      } else {
        wait_copies<0>();
      }
      const int stage = n % CACHE_STAGES, ok = oks >> 2 * stage & 3;
      const uint32_t src = lds0 + stage * 2 * RUN;
      const int k0 = (c0 + n * CACHE_WAVES) * CHUNK;
      if (ok == 3 && k0 >= lo_max && k0 + CHUNK <= hi_min) work(src, k0, ok, std::integral_constant<bool, false>());
      else work(src, k0, ok, std::integral_constant<bool, true>());
    }
  }
  __syncthreads();  // the waves' copies share their place with what follows

  // the waves meet in LDS: numerators [wave][row][D], then references and sums
  float *s_o = (float *)smem;
  float *s_ref = s_o + CACHE_WAVES * ROWS * (D + 4), *s_l = s_ref + CACHE_WAVES * ROWS;
  l = row_sum(l);
  float *mine = s_o + (wv * ROWS + col) * (D + 4);
#pragma unroll
  for (int g = 0; g < G; ++g) M[g] = row_sum(M[g]);
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const float f = n & 1 ? 0x1p20f : 0x1p24f;
    *(f4 *)(mine + 16 * n + 4 * h) = O[n] * f + M[n / TPG];
  }
  if (h == 0) {
    s_ref[wv * ROWS + col] = m + (float)(E - 8);
    s_l[wv * ROWS + col] = l;
  }
  __syncthreads();
  const int row = tid >> 4, part = tid & 15;  // 16 threads a row, D / 16 channels each
  if (rt * ROWS + row >= R) return;
  float ref = -__FLT_MAX__, sum = 0.f, f[CACHE_WAVES];
#pragma unroll
  for (int w = 0; w < CACHE_WAVES; ++w)
    if (s_l[w * ROWS + row] != 0.f) ref = fmaxf(ref, s_ref[w * ROWS + row]);
#pragma unroll
  for (int w = 0; w < CACHE_WAVES; ++w) {
    const float lw = s_l[w * ROWS + row];
    f[w] = lw != 0.f ? __builtin_amdgcn_exp2f(s_ref[w * ROWS + row] - ref) : 0.f;
    sum += lw * f[w];
  }
  f4 out[D / 64];
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    out[i] = (f4){};
#pragma unroll
    for (int w = 0; w < CACHE_WAVES; ++w)
      if (f[w] != 0.f) out[i] += *(const f4 *)(s_o + (w * ROWS + row) * (D + 4) + 64 * i + 4 * part) * f[w];
  }
  const int q_row = rt * ROWS + row;
  if (a.splits == 1) {
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    uint16_t *y = a.y + (int64_t)(b * a.q_len + q_row / shared) * a.ldy + (kvh * shared + q_row % shared) * D;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      const f4 o = out[i] * inv;
      *(u2 *)(y + 64 * i + 4 * part) =
          (u2){(uint32_t)f32_to_bf16_bits(o[0]) | (uint32_t)f32_to_bf16_bits(o[1]) << 16,
               (uint32_t)f32_to_bf16_bits(o[2]) | (uint32_t)f32_to_bf16_bits(o[3]) << 16};
    }
    return;
  }
  const int64_t at = (((int64_t)b * c.heads + kvh) * R + q_row) * a.splits + sp;
#pragma unroll
  for (int i = 0; i < D / 64; ++i) *(f4 *)(a.part + at * D + 64 * i + 4 * part) = out[i];
  if (part == 0) *(float2 *)(a.sums + 2 * at) = make_float2(ref, sum);
}

// Joins the key ranges of a row: a block a row, D / 4 threads a range, four
// channels a thread.
template <int D>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnCacheArgs a) {
  constexpr int T = D / 4, N = 256 / T;
  __shared__ f4 s_o[N][T];
  __shared__ float s_l[N];
  const int tid = threadIdx.x, lane = tid & 63, part = tid % T, first = tid / T;
  const int shared = a.heads / a.c.heads, R = shared * a.q_len;
  const int64_t at = blockIdx.x;
  const float2 *sums = (const float2 *)a.sums + at * a.splits;
  float ref = -__FLT_MAX__;
  for (int s = lane; s < a.splits; s += 64)
    if (sums[s].y != 0.f) ref = fmaxf(ref, sums[s].x);
  for (int d = 32; d; d >>= 1) ref = fmaxf(ref, __shfl_xor(ref, d));
  float sum = 0.f;
  f4 o = {};
  const f4 *num = (const f4 *)(a.part + at * a.splits * D) + part;
#pragma unroll 4
  for (int s = first; s < a.splits; s += N) {
    const float2 x = sums[s];
    const f4 v = num[(int64_t)s * T];
    const float f = x.y != 0.f ? __builtin_amdgcn_exp2f(x.x - ref) : 0.f;
    sum += x.y * f;
    o += v * f;  // a range without keys has left zeros
  }
  s_o[first][part] = o;
  if (part == 0) s_l[first] = sum;
  __syncthreads();
  if (tid >= T) return;
  for (int n = 1; n < N; ++n) {
    o += s_o[n][part];
    sum += s_l[n];
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int q_row = (int)(at % R), kvh = (int)(at / R % a.c.heads);
  const int64_t b = at / R / a.c.heads;
  uint16_t *y = a.y + (b * a.q_len + q_row / shared) * a.ldy + (kvh * shared + q_row % shared) * D + 4 * part;
  o *= inv;
  *(u2 *)y = (u2){(uint32_t)f32_to_bf16_bits(o[0]) | (uint32_t)f32_to_bf16_bits(o[1]) << 16,
                  (uint32_t)f32_to_bf16_bits(o[2]) | (uint32_t)f32_to_bf16_bits(o[3]) << 16};
}

template <int D, int GROUP>
hipError_t launch_cache(const AttnCacheArgs &a, hipStream_t s) {
  constexpr int G = D / GROUP, copies = CACHE_STAGES * 2 * (16 * D + 128 * G), joined = ROWS * (D + 6) * 4;
  constexpr size_t lds = (size_t)CACHE_WAVES * (copies > joined ? copies : joined);
  const hipError_t e = allow_smem(attn_cache_kernel<D, GROUP>, lds);
  if (e != hipSuccess) return e;
  const int64_t blocks = (int64_t)a.batch * a.row_tiles * a.splits * a.c.heads;
  attn_cache_kernel<D, GROUP><<<dim3((unsigned)blocks), 64 * CACHE_WAVES, lds, s>>>(a);
  if (a.splits > 1) {
    const int64_t rows = (int64_t)a.batch * a.heads * a.q_len;
    attn_join_kernel<D><<<dim3((unsigned)rows), 256, 0, s>>>(a);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_write(const KvWriteArgs &a, hipStream_t s) {
  const dim3 grid((unsigned)((a.tokens + 15) / 16), a.c.heads);
  switch (a.c.dim) {
    case 64:
      kv_write_kernel<64, 0><<<grid, 256, 0, s>>>(a);
      kv_write_kernel<64, 1><<<grid, 256, 0, s>>>(a);
      break;
    case 128:
      kv_write_kernel<128, 0><<<grid, 256, 0, s>>>(a);
      kv_write_kernel<128, 1><<<grid, 256, 0, s>>>(a);
      break;
    default:
      kv_write_kernel<256, 0><<<grid, 256, 0, s>>>(a);
      kv_write_kernel<256, 1><<<grid, 256, 0, s>>>(a);
  }
  return hipGetLastError();
}

hipError_t launch_kv_read(const KvReadArgs &a, hipStream_t s) {
  const dim3 grid((unsigned)((a.tokens + 15) / 16), a.c.heads);
  switch (a.c.dim) {
    case 64:
      kv_read_kernel<64, 0><<<grid, 256, 0, s>>>(a);
      kv_read_kernel<64, 1><<<grid, 256, 0, s>>>(a);
      break;
    case 128:
      kv_read_kernel<128, 0><<<grid, 256, 0, s>>>(a);
      kv_read_kernel<128, 1><<<grid, 256, 0, s>>>(a);
      break;
    default:
      kv_read_kernel<256, 0><<<grid, 256, 0, s>>>(a);
      kv_read_kernel<256, 1><<<grid, 256, 0, s>>>(a);
  }
  return hipGetLastError();
}

hipError_t launch_attn_cache(const AttnCacheArgs &a, hipStream_t s) {
  const int group = 1 << a.c.group_shift;
  switch (a.c.dim) {
    case 64: return group == 32 ? launch_cache<64, 32>(a, s) : launch_cache<64, 64>(a, s);
    case 128:
      return group == 32   ? launch_cache<128, 32>(a, s)
             : group == 64 ? launch_cache<128, 64>(a, s)
                           : launch_cache<128, 128>(a, s);
    default:
      return group == 32   ? launch_cache<256, 32>(a, s)
             : group == 64 ? launch_cache<256, 64>(a, s)
                           : launch_cache<256, 128>(a, s);
  }
}

}  // namespace svq
