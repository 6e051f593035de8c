// The 4-bit cache of keys and values (include/svq_attn.h): quantising tokens
// into it, reading them back, attention over it.
#include <type_traits>

#include "svq_attn.h"
#include "svq_device.h"

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
  bool plain;     // a normal scale, and differences that fp32 holds
};
// The parameters of a group of greatest value hi and least value -nlo.  A NaN
// among its values has made hi infinite.
__device__ __forceinline__ KvScale kv_scale(float hi, float nlo) {
  KvScale p;
  if (!(hi < __builtin_inff()) || !(nlo < __builtin_inff())) {
    p.s = p.m = p.r = 0.f;
    p.bits = 0x7FC07FC0u;
    p.plain = false;
    return p;
  }
  p.m = -nlo;
  // The product with 1/15 is off from the quotient by a step of 64 bits, and
  // rounds to the same fp32 number: a difference of two 8-bit numbers is 15
  // times the midpoint of two fp32 numbers, whose quotient is exact to 2^-52, or
  // further than that from it.
  const uint32_t sb = f32_to_bf16_bits((float)(((double)hi - (double)p.m) * (1.0 / 15.0)));
  p.s = bf16_bits_to_f32(sb);
  p.r = __builtin_amdgcn_rcpf(p.s);
  p.plain = p.s >= 0x1p-126f && hi + nlo < __builtin_inff();
  p.bits = sb | (__builtin_bit_cast(uint32_t, p.m) & 0xFFFF0000u);
  return p;
}
// Codes of N values, the nearest whole numbers to (x - m) / s (of two as near
// the even one), two to a dword: of x[i] in the lower half, of x[i + N / 2]
// (STEP 8) or x[i + 1] in the upper one, each plus KV_CODE0.  The fp32 quotient
// of a plain group is off by less than 4e-6 and less than 15.1; a sum with 192 +
// 1/2 + 2^-16 has the code in its upper half and, in the lower one, 2^16 times
// what the quotient is beyond the border below it plus one, rounded.
constexpr uint32_t KV_CODE0 = 0x43404340u;
// A value at a border, its lower half 0 or 1, is held against it: x - m is d and
// a rest, and d less the border (n - 1/2) s an fp32 number, a multiple of d's
// last place and not greater than d.  (Borders are met often, all numbers being
// 8-bit ones times powers of two.)  Where d is on the border and has a rest, or
// the group is not plain, 64 bits decide, in which the difference of two bf16
// values 2^45 apart and less is exact.
template <int N, int STEP>
__device__ __forceinline__ void kv_codes(const float (&x)[N], const KvScale &p, uint32_t (&code)[N / 2]) {
  uint32_t u[N];
  bool wide = !p.plain;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float d = x[i] - p.m;
    u[i] = __builtin_bit_cast(uint32_t, fmaf(d, p.r, 192.5f + 0x1p-16f));
    if ((uint16_t)u[i] < 2) {
      const float off = fmaf(192.5f - floorf(__builtin_bit_cast(float, u[i])), p.s, d), y = d - x[i];
      wide = wide || (off == 0.f && (x[i] - (d - y)) - (p.m + y) != 0.f);
      if (off < 0.f || (off == 0.f && (u[i] & 0x10000u))) u[i] -= 0x10000u;  // to the even one
    }
  }
  if (__builtin_expect(wide, 0)) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const double q = p.s == 0.f ? 0. : fmin(rint(((double)x[i] - (double)p.m) / (double)p.s), 15.);
      u[i] = ((uint32_t)q << 16) + (KV_CODE0 & 0xFFFF0000u);
    }
  }
#pragma unroll
  for (int i = 0; i < N / 2; ++i) code[i] = STEP == 1 ? __builtin_amdgcn_perm(u[2 * i + 1], u[2 * i], 0x07060302u) : __builtin_amdgcn_perm(u[i + N / 2], u[i], 0x07060302u);
}
// A key word of eight codes: pair i at nibble i of both halves.
__device__ __forceinline__ uint32_t kv_word(const uint32_t (&c)[4]) {
  return (((((c[3] << 4) + c[2]) << 4) + c[1]) << 4) + c[0] - KV_CODE0 * 0x1111u;
}

typedef __bf16 b2 __attribute__((ext_vector_type(2)));
typedef float f2 __attribute__((ext_vector_type(2)));
typedef double d4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ uint32_t pk_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2){a, b}, b2));
}
__device__ __forceinline__ float lo_bf16(uint32_t p) { return bf16_bits_to_f32(p & 0xFFFFu); }
__device__ __forceinline__ float hi_bf16(uint32_t p) { return __builtin_bit_cast(float, p & 0xFFFF0000u); }

// v of the lane 32 (16) lanes away beside the lane's own, over the lanes that
// share lane % 16: maximum, sum.
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

// v, with no part of what is made of it moved ahead of the branch it stands in.
__device__ __forceinline__ uint32_t hidden(uint32_t v) {
  asm volatile("" : "+v"(v));
  return v;
}

// Lanes of the key side: token lane % 16 of the wave's 16, channels 32c + 8h ..
// 32c + 8h + 7 of every step c with h = i = lane / 16, so that a lane's codes
// are one piece of the layout and the wave's 16 tokens one stretch.  Lanes of
// the value side: D / 16 a token, lane i the 16 channels of tile i.  blockIdx.y
// is the head, blockIdx.z the side; tokens come first (heads first, so that the
// blocks of a row run together: 32768 tokens written in 70 us against 68, read
// in 53 against 50).
struct KvPlace {
  int64_t t;     // token
  int32_t slot;  // of the cache, or one that is not there
  int i;
};
template <int D>
__device__ __forceinline__ KvPlace kv_place(const int32_t *slots, int64_t tokens, int side) {
  constexpr int T = D / 16;
  const int lane = threadIdx.x & 63;
  const int64_t wave = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  KvPlace p;
  p.t = side ? wave * (64 / T) + lane / T : wave * 16 + (lane & 15);
  p.i = side ? lane % T : lane >> 4;
  p.slot = p.t < tokens ? slots[p.t] : -1;
  return p;
}
// Whether the token has a place: asked for after the loads that do not need it,
// which then are on their way with the slot.
__device__ __forceinline__ bool kv_in(const KvView &c, KvPlace &p) {
  asm volatile("" : "+v"(p.slot)::"memory");
  return p.slot >= 0 && p.slot < c.pages << c.page_shift;
}

// An exchange with the lane whose number differs in its lowest bits: 7 - i, and
// the two quad forms.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}
// Half the words of `w` (N of them) from the lane across, or-ed to the lane's
// own: `upper` lanes keep the upper half.
template <int CTRL, int N>
__device__ __forceinline__ void or_half(uint32_t *w, bool upper) {
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    const uint32_t mine = upper ? w[i + N / 2] : w[i], other = upper ? w[i] : w[i + N / 2];
    w[i] = mine | dpp<CTRL>(other);
  }
}

// One pass: a value is read once and leaves as a nibble.  Bound by instructions,
// about 20 a value, a third of them extremes, exchanges and the parameters in 64
// bits, and by those of waves without a token: a block takes 64 tokens of the key
// side but 4096 / D of the value side, whose number the grid has for both, so at
// 128 channels every second block of the key side, at 256 three of four, do all
// of it for the last token and store nothing (a third and three fifths of the
// instructions).  The registers are held to what lets 8 waves a SIMD run, 5 at 256
// channels, where 4 and 6 take 71 and 66 us against 63 (chosen with those waves).
// 32768 tokens of 8 heads of 128 channels 45 us, 3.8 TB/s read and written, where
// a copy of as many bytes takes 35.
template <int D>
__global__ __launch_bounds__(256, D == 256 ? 5 : 8) void kv_write_kernel(KvWriteArgs a) {
  constexpr int NS = D / 32;
  const int head = blockIdx.y, side = blockIdx.z;
  KvPlace P = kv_place<D>(a.slots, a.tokens, side);
  const int64_t t = min(P.t, a.tokens - 1);
  if (side == 0) {
    const uint16_t *src = a.k + t * a.ldk + head * D + 8 * P.i;
    u4 raw[NS];
#pragma unroll
    for (int s = 0; s < NS; ++s) raw[s] = *(const u4 *)(src + 32 * s);
    const bool in = kv_in(a.c, P);
    uint8_t *blk = kv_block(a.c, in ? P.slot >> a.c.page_shift : 0, head);
    const int place = P.slot & ((1 << a.c.page_shift) - 1);
    float hi[NS], nlo[NS];
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      uint32_t mag = 0;
      hi[s] = nlo[s] = -__builtin_inff();
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float u = lo_bf16(raw[s][w]), v = hi_bf16(raw[s][w]);
        mag = pk_max_mag(mag, raw[s][w]);
        hi[s] = fmaxf(fmaxf(hi[s], u), v);
        nlo[s] = fmaxf(fmaxf(nlo[s], -u), -v);
      }
      if ((mag & 0xFFFF) >= 0x7F80 || mag >= 0x7F800000u) hi[s] = __builtin_inff();  // not finite
    }
    const int steps = 1 << (a.c.group_shift - 5);  // of a group: 1, 2 or 4
    uint32_t word[NS];
    KvScale p;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      if (s % steps == 0) {
        float h = hi[s], l = nlo[s];
#pragma unroll
        for (int e = 1; e < 4; ++e)
          if (e < steps && s + e < NS) {
            h = fmaxf(h, hi[s + e < NS ? s + e : s]);
            l = fmaxf(l, nlo[s + e < NS ? s + e : s]);
          }
        p = kv_scale(row_max(h), row_max(l));
        if (in && P.i == 0) *(uint32_t *)(blk + kv_param(a.c, 0, place, s / steps)) = p.bits;
      }
      float x[8];
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t pair = hidden(raw[s][w]);  // taken apart again: all at once they would fill the registers
        x[2 * w] = lo_bf16(pair);
        x[2 * w + 1] = hi_bf16(pair);
      }
      uint32_t code[4];
      kv_codes<8, 1>(x, p, code);
      word[s] = kv_word(code);  // channel j at nibble kv_nibble(j)
    }
    if (in) __builtin_memcpy(__builtin_assume_aligned(blk + kv_key_word(a.c, place, P.i), D == 64 ? 8 : 16), word, sizeof(word));
  } else {
    // a lane has the 16 channels of tile i
    const u4 *src = (const u4 *)(a.v + t * a.ldv + head * D + 16 * P.i);
    float x[16], hi = -__builtin_inff(), nlo = hi;
    uint32_t mag = 0;
    const u4 raw[2] = {src[0], src[1]};
    const bool in = kv_in(a.c, P);  // of all lanes of a token
    uint8_t *blk = kv_block(a.c, in ? P.slot >> a.c.page_shift : 0, head);
    const int place = P.slot & ((1 << a.c.page_shift) - 1);
#pragma unroll
    for (int n = 0; n < 2; ++n) {
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float u = lo_bf16(raw[n][w]), v = hi_bf16(raw[n][w]);
        mag = pk_max_mag(mag, raw[n][w]);
        hi = fmaxf(fmaxf(hi, u), v);
        nlo = fmaxf(fmaxf(nlo, -u), -v);
        x[8 * n + 2 * w] = u;
        x[8 * n + 2 * w + 1] = v;
      }
    }
    if ((mag & 0xFFFF) >= 0x7F80 || mag >= 0x7F800000u) hi = __builtin_inff();  // not finite
    const int tiles = 1 << (a.c.group_shift - 4);  // of a group: 2, 4 or 8
    const KvScale p = kv_scale(lanes_max(hi, tiles), lanes_max(nlo, tiles));
    if (in && P.i % tiles == 0) *(uint32_t *)(blk + kv_param(a.c, 1, place, P.i / tiles)) = p.bits;
    uint32_t w[8];  // codes of runs r and r + 8
    kv_codes<16, 8>(x, p, w);
    // Lane i has nibble i of every run.  Exchanges among eight lanes (four with
    // 64 channels) leave whole dwords (half dwords).
    const int n = P.i & 7;
    if constexpr (D > 64) {
      // Lanes n and 7 - n: the lower takes runs 0 .. 7 of both, the upper the
      // rest, a code in either half of a dword, then each half shifted to its
      // nibble.
      const int e = n & 4 ? 7 - n : n;
      const uint32_t halves = n & 4 ? 0x03020706u : 0x05040100u;
      const us2_t shift = {(uint16_t)(4 * e), (uint16_t)(12 - 4 * e)};
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const uint32_t mine = w[r] - KV_CODE0;
        w[r] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(us2_t, __builtin_amdgcn_perm(dpp<0x141>(mine), mine, halves)) << shift);
      }
      or_half<0x4E, 8>(w, n & 2);    // lane n ^ 2
      or_half<0xB1, 4>(w, n & 1);    // lane n ^ 1
      if (!in) return;
      const int run = (n & 4 ? 8 : 0) + (n & 2 ? 4 : 0) + (n & 1 ? 2 : 0);
#pragma unroll
      for (int e = 0; e < 2; ++e) *(uint32_t *)(blk + kv_value_run(a.c, place, run + e) + 4 * (P.i >> 3)) = w[e];
    } else {
#pragma unroll
      for (int r = 0; r < 8; ++r) w[r] = (w[r] - KV_CODE0) << 4 * n;
      or_half<0x4E, 8>(w, n & 2);
      or_half<0xB1, 4>(w, n & 1);
      if (!in) return;
      const int run = (n & 2 ? 4 : 0) + (n & 1 ? 2 : 0);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        *(uint16_t *)(blk + kv_value_run(a.c, place, run + e)) = (uint16_t)w[e];
        *(uint16_t *)(blk + kv_value_run(a.c, place, run + e + 8)) = (uint16_t)(w[e] >> 16);
      }
    }
  }
}

// The other way, of the same lanes; bound by its writes (32768 tokens of 8 heads
// of 128 channels to bf16 48.7 us, 2.8 TB/s written, where a large copy writes
// 2.4; past the caches, as streams, 2048 tokens take 18 us instead of 14) and by
// latency where tokens are few (777 tokens 4.4 us).
template <int D>
__global__ __launch_bounds__(256) void kv_read_kernel(KvReadArgs a) {
  constexpr int NS = D / 32;
  const int head = blockIdx.y, side = blockIdx.z;
  KvPlace P = kv_place<D>(a.slots, a.tokens, side);
  const bool in = kv_in(a.c, P);
  const uint8_t *blk = kv_block(a.c, in ? P.slot >> a.c.page_shift : 0, head);
  const int place = in ? P.slot & ((1 << a.c.page_shift) - 1) : 0;
  // eight values from element `at` on
  auto store = [&](void *out, int64_t at, const float (&x)[8]) {
    if (a.f32) {
      f4 *y = (f4 *)((float *)out + at);
      y[0] = (f4){x[0], x[1], x[2], x[3]};
      y[1] = (f4){x[4], x[5], x[6], x[7]};
    } else {
      u4 y;
#pragma unroll
      for (int w = 0; w < 4; ++w) y[w] = pk_bf16(x[2 * w], x[2 * w + 1]);
      *(u4 *)((uint16_t *)out + at) = y;
    }
  };
  // the parameters of a slot that is not there are zeros, and so its values
  auto param = [&](int s, int g) { return in ? *(const uint32_t *)(blk + kv_param(a.c, s, place, g)) : 0u; };
  auto value = [&](uint32_t p, uint32_t code) { return fmaf((float)code, lo_bf16(p), hi_bf16(p)); };
  if (side == 0) {
    if (P.t >= a.tokens) return;
    uint32_t word[NS];
    __builtin_memcpy(word, __builtin_assume_aligned(blk + kv_key_word(a.c, place, P.i), D == 64 ? 8 : 16), sizeof(word));
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const uint32_t p = param(0, s >> (a.c.group_shift - 5));
      // nibble n in byte n / 2 of one of two words: a conversion each
      const uint32_t nibbles[2] = {word[s] & 0x0F0F0F0Fu, word[s] >> 4 & 0x0F0F0F0Fu};
      float x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = value(p, nibbles[kv_nibble(j) & 1] >> 8 * (kv_nibble(j) >> 1) & 255);
      store(a.k, P.t * a.ldk + head * D + 32 * s + 8 * P.i, x);
    }
  } else {
    // the lanes of a token bring two (four of 64 channels) runs each and hand
    // them round: lane i takes nibble i of every run
    constexpr int T = D / 16, PER = 16 / (T < 8 ? T : 8);
    const int n = P.i & 7, first = (threadIdx.x & 63) - n;  // of the token's lanes, by dword of a run
    uint32_t own[PER];
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      const uint8_t *run = blk + kv_value_run(a.c, place, n * PER + e);
      own[e] = D == 64 ? *(const uint16_t *)run : *(const uint32_t *)(run + 4 * (P.i >> 3));
    }
    const uint32_t p = param(1, P.i >> (a.c.group_shift - 4));
    float x[2][8];
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const uint32_t w = (uint32_t)__shfl((int)own[r % PER], first + r / PER);
      x[r >> 3][r & 7] = value(p, w >> 4 * n & 15);
    }
    if (P.t >= a.tokens) return;
#pragma unroll
    for (int e = 0; e < 2; ++e) store(a.v, P.t * a.ldv + head * D + 16 * P.i + 8 * e, x[e]);
  }
}

// ---- attention over the cache -------------------------------------------
//
// A block takes 16 rows (query token t of q_len, query head g of the G that
// share a key head: row t * G + g) of one sequence and key head, and one of
// `splits` ranges of its keys; a wave every fourth chunk of 32 keys in it.
// Codes enter the matrix cores as they are: a nibble brought to bits 4 .. 7 of a
// half is a subnormal fp16 number, 16 c * 2^-24, which v_mfma_f32_16x16x32_f16
// multiplies exactly.  It adds 32 products at the greatest exponent of their
// operands, to about 2^-24.5 of it, and takes a subnormal for 2^-14: a code in
// bits 4 .. 7 is short of that by 2 bits, and a product kept within 2^-22 of the
// greatest code times the greatest weight; one in bits 0 .. 3, a shift less for
// half of the codes (2 % of the time), by 6 and within 2^-18.  So, transposed (a
// lane holds one row, and four keys of each 16):
//
//   A_g[key][row] = sum over the group's channels of c * q     (q in fp16
//        under a power-of-two scale per row, per group where a row's channels
//        need it)
//   score         = sum over groups of s_g A_g + m_g sum q     (fp32)
//   O_t[channel][row] += sum over keys of c * (p s_g)          (p s_g in units
//        of 2^(E - 8) as the sum of two fp16 numbers, 22 bits: the minimum's
//        term below cancels much of this one, and with 11 bits a value near
//        zero would carry the rounding of its whole range)
//   M_g[row]          += sum over keys of p m_g                (fp32, in the same units)
//
// and the row is 2^(E - 8) (2^20 O + M) / sum p.  The weight p is exp2 of (score
// - m) times the scale: m a running maximum, raised once a weight exceeds 2^6, E
// the exponent of the greatest scale or minimum that the row sees in a wave's
// first chunk, raised once a p s_g overflows fp16.  The two are kept apart: in
// one fp32 number a maximum from 2^24 on would round E away.
//
// What bounds it: vector instructions, which take 90 % of the cycles at 64
// sequences of up to 8192 tokens (77 us, 4.0 TB/s of the cache, 64 us at the
// rate of a copy): 16 rows are what one product takes, so the codes of a key are
// unpacked once for up to 16 query heads, and the weights (12 instructions a
// pair and group) cost more than the codes.  A wave's chunks reach LDS by
// copies one chunk ahead (into registers instead: 110 us); three stages gain
// nothing.  Short contexts are latency: one sequence of 777 tokens 8.5 us, of
// it 6 this launch (the length, the page, the first chunk, code that is not
// in the instruction cache yet) and 2.3 the join.  More waves a block (8) or
// more and shorter ranges cost what they gain.
constexpr int CACHE_WAVES = 4, CACHE_STAGES = 2, CHUNK = 32, ROWS = 16;

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
// v as one value to all that use it.
__device__ __forceinline__ h2 once(h2 v) {
  asm("" : "+v"(v));
  return v;
}
typedef __attribute__((address_space(3))) uint8_t lds_t;
typedef __attribute__((address_space(3))) uint32_t lds_u32;
// LDS bytes of a block: the waves' stages of chunks, whose place what they bring
// together takes after the last, and 8 bytes a wave and row for the powers of
// two of its query's groups.
template <int D, int G>
constexpr uint32_t cache_lds() {
  constexpr int copies = CACHE_STAGES * 2 * (16 * D + 128 * G), joined = ROWS * (D + 7) * 4;
  return CACHE_WAVES * ((copies > joined ? copies : joined) + ROWS * 8);
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

// A key word's 8 channels as fp16 pairs (see kv_nibble).
__device__ __forceinline__ u4 nibbles(uint32_t w) {
  return (u4){w << 4 & 0x00F000F0u, w & 0x00F000F0u, w >> 4 & 0x00F000F0u, w >> 8 & 0x00F000F0u};
}

__device__ __forceinline__ f4 mfma_f16(const u4 &a, const u4 &b, const f4 &c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, a), __builtin_bit_cast(h8, b), c, 0, 0, 0);
}
__device__ __forceinline__ u2 row_bf16(const f4 &v) { return (u2){pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3])}; }
// The dwords of lane-consecutive pieces of N dwords.
template <int N>
__device__ __forceinline__ void lds_words(uint32_t at, uint32_t (&w)[N]) {
  if constexpr (N == 2) {
    const u2 x = *(const __attribute__((address_space(3))) u2 *)(lds_t *)(uintptr_t)at;
    w[0] = x[0];
    w[1] = x[1];
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const u4 x = lds_u128(at + 4 * i);
#pragma unroll
      for (int e = 0; e < 4; ++e) w[i + e] = x[e];
    }
  }
}

// Whether the greater magnitudes of two halves (pk_max_mag) are not finite.
__device__ __forceinline__ bool not_finite(uint32_t mag) { return (mag & 0xFFFF) >= 0x7F80 || mag >= 0x7F800000u; }

template <int D, int GROUP>
__global__ __launch_bounds__(64 * CACHE_WAVES, D / GROUP == 8 ? 1 : 2) void attn_cache_kernel(AttnCacheArgs a) {
  constexpr int G = D / GROUP, NS = D / 32, NT = D / 16, TPG = GROUP / 16, SPG = GROUP / 32;
  const KvView &c = a.c;
  const int tid = threadIdx.x, lane = tid & 63, col = lane & 15, h = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int kvh = blockIdx.x, b = blockIdx.z;
  int sp = blockIdx.y, rt = 0;
  if (a.row_tiles > 1) {
    rt = sp / a.splits;
    sp -= rt * a.splits;
  }
  const int shared = a.heads / c.heads, R = shared * a.q_len;
  // row r: query token r / shared, query head r % shared
  const int r = min(rt * ROWS + col, R - 1), r_token = a.q_len > 1 ? r / shared : 0;
  const int len = __builtin_amdgcn_readfirstlane(min(max(a.lens[b], 0), a.max_len));
  u4 raw[NS];
  {
    const uint16_t *q = a.q + (int64_t)(b * a.q_len + r_token) * a.ldq + (kvh * shared + r - r_token * shared) * D + 8 * h;
#pragma unroll
    for (int s = 0; s < NS; ++s) raw[s] = *(const u4 *)(q + 32 * s);
  }

  // what a row sees: keys [lo, hi); the greatest and least of the tile's rows
  const int first = len - a.q_len + 1;
  const int t_first = a.q_len > 1 ? rt * ROWS / shared : 0, t_last = a.q_len > 1 ? (min(rt * ROWS + ROWS, R) - 1) / shared : 0;
  auto hi_of = [&](int token) { return max(first + token, 0); };
  auto lo_of = [&](int token) { return a.window > 0 ? max(0, first + token - a.window) : 0; };
  const int lo_min = lo_of(t_first), lo_max = lo_of(t_last), hi_min = hi_of(t_first), hi_max = hi_of(t_last);
  const int c_first = lo_min / CHUNK, chunks = max((hi_max + CHUNK - 1) / CHUNK - c_first, 0);
  const int per = a.splits > 1 ? (chunks + a.splits - 1) / a.splits : chunks;
  const int c0 = c_first + min(sp * per, chunks) + wv, c1 = c_first + min(sp * per + per, chunks);
  const int count = c0 < c1 ? (c1 - c0 + CACHE_WAVES - 1) / CACHE_WAVES : 0;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];

  // pages of 32 chunks of the wave at a time: lane 2i + j holds that of run j
  // of chunk i
  const int32_t *table = a.table + b * a.ld_table;
  int32_t pages = -1;
  auto load_pages = [&](int n) {
    const int ch = c0 + (n + (lane >> 1)) * CACHE_WAVES, key = ch * CHUNK + 16 * (lane & 1);
    pages = ch < c1 && key < hi_max ? table[key >> c.page_shift] : -1;
    asm volatile("" : "+v"(pages));  // waited for here, not at every use among the copies
  };
  // A wave copies its chunks into its own part of LDS, CACHE_STAGES of them in
  // flight: per run of 16 keys the key words, the value runs and the
  // parameters of both, each one stretch of the page.
  constexpr int KB = 8 * D, PB = 64 * G, RUN = 2 * KB + 2 * PB;
  constexpr int COPIES = 2 * (2 * KB / 1024 + (2 * PB + 1023) / 1024);  // copies a chunk
  const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_t *)smem + wv * CACHE_STAGES * 2 * RUN;
  const uint32_t code_off = D == 64 && lane >= 32 ? c.off_v + (lane - 32) * 16 : lane * 16;
  const uint32_t par_off = lane < PB / 16 ? lane * 16 : c.off_vp - c.off_kp + (lane - PB / 16) * 16;
  int oks = 0;  // two bits a stage: which runs' pages exist
  auto fetch = [&](int n) {
    if (n % 32 == 0 && n > 0) load_pages(n);
    const int stage = n % CACHE_STAGES, ch = c0 + n * CACHE_WAVES;
    int ok = 0;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int32_t page = __builtin_amdgcn_readlane(pages, 2 * (n % 32) + j);
      const bool in = page >= 0 && page < c.pages;
      ok |= in ? 1 << j : 0;
      const int place = (ch * CHUNK + 16 * j) & ((1 << c.page_shift) - 1);
      const uint8_t *blk = kv_block(c, in ? page : 0, kvh);
      const uint32_t dst = lds0 + (stage * 2 + j) * RUN;
      const uint8_t *codes = blk + place * (D / 2), *par = blk + c.off_kp + place * (G * 4);
      if constexpr (D == 64) {
        copy_to_lds(codes, code_off, dst);
      } else {
#pragma unroll
        for (int i = 0; i < KB / 1024; ++i) {
          copy_to_lds(codes + i * 1024, code_off, dst + i * 1024);
          copy_to_lds(codes + c.off_v + i * 1024, code_off, dst + KB + i * 1024);
        }
      }
      if (lane < 2 * PB / 16) copy_to_lds(par, par_off, dst + 2 * KB);
    }
    oks = (oks & ~(3 << 2 * stage)) | ok << 2 * stage;
  };
  if (count > 0) load_pages(0);
#pragma unroll
  for (int s = 0; s < NS; ++s) asm volatile("" : "+v"(raw[s]));  // arrived; not waited for behind the copies
#pragma unroll
  for (int n = 0; n < CACHE_STAGES - 1; ++n)
    if (n < count) fetch(n);

  // Queries: step s takes channels 32s + 8h + j, a sixteenth of them (for the 16
  // c), so all bits of a channel down to 2^-28 of the row's greatest.  A row with a
  // smaller one takes a further power of two for each group from its own greatest;
  // the group's products are divided by it again, from LDS, for want of registers.
  u4 qf[NS];
  float qsum[G];
  const uint32_t drops = (uint32_t)(uintptr_t)(lds_t *)smem + cache_lds<D, G>() - CACHE_WAVES * ROWS * 8 + (wv * ROWS + col) * 8;
  uint32_t drop[(G + 3) / 4];
  bool any_drop = false;
  uint32_t mx = 0;
#pragma unroll
  for (int s = 0; s < NS; ++s)
#pragma unroll
    for (int w = 0; w < 4; ++w) mx = pk_max_mag(mx, raw[s][w]);
  if (__builtin_expect(__any(not_finite(mx)), 0)) {
    mx = 0;
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
      for (int w = 0; w < 4; ++w) mx = pk_max_finite(mx, raw[s][w]);
  }
  const uint32_t flip = a.scale < 0.f ? 0x80008000u : 0u;
  const float q_top = row_max(fmaxf(lo_bf16(mx), hi_bf16(mx)));
  const int qe = q_top > 0.f ? 15 - __builtin_amdgcn_frexp_expf(q_top) : 0;
#pragma unroll
  for (int g = 0; g < (G + 3) / 4; ++g) drop[g] = 0;
  if constexpr (G > 1) {
    us2_t least = {0xFFFF, 0xFFFF};  // a magnitude's bits less one, zeros on top
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
      for (int w = 0; w < 4; ++w)
        least = __builtin_elementwise_min(least, __builtin_bit_cast(us2_t, raw[s][w] & 0x7FFF7FFFu) - (us2_t){1, 1});
    // below 2^(-13 - qe)
    const int bound = max(-13 - qe + 127, 1) << 7;
    const bool small = min(least[0], least[1]) < bound - 1;
    if (__builtin_expect(__any(small), 0)) {
      const bool row_small = row_max(small ? 1.f : 0.f) > 0.f;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        uint32_t top = 0;
#pragma unroll
        for (int s = g * SPG; s < (g + 1) * SPG; ++s)
#pragma unroll
          for (int w = 0; w < 4; ++w) top = pk_max_finite(top, hidden(raw[s][w]));
        const float most = row_max(fmaxf(lo_bf16(top), hi_bf16(top)));
        const int more = row_small && most > 0.f ? min(15 - __builtin_amdgcn_frexp_expf(most) - qe, 255) : 0;
        drop[g / 4] |= (uint32_t)more << 8 * (g % 4);
      }
      any_drop = __any(drop[0] != 0 || drop[(G - 1) / 4] != 0);
#pragma unroll
      for (int g = 0; g < (G + 3) / 4; ++g) *(lds_u32 *)(lds_t *)(uintptr_t)(drops + 4 * g) = drop[g];
    }
  }
#pragma unroll
  for (int g = 0; g < G; ++g) qsum[g] = 0.f;
#pragma unroll
  for (int s = 0; s < NS; ++s)
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float x = lo_bf16(raw[s][w] ^ flip), y = hi_bf16(raw[s][w] ^ flip);
      qsum[s / SPG] += ldexpf(x, -8) + ldexpf(y, -8);  // 256 of the greatest numbers stay a number
      const int e = qe + (int)(drop[s / SPG / 4] >> 8 * (s / SPG % 4) & 255) - 4;
      qf[s][w] = __builtin_bit_cast(uint32_t, (h2){(_Float16)ldexpf(x, e), (_Float16)ldexpf(y, e)});
    }
#pragma unroll
  for (int g = 0; g < G; ++g) qsum[g] = ldexpf(row_sum(qsum[g]), qe + 8 - 24);
  const float sc = exponent_scale(a.scale);
  const int se = 24 - qe;

  f4 O[NT];
  float M[G], l = 0.f, m = -__FLT_MAX__, above = m;  // above: the greatest score without a new maximum
  int E = -110;  // 2^(8 - E) times a weight of 2^6 is a number, and the least value far above 2^(E - 32)
#pragma unroll
  for (int t = 0; t < NT; ++t) O[t] = (f4){};
#pragma unroll
  for (int g = 0; g < G; ++g) M[g] = 0.f;
  auto rescale = [&](float f) {
#pragma unroll
    for (int g = 0; g < G; ++g) M[g] *= f;
#pragma unroll
    for (int n = 0; n < NT; ++n) O[n] *= f;
  };

#pragma unroll 1
  for (int n = 0; n < count; ++n) {
    // the last chunk's reads are over before its place is written again
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

    float t[2][4];
    auto scores = [&](auto divided) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t kw[NS];
        lds_words<NS>(src + j * RUN + lane * (4 * NS), kw);
#pragma unroll
        for (int i = 0; i < 4; ++i) t[j][i] = 0.f;
#pragma unroll
        for (int g = 0; g < G; ++g) {
          f4 A = {};
#pragma unroll
          for (int s = 0; s < SPG; ++s) A = mfma_f16(nibbles(kw[g * SPG + s]), qf[g * SPG + s], A);
          if constexpr (divided) {
            const int by = *(lds_u32 *)(lds_t *)(uintptr_t)(drops + 4 * (g / 4)) >> 8 * (g % 4) & 255;
#pragma unroll
            for (int i = 0; i < 4; ++i) A[i] = ldexpf(A[i], -by);
          }
          const u4 kp = lds_u128(src + j * RUN + 2 * KB + (h * G + g) * 16);
#pragma unroll
          for (int i = 0; i < 4; ++i) t[j][i] = fmaf(lo_bf16(kp[i]), A[i], fmaf(hi_bf16(kp[i]), qsum[g], t[j][i]));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) t[j][i] = ldexpf(t[j][i], se);
      }
    };
    if (__builtin_expect(any_drop, 0))
      scores(std::true_type());
    else
      scores(std::false_type());
    u4 vp[2][G];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int g = 0; g < G; ++g) vp[j][g] = lds_u128(src + j * RUN + 2 * KB + PB + (h * G + g) * 16);
    if (!(ok == 3 && k0 >= lo_max && k0 + CHUNK <= hi_min)) {
      // some row does not see all of it: hidden keys have the weight zero and
      // zeros for parameters, whatever lies there
      const int of_row = (int)hidden(r_token), lo = lo_of(of_row), hi = hi_of(of_row);  // (formed here: two registers less)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = k0 + 16 * j + 4 * h + i;
          const bool seen = key >= lo && key < hi && (ok >> j & 1);
          t[j][i] = seen ? t[j][i] : -__builtin_inff();
#pragma unroll
          for (int g = 0; g < G; ++g) vp[j][g][i] = seen ? vp[j][g][i] : 0u;
        }
    }
    float top = t[0][0];
#pragma unroll
    for (int i = 1; i < 8; ++i) top = fmaxf(top, t[i >> 2][i & 3]);
    if (__any(top > above)) {
      // of the rows that need one (the others keep every bit, whatever the
      // tile's other rows see)
      const float high = row_max(top), now = high > above ? high : m, f = __builtin_amdgcn_exp2f((m - now) * sc);
      l *= f;
      rescale(f);
      m = now;
      above = raised_by(m, 6.f, sc);
    }
    float p[2][4], pm[G];
    u4 w[G], rest[G];
    // E to the greatest finite scale or minimum that the row sees here, where it
    // needs it; by how much it has risen
    auto raise = [&](bool need) {
      uint32_t most = 0;
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) most = pk_max_mag(most, hidden(vp[j][g][i]));
      if (__builtin_expect(__any(not_finite(most)), 0)) {
        most = 0;
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) most = pk_max_finite(most, hidden(vp[j][g][i]));
      }
      const float big = row_max(fmaxf(lo_bf16(most), hi_bf16(most)));
      const int by = need && big > 0.f ? max(__builtin_amdgcn_frexp_expf(big) - E, 0) : 0;
      rescale(ldexpf(1.f, -by));
      E += by;
      return by;
    };
    if (n == 0) raise(true);
#pragma unroll 1
    for (;;) {
      const float unit = ldexpf(1.f, 8 - E);
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i >> 2][i & 3] = __builtin_amdgcn_exp2f((t[i >> 2][i & 3] - m) * sc) * unit;
      us2_t most = {0, 0};
      float far = 0.f;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        pm[g] = 0.f;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < 4; i += 2) {
            const float s0 = lo_bf16(vp[j][g][i]), s1 = lo_bf16(vp[j][g][i + 1]);
            pm[g] = fmaf(p[j][i], hi_bf16(vp[j][g][i]), pm[g]);
            pm[g] = fmaf(p[j][i + 1], hi_bf16(vp[j][g][i + 1]), pm[g]);
            // (the compiler would round it twice, from fp32 for the product and at
            // once for the rest, and one weight in 8000 would get a rest that is
            // not its own)
            const h2 x = once((h2){(_Float16)(p[j][i] * s0), (_Float16)(p[j][i + 1] * s1)});
            const h2 y = {(_Float16)fmaf(p[j][i], s0, -(float)x[0]), (_Float16)fmaf(p[j][i + 1], s1, -(float)x[1])};
            w[g][2 * j + (i >> 1)] = __builtin_bit_cast(uint32_t, x);
            rest[g][2 * j + (i >> 1)] = __builtin_bit_cast(uint32_t, y);
            most = __builtin_elementwise_max(most, __builtin_bit_cast(us2_t, x));  // weights are not negative
          }
        far = fmaxf(far, fabsf(pm[g]));
      }
      const bool over = most[0] >= 0x7C00 || most[1] >= 0x7C00 || far > 0x1p100f;
      if (__builtin_expect(!__any(over), 1)) break;
      const int by = raise(row_max(over ? 1.f : 0.f) > 0.f);
      if (!__any(by > 0)) break;  // what does not fit then is not finite
    }
    float weights = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) weights += p[i >> 2][i & 3];
    l += ldexpf(weights, E - 8);
#pragma unroll
    for (int g = 0; g < G; ++g) M[g] += pm[g];
    // value runs: dword w of a key holds tiles 8w .. 8w + 7 (at 64 channels
    // a half dword, two keys a dword)
    uint32_t vw[2][NS];
#pragma unroll
    for (int j = 0; j < 2; ++j) lds_words<NS>(src + j * RUN + KB + lane * (4 * NS), vw[j]);
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
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const u4 f = (e == 0 ? v4 << 4 : v4 >> 4 * (e - 1)) & 0x00F000F0u;
        const int tile = 4 * n4 + e, g = tile / TPG;
        O[tile] = mfma_f16(f, w[g], O[tile]);
        O[tile] = mfma_f16(f, rest[g], O[tile]);
      }
    }
  }
  __syncthreads();  // the waves' copies share their place with what follows

  // the waves meet in LDS: numerators [wave][row][D], then maxima, exponents and
  // sums (a wave without keys brings zeros under the least maximum)
  float *s_o = (float *)smem;
  float *s_m = s_o + CACHE_WAVES * ROWS * (D + 4), *s_l = s_m + CACHE_WAVES * ROWS;
  int *s_e = (int *)(s_l + CACHE_WAVES * ROWS);
  l = row_sum(l);
  float *mine = s_o + (wv * ROWS + col) * (D + 4);
#pragma unroll
  for (int g = 0; g < G; ++g) M[g] = row_sum(M[g]);
#pragma unroll
  for (int n = 0; n < NT; ++n) *(f4 *)(mine + 16 * n + 4 * h) = O[n] * 0x1p20f + M[n / TPG];
  if (h == 0) {
    s_m[wv * ROWS + col] = m;
    s_l[wv * ROWS + col] = l;
    s_e[wv * ROWS + col] = E - 8;
  }
  __syncthreads();
  const int row = tid >> 4, part = tid & 15;  // 16 threads a row, D / 16 channels each
  const int q_row = rt * ROWS + row;
  if (q_row >= R) return;
  float most = -__FLT_MAX__, sum = 0.f, f[CACHE_WAVES];
#pragma unroll
  for (int w = 0; w < CACHE_WAVES; ++w) most = fmaxf(most, s_m[w * ROWS + row]);
  int unit = -1024;  // the greatest exponent of those whose weights count
#pragma unroll
  for (int w = 0; w < CACHE_WAVES; ++w) {
    f[w] = __builtin_amdgcn_exp2f((s_m[w * ROWS + row] - most) * sc);
    sum += s_l[w * ROWS + row] * f[w];
    unit = f[w] > 0.f ? max(unit, s_e[w * ROWS + row]) : unit;
  }
#pragma unroll
  for (int w = 0; w < CACHE_WAVES; ++w) f[w] = ldexpf(f[w], s_e[w * ROWS + row] - unit);
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  f4 out[D / 64];
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    out[i] = (f4){};
#pragma unroll
    for (int w = 0; w < CACHE_WAVES; ++w) out[i] += *(const f4 *)(s_o + (w * ROWS + row) * (D + 4) + 64 * i + 4 * part) * f[w];
    out[i] *= inv;
#pragma unroll
    for (int e = 0; e < 4; ++e) out[i][e] = ldexpf(out[i][e], unit);
  }
  if (a.splits == 1) {
    const int token = a.q_len > 1 ? q_row / shared : 0;
    uint16_t *y = a.y + (int64_t)(b * a.q_len + token) * a.ldy + (kvh * shared + q_row - token * shared) * D + 4 * part;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) *(u2 *)(y + 64 * i) = row_bf16(out[i]);
    return;
  }
  const int64_t at = (((int64_t)b * c.heads + kvh) * R + q_row) * a.splits + sp;
#pragma unroll
  for (int i = 0; i < D / 64; ++i) *(f4 *)(a.part + at * D + 64 * i + 4 * part) = out[i];
  if (part == 0) *(float2 *)(a.sums + 2 * at) = make_float2(most, sum);
}

// Joins the key ranges of a row, each range's own result under its sum of
// weights, added in a fixed order: a block a row, D / 4 threads a range, four
// channels a thread.  (Sums in 64 bits: the weights' sums reach 2^36 where the
// results may be any fp32 number.)  Latency (2.4 to 5 us); the reads are what the
// ranges have just written.
template <int D>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnCacheArgs a) {
  constexpr int T = D / 4, N = 256 / T;
  __shared__ d4 s_o[N][T];
  __shared__ float s_l[N];
  const int tid = threadIdx.x, lane = tid & 63, part = tid % T, first = tid / T;
  const int shared = a.heads / a.c.heads, R = shared * a.q_len;
  const int64_t at = blockIdx.x;
  const float sc = exponent_scale(a.scale);
  const float2 *sums = (const float2 *)a.sums + at * a.splits;
  float m = -__FLT_MAX__;
  for (int s = lane; s < a.splits; s += 64) m = fmaxf(m, sums[s].x);
  m = row_max(lanes_max(m, 16));
  float sum = 0.f;
  d4 o = {};
  const f4 *value = (const f4 *)(a.part + at * a.splits * D) + part;
#pragma unroll 4
  for (int s = first; s < a.splits; s += N) {
    const float2 x = sums[s];
    const f4 v = value[(int64_t)s * T];
    const float w = x.y * __builtin_amdgcn_exp2f((x.x - m) * sc);  // 0 of a range without keys
    sum += w;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] += (double)v[e] * w;
  }
  s_o[first][part] = o;
  if (part == 0) s_l[first] = sum;
  __syncthreads();
  if (tid >= T) return;
#pragma unroll 4
  for (int n = 1; n < N; ++n) {
    o += s_o[n][part];
    sum += s_l[n];
  }
  const double inv = sum == 0.f ? 0. : (double)(1.f / sum);
  const int q_row = (int)(at % R), kvh = (int)(at / R % a.c.heads);
  const int64_t b = at / R / a.c.heads;
  f4 y;
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] = (float)(o[e] * inv);
  *(u2 *)(a.y + (b * a.q_len + q_row / shared) * a.ldy + (kvh * shared + q_row % shared) * D + 4 * part) = row_bf16(y);
}

template <int D, int GROUP>
hipError_t launch_cache(const AttnCacheArgs &a, hipStream_t s) {
  constexpr size_t lds = cache_lds<D, D / GROUP>();
  const hipError_t e = allow_smem(attn_cache_kernel<D, GROUP>, lds);
  if (e != hipSuccess) return e;
  attn_cache_kernel<D, GROUP><<<dim3(a.c.heads, a.row_tiles * a.splits, a.batch), 64 * CACHE_WAVES, lds, s>>>(a);
  if (a.splits > 1) {
    const int64_t rows = (int64_t)a.batch * a.heads * a.q_len;
    attn_join_kernel<D><<<dim3((unsigned)rows), 256, 0, s>>>(a);
  }
  return hipGetLastError();
}

}  // namespace

// Blocks of 4 waves: 64 tokens of the key side, 4096 / dim of the value side.
// Where the value side has more blocks, those of the key side past the last token
// return at once when reading, and store nothing when writing.
static dim3 kv_grid(const KvView &c, int64_t tokens) {
  const int per = 4096 / c.dim < 64 ? 4096 / c.dim : 64;
  return dim3((unsigned)((tokens + per - 1) / per), c.heads, 2);
}

hipError_t launch_kv_write(const KvWriteArgs &a, hipStream_t s) {
  const dim3 grid = kv_grid(a.c, a.tokens);
  switch (a.c.dim) {
    case 64: kv_write_kernel<64><<<grid, 256, 0, s>>>(a); break;
    case 128: kv_write_kernel<128><<<grid, 256, 0, s>>>(a); break;
    default: kv_write_kernel<256><<<grid, 256, 0, s>>>(a);
  }
  return hipGetLastError();
}

hipError_t launch_kv_read(const KvReadArgs &a, hipStream_t s) {
  const dim3 grid = kv_grid(a.c, a.tokens);
  switch (a.c.dim) {
    case 64: kv_read_kernel<64><<<grid, 256, 0, s>>>(a); break;
    case 128: kv_read_kernel<128><<<grid, 256, 0, s>>>(a); break;
    default: kv_read_kernel<256><<<grid, 256, 0, s>>>(a);
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
