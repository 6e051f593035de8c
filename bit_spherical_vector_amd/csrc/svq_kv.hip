// The 4-bit cache of keys and values (include/svq_attn.h): quantising tokens
// into it, reading them back, attention over it.
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
      const int p8 = (n & 3) * (D / 32) + (n >> 2);
      if (N > 4 || !(r & 1)) *(uint32_t *)(blk + kv_key_word(a.c, place, p8)) = word[w];
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
      const uint32_t w = *(const uint32_t *)(blk + kv_key_word(a.c, place, (n & 3) * (D / 32) + (n >> 2)));
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

// A wave a (row, query head): 64 keys at a time, one a lane, for the scores
// and the running maximum and sum; then every lane D/64 channels over them.
template <int D>
__global__ __launch_bounds__(256) void attn_cache_kernel(AttnCacheArgs a) {
  const KvView &c = a.c;
  const int lane = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (row >= (int64_t)a.batch * a.q_len) return;
  const int h = blockIdx.y, kvh = h / (a.heads / c.heads);
  const int b = (int)(row / a.q_len), t = (int)(row % a.q_len);
  const int len = min(max(a.lens[b], 0), a.max_len), pos = len - a.q_len + t;
  const int lo = a.window > 0 ? max(0, pos - a.window + 1) : 0, hi = max(0, pos + 1);
  const uint16_t *q = a.q + row * a.ldq + h * D;
  float m = -__builtin_inff(), l = 0.f, acc[D / 64] = {};
  for (int k0 = lo; k0 < hi; k0 += 64) {
    const int j = k0 + lane;
    int32_t page = -1;
    if (j < hi) page = a.table[b * a.ld_table + (j >> c.page_shift)];
    const bool in = page >= 0 && page < c.pages;
    const uint8_t *blk = kv_block(c, in ? page : 0, kvh);
    const int place = in ? j & ((1 << c.page_shift) - 1) : 0;
    float s = 0.f;
    if (in)
      for (int n = 0; n < D / 8; ++n) {
        const uint32_t w = *(const uint32_t *)(blk + kv_key_word(c, place, (n & 3) * (D / 32) + (n >> 2)));
        const uint32_t p = *(const uint32_t *)(blk + kv_param(c, 0, place, 8 * n >> c.group_shift));
        for (int e = 0; e < 8; ++e)
          s += bf16_bits_to_f32(q[8 * n + e]) * fmaf((float)((w >> 4 * kv_nibble(e)) & 15), bf16_bits_to_f32(p & 0xFFFFu),
                                                     __builtin_bit_cast(float, p & 0xFFFF0000u));
      }
    s = in ? s * a.scale : -__builtin_inff();
    float top = s;
    for (int o = 32; o; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
    const float mn = fmaxf(m, top), ref = mn == -__builtin_inff() ? 0.f : mn;
    const float p = in ? expf(s - ref) : 0.f, alpha = m == -__builtin_inff() ? 0.f : expf(m - ref);
    float sum = p;
    for (int o = 32; o; o >>= 1) sum += __shfl_xor(sum, o);
    l = l * alpha + sum;
    m = mn;
    for (int i = 0; i < D / 64; ++i) acc[i] *= alpha;
    for (int e = 0; e < 64 && k0 + e < hi; ++e) {
      const float pe = __shfl(p, e);
      const int pg = __shfl(in ? page : -1, e), pl = (k0 + e) & ((1 << c.page_shift) - 1);
      if (pg < 0) continue;
      const uint8_t *vb = kv_block(c, pg, kvh);
      for (int i = 0; i < D / 64; ++i) {
        const int d = lane + 64 * i, tile = d >> 4;
        const uint32_t pr = *(const uint32_t *)(vb + kv_param(c, 1, pl, d >> c.group_shift));
        const uint32_t code = (vb[kv_value_run(c, pl, d & 15) + (tile >> 1)] >> 4 * (tile & 1)) & 15;
        acc[i] += pe * fmaf((float)code, bf16_bits_to_f32(pr & 0xFFFFu), __builtin_bit_cast(float, pr & 0xFFFF0000u));
      }
    }
  }
  for (int i = 0; i < D / 64; ++i)
    a.y[row * a.ldy + h * D + lane + 64 * i] = f32_to_bf16_bits(l == 0.f ? 0.f : acc[i] / l);
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
  const dim3 grid((unsigned)(((int64_t)a.batch * a.q_len + 3) / 4), a.heads);
  switch (a.c.dim) {
    case 64: attn_cache_kernel<64><<<grid, 256, 0, s>>>(a); break;
    case 128: attn_cache_kernel<128><<<grid, 256, 0, s>>>(a); break;
    default: attn_cache_kernel<256><<<grid, 256, 0, s>>>(a);
  }
  return hipGetLastError();
}

}  // namespace svq
