// Attention over whole prompts (include/svq_attn.h).
#include "svq_attn.h"
#include "svq_device.h"

namespace svq {
namespace {

// A wave a (row, query head): 64 keys at a time, one a lane, for the scores
// and the running maximum and sum; then every lane D/64 channels over them.
template <int D>
__global__ __launch_bounds__(256) void attn_prompt_kernel(AttnPromptArgs a) {
  const int lane = threadIdx.x & 63;
  const int row = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (row >= a.tokens) return;
  const int h = blockIdx.y, kvh = h / (a.heads / a.kv_heads);
  int n = -1, t = 0, k_at = 0, keys = 0;
  for (int s = 0; s < a.sequences; ++s) {
    const int b = min(max(a.starts[s], 0), a.tokens), e = min(max(a.starts[s + 1], b), a.tokens);
    if (row >= b && row < e) {
      n = e - b;
      t = row - b;
      k_at = min(max(a.starts_k[s], 0), a.tokens_k);
      keys = min(max(a.starts_k[s + 1], k_at), a.tokens_k) - k_at;
      break;
    }
  }
  if (n < 0) return;
  const int pos = keys - n + t;
  const int lo = a.window > 0 ? max(0, pos - a.window + 1) : 0, hi = a.causal ? max(0, pos + 1) : keys;
  const uint16_t *q = a.q + row * a.ldq + h * D;
  float m = -__builtin_inff(), l = 0.f, acc[D / 64] = {};
  for (int k0 = lo; k0 < hi; k0 += 64) {
    const int j = k0 + lane;
    const bool in = j < hi;
    const uint16_t *k = a.k + (int64_t)(k_at + (in ? j : lo)) * a.ldk + kvh * D;
    float s = 0.f;
    for (int d = 0; d < D; ++d) s += bf16_bits_to_f32(q[d]) * bf16_bits_to_f32(k[d]);
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
      const uint16_t *v = a.v + (int64_t)(k_at + k0 + e) * a.ldv + kvh * D;
      for (int i = 0; i < D / 64; ++i) acc[i] += pe * bf16_bits_to_f32(v[lane + 64 * i]);
    }
  }
  for (int i = 0; i < D / 64; ++i)
    a.y[row * a.ldy + h * D + lane + 64 * i] = f32_to_bf16_bits(l == 0.f ? 0.f : acc[i] / l);
}

}  // namespace

hipError_t launch_attn_prompt(const AttnPromptArgs &a, hipStream_t s) {
  const dim3 grid((unsigned)((a.tokens + 3) / 4), a.heads);
  switch (a.dim) {
    case 64: attn_prompt_kernel<64><<<grid, 256, 0, s>>>(a); break;
    case 128: attn_prompt_kernel<128><<<grid, 256, 0, s>>>(a); break;
    default: attn_prompt_kernel<256><<<grid, 256, 0, s>>>(a);
  }
  return hipGetLastError();
}

}  // namespace svq
