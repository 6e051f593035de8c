// Device side of the products' epilogues: bias, activation, residual.
//
// An epilogue runs where the product's fp32 sum ends, before its one rounding
// to the output type, so bias, activation and residual cost no launch and no
// round trip of the product through memory.
#pragma once
#include "svq_device.h"
#include "../../include/svq_ffn.h"

namespace svq {

// Activations, each from the exponential of a non-positive or harmlessly
// overflowing argument so that no difference of near-equal numbers is
// rounded:
//   silu(v)      = v / (1 + e^-v)
//   gelu(v)      = v/2 * erfc(-v / sqrt 2)
//   gelu_tanh(v) = v / (1 + e^(-2z)), z = sqrt(2/pi) (v + 0.044715 v^3)
//                  (v/2 (1 + tanh z) with tanh written by the exponential)
// relu keeps a NaN.
__device__ __forceinline__ float act_apply(float v, int act) {
  switch (act) {
    case SVQ_ACT_RELU: return v < 0.f ? 0.f : v;
    case SVQ_ACT_SILU: return v / (1.f + expf(-v));
    case SVQ_ACT_GELU: return 0.5f * v * erfcf(-0.70710678118654752f * v);
    case SVQ_ACT_GELU_TANH: {
      const float z = 0.79788456080286536f * __builtin_fmaf(0.044715f * v * v, v, v);
      return v / (1.f + expf(-2.f * z));
    }
    default: return v;
  }
}

// Cheaper forms for values that are rounded to 11 bits or fewer next: the
// hardware's exp2 and reciprocal (each within about 1 ulp) in place of expf
// and a division; the argument's rounding adds |v| 2^-24.
template <int ACT>
__device__ __forceinline__ float act_fast(float v) {
  if constexpr (ACT == SVQ_ACT_RELU) return v < 0.f ? 0.f : v;
  if constexpr (ACT == SVQ_ACT_SILU)
    return v * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.44269504088896341f * v));
  if constexpr (ACT == SVQ_ACT_GELU) return act_apply(v, SVQ_ACT_GELU);
  if constexpr (ACT == SVQ_ACT_GELU_TANH) {
    const float z = v * __builtin_fmaf(0.044715f * v, v, 1.f);
    return v * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-2.f * 0.79788456080286536f * 1.44269504088896341f * z));
  }
  return v;
}
__device__ __forceinline__ float act_fast(float v, int act) {
  switch (act) {
    case SVQ_ACT_RELU: return act_fast<SVQ_ACT_RELU>(v);
    case SVQ_ACT_SILU: return act_fast<SVQ_ACT_SILU>(v);
    case SVQ_ACT_GELU: return act_fast<SVQ_ACT_GELU>(v);
    case SVQ_ACT_GELU_TANH: return act_fast<SVQ_ACT_GELU_TANH>(v);
    default: return v;
  }
}

// Beyond 16 rows, where tiles and the join of K ranges finish parts of one
// output: the cheap forms where it is rounded to bf16, in all of them, and
// expf and a division for an fp32 output.
__device__ __forceinline__ float act_out(float v, int act, bool bf) {
  return bf ? act_fast(v, act) : act_apply(v, act);
}

__device__ __forceinline__ float load_f(const void *p, size_t i, int f32) {
  return f32 ? ((const float *)p)[i] : bf16_bits_to_f32(((const uint16_t *)p)[i]);
}

// Four consecutive values from element i (vec: the address allows one load).
__device__ __forceinline__ f4 load_f4(const void *p, size_t i, int f32, bool vec) {
  if (vec && f32) return *(const f4 *)((const float *)p + i);
  if (vec) {
    const u2 b = *(const u2 *)((const uint16_t *)p + i);
    return (f4){bf16_bits_to_f32(b[0] & 0xFFFFu), __builtin_bit_cast(float, b[0] & 0xFFFF0000u),
                bf16_bits_to_f32(b[1] & 0xFFFFu), __builtin_bit_cast(float, b[1] & 0xFFFF0000u)};
  }
  return (f4){load_f(p, i, f32), load_f(p, i + 1, f32), load_f(p, i + 2, f32), load_f(p, i + 3, f32)};
}

// No epilogue: the product kernels' default.
struct NoEpi {
  static constexpr bool on = false, partial = false, f16 = false;
  __device__ __forceinline__ float operator()(float v, int, int) const { return v; }
};

struct Epi {
  static constexpr bool on = true, partial = false, f16 = false;
  EpiArgs a;
  bool bf = false;  // act_out's
  // output row `row`, column n
  __device__ __forceinline__ float operator()(float v, int row, int n) const {
    if (a.bias) v += load_f(a.bias, n, a.bias_f32);
    v = act_out(v, a.act, bf);
    if (a.res) v += load_f(a.res, (size_t)row * a.ldr + n, a.res_f32);
    return v;
  }
  // columns n0 .. n0 + 3 (n0 a multiple of 4; those below nlim) of row `row`
  __device__ __forceinline__ void store4(void *y, int64_t ldy, bool ybf, bool yvec, f4 v, int row, int n0,
                                         int nlim) const {
    const size_t at = (size_t)row * ldy + n0;
    if (n0 + 4 > nlim) {
      for (int l = 0; n0 + l < nlim; ++l) store_out(y, at + l, (*this)(v[l], row, n0 + l), ybf ? 0 : 1);
      return;
    }
    if (a.bias) v += load_f4(a.bias, n0, a.bias_f32, a.bias_vec != 0);
    if (a.act != SVQ_ACT_NONE)
#pragma unroll
      for (int l = 0; l < 4; ++l) v[l] = act_out(v[l], a.act, bf);
    if (a.res) v += load_f4(a.res, (size_t)row * a.ldr + n0, a.res_f32, a.res_vec != 0);
    store_f4(y, at, v, ybf, yvec);
  }
  static __device__ __forceinline__ void store_f4(void *y, size_t at, f4 v, bool bf, bool vec) {
    if (bf) {
      uint16_t *p = (uint16_t *)y + at;
      const u2 o = {(uint32_t)f32_to_bf16_bits(v[0]) | ((uint32_t)f32_to_bf16_bits(v[1]) << 16),
                    (uint32_t)f32_to_bf16_bits(v[2]) | ((uint32_t)f32_to_bf16_bits(v[3]) << 16)};
      if (vec) {
        *(u2 *)p = o;
      } else {
        p[0] = (uint16_t)o[0];
        p[1] = (uint16_t)(o[0] >> 16);
        p[2] = (uint16_t)o[1];
        p[3] = (uint16_t)(o[1] >> 16);
      }
    } else {
      float *p = (float *)y + at;
      if (vec) {
        *(f4 *)p = v;
      } else {
#pragma unroll
        for (int l = 0; l < 4; ++l) p[l] = v[l];
      }
    }
  }
};

// The sums go to an fp32 row that another block reads in the same launch:
// device-scope stores, coherent between the XCDs' caches.
struct PartEpi {
  static constexpr bool on = true, partial = true, f16 = false;
  float *row;
  __device__ __forceinline__ void put(float v, int, int n) const {
    __hip_atomic_store(row + n, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
};

// A gated pair whose sums meet in memory (see PairArgs).
struct PairEpi {
  static constexpr bool on = true;
  PairArgs a;
  __device__ __forceinline__ float operator()(float v, int, int) const { return v; }
};
__device__ __forceinline__ float pair_value(const PairArgs &a, float g, float u, int n) {
  if (a.bias_g) g += load_f(a.bias_g, n, a.bias_f32);
  if (a.bias_u) u += load_f(a.bias_u, n, a.bias_f32);
  return act_apply(g, a.act) * u;
}

// The epilogue of a kernel's optional EpiArgs argument.
__device__ __forceinline__ NoEpi make_epi() { return NoEpi(); }
__device__ __forceinline__ Epi make_epi(const EpiArgs &a) { return Epi{a}; }
__device__ __forceinline__ PairEpi make_epi(const PairArgs &a) { return PairEpi{a}; }

}  // namespace svq
