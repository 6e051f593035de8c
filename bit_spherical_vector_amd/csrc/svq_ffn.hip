// Kernels of the feed-forward calls (include/svq_ffn.h) that are not products:
// the gated pair's elementwise step, the sum over a token's experts and the
// router.
#include <cmath>

#include "svq_device.h"
#include "svq_epilogue.h"
#include "svq_ffn.h"

namespace svq {

// h[r][n] = act(g[r][n] + bg[n]) * (u[r][n] + bu[n]), four columns a thread;
// g and u fp32 [rows][ldp], ldp a multiple of 4.
__global__ __launch_bounds__(256) void glu_kernel(GluArgs a) {
  const int64_t per_row = (a.n + 3) / 4, total = a.rows * per_row;
  for (int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x; q < total; q += (int64_t)gridDim.x * 256) {
    const int64_t r = q / per_row;
    const int n0 = (int)(q - r * per_row) * 4;
    f4 g = *(const f4 *)(a.g + r * a.ldp + n0), u = *(const f4 *)(a.u + r * a.ldp + n0);
#pragma unroll
    for (int l = 0; l < 4; ++l) {
      if (n0 + l >= a.n) break;
      if (a.bias_g) g[l] += load_f(a.bias_g, n0 + l, a.bias_f32);
      if (a.bias_u) u[l] += load_f(a.bias_u, n0 + l, a.bias_f32);
      store_out(a.y, (size_t)r * a.ldy + n0 + l, act_apply(g[l], a.act) * u[l], a.ydt);
    }
  }
}

hipError_t launch_glu(const GluArgs &a, hipStream_t s) {
  const int64_t total = a.rows * ((a.n + 3) / 4);
  int64_t blocks = (total + 255) / 256;
  if (blocks > 65536) blocks = 65536;
  hipLaunchKernelGGL(glu_kernel, dim3((unsigned)blocks), dim3(256), 0, s, a);
  return hipGetLastError();
}

// y[t][n] = res[t][n] + sum_j w[t][j] d[t topk + j][n] in slot order, four
// columns a thread; slots with ids outside [0, E) are left out.
__global__ __launch_bounds__(256) void moe_combine_kernel(CombineArgs a) {
  const int64_t per_row = (a.n + 3) / 4, total = a.m * per_row;
  for (int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x; q < total; q += (int64_t)gridDim.x * 256) {
    const int64_t t = q / per_row;
    const int n0 = (int)(q - t * per_row) * 4;
    f4 v = {0.f, 0.f, 0.f, 0.f};
    for (int j = 0; j < a.topk; ++j) {
      const int64_t s = t * a.topk + j;
      const int e = a.ids[s];
      if (e < 0 || e >= a.num_experts) continue;
      const f4 d = *(const f4 *)(a.d + s * a.ldd + n0);
      const float w = a.weights[s];
#pragma unroll
      for (int l = 0; l < 4; ++l) v[l] = __builtin_fmaf(w, d[l], v[l]);
    }
#pragma unroll
    for (int l = 0; l < 4; ++l) {
      if (n0 + l >= a.n) break;
      if (a.res) v[l] += load_f(a.res, (size_t)t * a.ldr + n0 + l, a.res_f32);
      store_out(a.y, (size_t)t * a.ldy + n0 + l, v[l], a.ydt);
    }
  }
}

hipError_t launch_combine(const CombineArgs &a, hipStream_t s) {
  const int64_t total = a.m * ((a.n + 3) / 4);
  int64_t blocks = (total + 255) / 256;
  if (blocks > 65536) blocks = 65536;
  hipLaunchKernelGGL(moe_combine_kernel, dim3((unsigned)blocks), dim3(256), 0, s, a);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Router
// ---------------------------------------------------------------------------
//
// A block of 16 waves takes T tokens and all experts, so that logits, scores
// and the choice need one launch and no memory between them.  Wave w sums the
// logits of experts w + 16 i, eight at a time: a lane holds the eight
// channels 512c + 8 lane .. + 7 of its T tokens as doubles and multiplies
// them with the same channels of each expert's row, so a weight is converted
// once for T tokens.  Products of bf16 values are exact in double and the
// sums keep 53 bits: the choice is that of the exact logits up to differences
// of about 1e-15 of their size.  The vector units do double FMAs at the rate
// of the matrix cores' double MFMAs on this chip, without padding few tokens
// to 16 rows.
constexpr int RT_WAVES = 16;
constexpr int RT_EG = 8;  // experts a wave sums side by side

template <bool F32>
struct RtRow {
  u4 v[F32 ? 2 : 1];
};

// Channels k0 .. k0 + 7 of a row (zeros past k); vec: the row allows 16-byte
// loads and k is a multiple of 8.
template <bool F32>
__device__ __forceinline__ RtRow<F32> rt_load(const void *row, int k0, int k, bool vec) {
  RtRow<F32> r;
  if (vec) {
    const int at = min(k0, k - 8);  // clamped loads; the caller's x is zero past k
    if constexpr (F32) {
      r.v[0] = *(const u4 *)((const float *)row + at);
      r.v[1] = *(const u4 *)((const float *)row + at + 4);
    } else {
      r.v[0] = *(const u4 *)((const uint16_t *)row + at);
    }
  } else {
#pragma unroll
    for (int l = 0; l < 4; ++l) {
      const int a = min(k0 + 2 * l, k - 1), b = min(k0 + 2 * l + 1, k - 1);
      if constexpr (F32) {
        r.v[l >> 1][2 * (l & 1)] = ((const uint32_t *)row)[a];
        r.v[l >> 1][2 * (l & 1) + 1] = ((const uint32_t *)row)[b];
      } else {
        r.v[0][l] = (uint32_t)((const uint16_t *)row)[a] | ((uint32_t)((const uint16_t *)row)[b] << 16);
      }
    }
  }
  return r;
}
template <bool F32>
__device__ __forceinline__ double rt_get(const RtRow<F32> &r, int l) {
  if constexpr (F32) return (double)__builtin_bit_cast(float, (uint32_t)r.v[l >> 2][l & 3]);
  const uint32_t p = r.v[0][l >> 1];
  return (double)__builtin_bit_cast(float, (l & 1) ? p & 0xFFFF0000u : p << 16);
}

__device__ __forceinline__ double shfl_xor_f64(double v, int d) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__shfl_xor((int)(uint32_t)b, d), hi = (uint32_t)__shfl_xor((int)(b >> 32), d);
  return __builtin_bit_cast(double, (uint64_t)lo | ((uint64_t)hi << 32));
}
__device__ __forceinline__ int64_t shfl_xor_i64(int64_t v, int d) {
  return __builtin_bit_cast(int64_t, shfl_xor_f64(__builtin_bit_cast(double, v), d));
}

// Order-preserving integer of a key: NaN below every number, -0 equal to +0.
__device__ __forceinline__ int64_t rt_order(double key) {
  if (key != key) return INT64_MIN + 1;
  const int64_t b = __builtin_bit_cast(int64_t, key + 0.0);
  return b >= 0 ? b : (b ^ INT64_MAX);
}

template <int T, bool WF32>
__global__ __launch_bounds__(RT_WAVES * 64) void moe_route_topk_kernel(RouteArgs a) {
  __shared__ double s_logit[T][MAX_EXPERTS];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t t0 = (int64_t)blockIdx.x * T;
  const int k = a.k, E = a.num_experts;
  const bool vec = a.vec != 0;
  const size_t wsz = WF32 ? 4 : 2;
  const uint16_t *xr[T];
#pragma unroll
  for (int t = 0; t < T; ++t) xr[t] = a.x + min(t0 + t, a.m - 1) * a.ldx;

  for (int e0 = wv; e0 < E; e0 += RT_WAVES * RT_EG) {
    const char *wr[RT_EG];
#pragma unroll
    for (int i = 0; i < RT_EG; ++i)
      wr[i] = (const char *)a.w + (size_t)min(e0 + RT_WAVES * i, E - 1) * a.ldw * wsz;
    double acc[RT_EG][T];
#pragma unroll
    for (int i = 0; i < RT_EG; ++i)
#pragma unroll
      for (int t = 0; t < T; ++t) acc[i][t] = 0.0;
    for (int c = 0; c < k; c += 512) {
      const int k0 = c + 8 * lane;
      RtRow<WF32> wrow[RT_EG];
      RtRow<false> xrow[T];
#pragma unroll
      for (int t = 0; t < T; ++t) xrow[t] = rt_load<false>(xr[t], k0, k, vec);
#pragma unroll
      for (int i = 0; i < RT_EG; ++i) wrow[i] = rt_load<WF32>(wr[i], k0, k, vec);
#pragma unroll
      for (int l = 0; l < 8; ++l) {
        double xv[T];
#pragma unroll
        for (int t = 0; t < T; ++t) xv[t] = rt_get<false>(xrow[t], l);
        if (k0 + l < k) {
#pragma unroll
          for (int i = 0; i < RT_EG; ++i) {
            const double wd = rt_get<WF32>(wrow[i], l);
#pragma unroll
            for (int t = 0; t < T; ++t) acc[i][t] = __builtin_fma(xv[t], wd, acc[i][t]);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < RT_EG; ++i) {
#pragma unroll
      for (int t = 0; t < T; ++t) {
        double v = acc[i][t];
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) v += shfl_xor_f64(v, d);
        const int e = e0 + RT_WAVES * i;
        if (lane == 0 && e < E) s_logit[t][e] = v;
      }
    }
  }
  __syncthreads();
  if (wv >= T || t0 + wv >= a.m) return;

  // wave wv chooses for token t0 + wv; lane holds experts lane + 64 i
  constexpr int PL = MAX_EXPERTS / 64;
  const int64_t t = t0 + wv;
  double p[PL];
  int64_t key[PL];
  double mx = -INFINITY;
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    const int e = lane + 64 * i;
    p[i] = e < E ? s_logit[wv][e] : -INFINITY;
    if (!a.select_bias) key[i] = e < E ? rt_order(p[i]) : INT64_MIN;
    mx = fmax(mx, p[i]);
  }
  if (a.score == SVQ_ROUTE_SOFTMAX) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) mx = fmax(mx, shfl_xor_f64(mx, d));
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      p[i] = lane + 64 * i < E ? exp(p[i] - mx) : 0.0;
      sum += p[i];
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) sum += shfl_xor_f64(sum, d);
#pragma unroll
    for (int i = 0; i < PL; ++i) p[i] /= sum;
  } else {
#pragma unroll
    for (int i = 0; i < PL; ++i) p[i] = 1.0 / (1.0 + exp(-p[i]));
  }
  if (a.select_bias) {
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const int e = lane + 64 * i;
      key[i] = e < E ? rt_order(p[i] + (double)a.select_bias[min(e, E - 1)]) : INT64_MIN;
    }
  }
  double mine = 0.0, total = 0.0;  // lane j: the score of choice j
  int id = 0;
  for (int j = 0; j < a.topk; ++j) {
    int64_t bk = INT64_MIN;
    int be = MAX_EXPERTS;
    double bp = 0.0;
#pragma unroll
    for (int i = 0; i < PL; ++i)
      if (key[i] > bk) {  // equal keys keep the lower index (i ascending)
        bk = key[i];
        be = lane + 64 * i;
        bp = p[i];
      }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int64_t ok = shfl_xor_i64(bk, d);
      const int oe = __shfl_xor(be, d);
      const double op = shfl_xor_f64(bp, d);
      if (ok > bk || (ok == bk && oe < be)) {
        bk = ok;
        be = oe;
        bp = op;
      }
    }
#pragma unroll
    for (int i = 0; i < PL; ++i)
      if (lane + 64 * i == be) key[i] = INT64_MIN;
    if (lane == j) {
      mine = bp;
      id = be;
    }
    total += bp;
  }
  if (lane < a.topk) {
    if (a.renormalize) mine /= total;
    a.ids[t * a.topk + lane] = id;
    a.weights[t * a.topk + lane] = (float)(mine * (double)a.scale);
  }
}

template <int T>
static hipError_t launch_route_t(const RouteArgs &a, hipStream_t s) {
  const dim3 grid((unsigned)((a.m + T - 1) / T)), block(RT_WAVES * 64);
  if (a.w_f32)
    hipLaunchKernelGGL((moe_route_topk_kernel<T, true>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((moe_route_topk_kernel<T, false>), grid, block, 0, s, a);
  return hipGetLastError();
}

hipError_t launch_route(const RouteArgs &a, int cus, hipStream_t s) {
  if (a.m <= cus) return launch_route_t<1>(a, s);
  if (a.m <= 2 * (int64_t)cus) return launch_route_t<2>(a, s);
  return launch_route_t<4>(a, s);
}

}  // namespace svq
