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
// Two launches: logits in double to the workspace, then the choice.  Products
// of bf16 values are exact in double and the sums keep 53 bits, so the choice
// is that of the exact logits up to differences of about 1e-15 of their size.
// (One launch with a block per token and all experts in it was slower at
// every size: one token read the whole router matrix through one compute
// unit, 18.7 us against the two launches together; 512 tokens read it 256
// times.)

template <bool F32>
struct RtRow {
  u4 v[F32 ? 2 : 1];
};

// Channels k0 .. k0 + 7 of a row, zeros past k; vec: the row allows 16-byte
// loads and k is a multiple of 8.
template <bool F32>
__device__ __forceinline__ RtRow<F32> rt_load(const void *row, int k0, int k, bool vec) {
  RtRow<F32> r;
  if (vec) {
    const int at = min(k0, k - 8);
    if constexpr (F32) {
      r.v[0] = *(const u4 *)((const float *)row + at);
      r.v[1] = *(const u4 *)((const float *)row + at + 4);
    } else {
      r.v[0] = *(const u4 *)((const uint16_t *)row + at);
    }
    if (k0 >= k) {
      r.v[0] = (u4){0u, 0u, 0u, 0u};
      if constexpr (F32) r.v[1] = r.v[0];
    }
  } else {
#pragma unroll
    for (int l = 0; l < 8; ++l) {
      const int at = min(k0 + l, k - 1);
      if constexpr (F32) {
        const uint32_t b = ((const uint32_t *)row)[at];
        r.v[l >> 2][l & 3] = k0 + l < k ? b : 0u;
      } else {
        const uint32_t b = k0 + l < k ? ((const uint16_t *)row)[at] : 0u;
        r.v[0][l >> 1] = (l & 1) ? r.v[0][l >> 1] | (b << 16) : b;
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

// Few tokens: a wave per expert and RT_TOKENS tokens, the lanes along k (eight
// channels each), a double FMA per product, RT_CHUNKS chunks of 512 channels
// in flight.
constexpr int RT_TOKENS = 4;
constexpr int RT_CHUNKS = 4;
template <int T, bool WF32>
__global__ __launch_bounds__(256) void moe_logits_few_kernel(RouteArgs a) {
  const int lane = threadIdx.x & 63;
  const int e = (int)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  if (e >= a.num_experts) return;  // wave-uniform; no barrier in this kernel
  const int64_t t0 = (int64_t)blockIdx.y * T;
  const int k = a.k;
  const bool vec = a.vec != 0;
  const char *wr = (const char *)a.w + (size_t)e * a.ldw * (WF32 ? 4 : 2);
  const uint16_t *xr[T];
  double acc[T];
#pragma unroll
  for (int t = 0; t < T; ++t) {
    xr[t] = a.x + min(t0 + t, a.m - 1) * a.ldx;
    acc[t] = 0.0;
  }
  for (int c = 0; c < k; c += 512 * RT_CHUNKS) {
    RtRow<WF32> w[RT_CHUNKS];
    RtRow<false> x[RT_CHUNKS][T];
#pragma unroll
    for (int i = 0; i < RT_CHUNKS; ++i) w[i] = rt_load<WF32>(wr, c + 512 * i + 8 * lane, k, vec);
#pragma unroll
    for (int i = 0; i < RT_CHUNKS; ++i)
#pragma unroll
      for (int t = 0; t < T; ++t) x[i][t] = rt_load<false>(xr[t], c + 512 * i + 8 * lane, k, vec);
#pragma unroll
    for (int i = 0; i < RT_CHUNKS; ++i)
#pragma unroll
      for (int l = 0; l < 8; ++l) {
        const double wd = rt_get<WF32>(w[i], l);
#pragma unroll
        for (int t = 0; t < T; ++t) acc[t] = __builtin_fma(rt_get<false>(x[i][t], l), wd, acc[t]);
      }
  }
#pragma unroll
  for (int t = 0; t < T; ++t) {
    double v = acc[t];
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) v += shfl_xor_f64(v, d);
    if (lane == 0 && t0 + t < a.m) a.logits[(t0 + t) * a.num_experts + e] = v;
  }
}

// Many tokens: a block of W waves takes 16 N tokens x 16 N experts, each wave
// every W-th chunk of 32 channels through v_mfma_f64_16x16x4_f64 (element l
// of the eight channels a lane loads is one MFMA: its four k indices are
// channels 8g + l of the lane groups g), then the waves' tiles are summed in
// wave order.  One tile and 16 waves fill the chip from few tokens; 2 x 2
// tiles convert each value once for two MFMAs, for many.
typedef double d4 __attribute__((ext_vector_type(4)));
template <int N, int W, bool WF32>
__global__ __launch_bounds__(W * 64) void moe_logits_kernel(RouteArgs a) {
  __shared__ double s_red[W][N * N * 256];
  const int tid = threadIdx.x, lane = tid & 63, i = lane & 15, g = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int k = a.k, e0 = (int)blockIdx.x * 16 * N;
  const int64_t t0 = (int64_t)blockIdx.y * 16 * N;
  const bool vec = a.vec != 0;
  const uint16_t *xr[N];
  const char *wr[N];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    xr[n] = a.x + min(t0 + 16 * n + i, a.m - 1) * a.ldx;
    wr[n] = (const char *)a.w + (size_t)min(e0 + 16 * n + i, a.num_experts - 1) * a.ldw * (WF32 ? 4 : 2);
  }
  d4 c[N][N];
#pragma unroll
  for (int p = 0; p < N; ++p)
#pragma unroll
    for (int q = 0; q < N; ++q) c[p][q] = (d4){0.0, 0.0, 0.0, 0.0};
  constexpr int B = 4 / N;  // chunks in flight
  for (int c0 = 32 * wv; c0 < k; c0 += 32 * W * B) {
    RtRow<WF32> w[B][N];
    RtRow<false> x[B][N];
#pragma unroll
    for (int b = 0; b < B; ++b)
#pragma unroll
      for (int n = 0; n < N; ++n) {
        x[b][n] = rt_load<false>(xr[n], c0 + 32 * W * b + 8 * g, k, vec);
        w[b][n] = rt_load<WF32>(wr[n], c0 + 32 * W * b + 8 * g, k, vec);
      }
#pragma unroll
    for (int b = 0; b < B; ++b) {
      if (c0 + 32 * W * b >= k) break;  // wave-uniform
#pragma unroll
      for (int l = 0; l < 8; ++l) {
        double xd[N], wd[N];
#pragma unroll
        for (int n = 0; n < N; ++n) {
          xd[n] = rt_get<false>(x[b][n], l);
          wd[n] = rt_get<WF32>(w[b][n], l);
        }
#pragma unroll
        for (int p = 0; p < N; ++p)
#pragma unroll
          for (int q = 0; q < N; ++q) c[p][q] = __builtin_amdgcn_mfma_f64_16x16x4f64(xd[p], wd[q], c[p][q], 0, 0, 0);
      }
    }
  }
#pragma unroll
  for (int p = 0; p < N; ++p)
#pragma unroll
    for (int q = 0; q < N; ++q)
#pragma unroll
      for (int r = 0; r < 4; ++r) s_red[wv][(p * N + q) * 256 + 64 * r + lane] = c[p][q][r];
  __syncthreads();
  for (int o = tid; o < N * N * 256; o += W * 64) {
    double v = 0.0;
#pragma unroll
    for (int w = 0; w < W; ++w) v += s_red[w][o];
    // accumulator register r of lane 16 g + i: token g + 4 r, expert i
    const int64_t t = t0 + 16 * ((o >> 8) / N) + ((o >> 4) & 3) + 4 * ((o >> 6) & 3);
    const int e = e0 + 16 * ((o >> 8) % N) + (o & 15);
    if (t < a.m && e < a.num_experts) a.logits[t * a.num_experts + e] = v;
  }
}

// Order-preserving integer of a key: NaN below every number, -0 equal to +0.
__device__ __forceinline__ int64_t rt_order(double key) {
  if (key != key) return INT64_MIN + 1;
  const int64_t b = __builtin_bit_cast(int64_t, key + 0.0);
  return b >= 0 ? b : (b ^ INT64_MAX);
}

// The choice of one token: an expert's place is the number of experts before
// it (larger key, or equal key and lower index), so all places are found at
// once and no place waits for the one before.  Thread e of each part of the
// block counts a part of the experts for expert e; the first part holds the
// scores.  Four parts while all blocks are resident at once (one token:
// 3.4 us against 5.7 with one part; 512: 4.8 against 7.5), one beyond.
template <int TK_PARTS>
__global__ __launch_bounds__(TK_PARTS * MAX_EXPERTS) void moe_topk_kernel(RouteArgs a) {
  constexpr int W = MAX_EXPERTS / 64;
  __shared__ double s_mx[W], s_sum[W], s_p[ROUTE_MAX_TOPK];
  __shared__ int64_t s_key[MAX_EXPERTS];
  __shared__ int s_place[MAX_EXPERTS];
  const int e = threadIdx.x & (MAX_EXPERTS - 1), E = a.num_experts;
  const int part = __builtin_amdgcn_readfirstlane((int)threadIdx.x / MAX_EXPERTS);
  const int64_t t = blockIdx.x;
  const bool in = e < E, soft = a.score == SVQ_ROUTE_SOFTMAX;
  double l = 0.0, p = 0.0;
  if (part == 0) {
    l = in ? a.logits[t * E + e] : -INFINITY;
    s_place[e] = 0;
    if (soft) {
      double mx = l;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) mx = fmax(mx, shfl_xor_f64(mx, d));
      if ((e & 63) == 0) s_mx[e >> 6] = mx;
    } else {
      p = 1.0 / (1.0 + exp(-l));
    }
    if (!a.select_bias) s_key[e] = in ? rt_order(l) : INT64_MIN;
  }
  __syncthreads();
  if (part == 0 && soft) {
    double mx = s_mx[0];
#pragma unroll
    for (int w = 1; w < W; ++w) mx = fmax(mx, s_mx[w]);
    p = in ? exp(l - mx) : 0.0;
    double sum = p;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) sum += shfl_xor_f64(sum, d);
    if ((e & 63) == 0) s_sum[e >> 6] = sum;
  }
  if (a.select_bias) {  // keys need the scores
    __syncthreads();
    if (part == 0) {
      double sum = 0.0;
#pragma unroll
      for (int w = 0; w < W; ++w) sum += s_sum[w];
      const double q = soft ? p / sum : p;
      s_key[e] = in ? rt_order(q + (double)a.select_bias[e]) : INT64_MIN;
    }
    __syncthreads();
  }
  if (in) {
    const int64_t key = s_key[e];
    const int per = (E + TK_PARTS - 1) / TK_PARTS, j0 = part * per, j1 = min(E, j0 + per);
    int before = 0;
#pragma unroll 8
    for (int j = j0; j < j1; ++j) {
      const int64_t other = s_key[j];
      before += other > key || (other == key && j < e) ? 1 : 0;
    }
    if (before) atomicAdd(&s_place[e], before);
  }
  __syncthreads();
  const int place = s_place[e];
  if (part == 0 && in && place < a.topk) {
    double sum = 1.0;
    if (soft) {
      sum = 0.0;
#pragma unroll
      for (int w = 0; w < W; ++w) sum += s_sum[w];
    }
    a.ids[t * a.topk + place] = e;
    s_p[place] = p / sum;
  }
  __syncthreads();
  if (part == 0 && e < a.topk) {
    double v = s_p[e];
    if (a.renormalize) {
      double total = 0.0;
      for (int j = 0; j < a.topk; ++j) total += s_p[j];
      v /= total;
    }
    a.weights[t * a.topk + e] = (float)(v * (double)a.scale);
  }
}

template <int N, int W, bool WF32>
static void launch_logit_tiles(const RouteArgs &a, hipStream_t s) {
  hipLaunchKernelGGL((moe_logits_kernel<N, W, WF32>),
                     dim3((unsigned)((a.num_experts + 16 * N - 1) / (16 * N)), (unsigned)((a.m + 16 * N - 1) / (16 * N))),
                     dim3(W * 64), 0, s, a);
}
template <bool WF32>
static void launch_logits(const RouteArgs &a, int cus, hipStream_t s) {
  const unsigned eb = (unsigned)((a.num_experts + 3) / 4);
  if (a.m == 1)
    hipLaunchKernelGGL((moe_logits_few_kernel<1, WF32>), dim3(eb), dim3(256), 0, s, a);
  else if (a.m <= ROUTE_FEW)
    hipLaunchKernelGGL((moe_logits_few_kernel<RT_TOKENS, WF32>),
                       dim3(eb, (unsigned)((a.m + RT_TOKENS - 1) / RT_TOKENS)), dim3(256), 0, s, a);
  else if ((a.m + 31) / 32 * ((a.num_experts + 31) / 32) < cus)  // one 2 x 2 block per compute unit at least
    launch_logit_tiles<1, 16, WF32>(a, s);
  else
    launch_logit_tiles<2, 8, WF32>(a, s);
}

hipError_t launch_route(const RouteArgs &a, int cus, hipStream_t s) {
  if (a.w_f32) launch_logits<true>(a, cus, s);
  else launch_logits<false>(a, cus, s);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (a.m <= 2 * (int64_t)cus)
    hipLaunchKernelGGL(moe_topk_kernel<4>, dim3((unsigned)a.m), dim3(4 * MAX_EXPERTS), 0, s, a);
  else
    hipLaunchKernelGGL(moe_topk_kernel<1>, dim3((unsigned)a.m), dim3(MAX_EXPERTS), 0, s, a);
  return hipGetLastError();
}

}  // namespace svq
