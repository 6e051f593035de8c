// Small-batch dequant path of libsvq (EXACT_MAX_M < m <= SB_MAX_M) for
// gfx950.
//
// Method: "SAGE: Pushing 2-Bit Vector-Quantized LLMs toward Real-World
// Usability".  A weight subvector is rebuilt on demand from its sign bits,
// direction index and radius index (Fig. 2 caption) inside the product
// (Fig. 1 / Fig. 5 captions) with the subvector's eight reordered
// activations (Fig. 6 caption).  The decoded weight R * D is never rounded:
// the matrix's 1024-row fp16 table (one row per 10-bit direction/radius
// index, built by svq_pack) holds hi and lo with hi + lo = R * D * 2^s
// exactly, and both halves, with the code's signs, are MFMA operands
// against the same fp16 activations (a power-of-two scale per activation
// row and unit, as in the m <= 4 path), so products and their sum are exact
// in the fp32 accumulators; 2^-s and the activation scales are applied to
// the fp32 sums.
//
// At a few activation rows the product is still bound by the code stream
// and by the per-code decode, not by the matrix cores, so the decoded
// weights never go through LDS: one code decodes to exactly two B operands
// of v_mfma_f32_16x16x32_f16 (8 consecutive k of one output column, hi and
// lo), in the lane that loaded it.
//
// 16x16x32 operands: lane L holds A row L & 15 and B column L & 15, both for
// k = 8(L >> 4)..+7; accumulator element i of lane L is row 4(L >> 4) + i,
// column L & 15.  With A = activations (row = activation row m) and
// B = weights (column = output row n of the 16-row tile) one MFMA covers one
// code of each of the 16 rows for four code columns.
//
// Code mapping.  The unit layout (svq_internal.h) gives lane 4b + j the
// codes 4ri + ci at row 4ri + j, code column 16ci + b.  The MFMA needs the
// 16 lanes of each k slice to hold one code column, so here lane
// L = 16s + 4b0 + j takes, for MFMA f = 4ci + q, the code at row 4b0 + j,
// column 16ci + 4s + q: code 4b0 + ci of lane record 16s + 4q + j.  It loads
// those records' bytes directly (for each q: the record's 16 sign bytes, the
// index-low dword b0 and the index-high dword), so no data moves between
// lanes; every byte of the unit is still fetched once per wave (lanes that
// share a record share the address).
//
// Activations: a prep launch writes every matrix's permuted activations in
// fragment order, unit by unit: 16 fragments of 1 KB (f = 4ci + q), lane L's
// 16 bytes = activation row L & 15 at the eight slots of code column
// 16ci + 4(L >> 4) + q, in fp16 after the row's power-of-two scale for the
// unit (largest magnitude scaled into [2^14, 2^15)).  A wave loads the 16
// fragments of its unit once (64 VGPRs) with the unit's inverse scales of
// its four accumulator rows, and reuses them for every row tile it covers.
//
// Work split.  A work item is one coded unit of one row tile.  A block of
// 4 waves owns up to SB_TMAX consecutive row tiles and a K range of units
// (the whole K unless the matrix has more than SB_MAX_RANGE units); its
// items, ordered unit by unit, are cut into 4 contiguous runs of at most
// SB_NMAX items, one per wave, so a wave reloads its activation fragments
// only when its run crosses to the next unit.  A wave streams its run with
// the codes of the next two items in flight and adds each item's 16 x 16
// result into its own LDS slot for the item's tile; after one barrier the
// block sums the four waves' slots in wave order.  For a matrix cut into K
// ranges the block writes fp32 partial tiles, and the last block of a tile
// group to arrive (an arrival counter, cleared by the prep launch) adds
// them in range order and writes the output, so results do not depend on
// timing.
#include <type_traits>

#include "svq_device.h"
#include "svq_epilogue.h"
#include "../../include/svq.h"

namespace svq {

typedef __attribute__((address_space(3))) const u4 sb_lds_u4_t;

// LDS (absolute addresses; these kernels declare no static LDS): the fp16
// split table at 0, then the per-wave tile results, then the arrival flag.
constexpr int SB_OFF_XTAB = 0;
constexpr int SB_OFF_RED = XTAB_BYTES;
constexpr int SB_RED_BYTES = SB_WAVES * SB_TMAX * 1024;
constexpr int SB_OFF_FLAG = SB_OFF_RED + SB_RED_BYTES;
constexpr int SB_SMEM = SB_OFF_FLAG + 16;
static_assert(SB_SMEM <= 64 * 1024, "small-batch LDS");

__device__ __forceinline__ u4 sb_lds(uint32_t addr) { return *(sb_lds_u4_t *)(size_t)addr; }

// Table rows of the four codes (ci = 0..3) of MFMA group q: the hi and lo
// halves of each code's exact split (32-byte rows by 10-bit index).  HI: the
// high halves alone, RNE_fp16(R*D*2^s), 16-byte rows.
// TAB: LDS address of the table.
template <bool HI, int TAB = SB_OFF_XTAB>
__device__ __forceinline__ void sb_reads(uint32_t Lw, uint32_t H, const SbShifts &sh, u4 (&Dh)[4],
                                         u4 (&Dl)[4]) {
#pragma unroll
  for (int ci = 0; ci < 4; ++ci) {
    const uint32_t lo = __builtin_amdgcn_ubfe(Lw, 8 * ci, 8);
    const uint32_t hi = __builtin_amdgcn_ubfe(H, sh.hi[ci], 2);
    const uint32_t a = TAB + ((lo | (hi << 8)) << (HI ? 4 : 5));
    Dh[ci] = sb_lds(a);
    Dl[ci] = HI ? Dh[ci] : sb_lds(a + 16);
  }
}

// Packed fp16 values with infinities (and NaN) as zeros.
__device__ __forceinline__ u4 sb_finite(const u4 &a) {
  u4 r;
#pragma unroll
  for (int l = 0; l < 4; ++l) {
    const uint32_t lo = a[l] & 0xFFFFu, hi = a[l] & 0xFFFF0000u;
    r[l] = ((lo & 0x7C00u) == 0x7C00u ? 0u : lo) | ((hi & 0x7C000000u) == 0x7C000000u ? 0u : hi);
  }
  return r;
}

// Signs of the four codes of group q, then their MFMAs.  A 64-bit shift of
// the record's sign dwords (S1:S0, S3:S2) by 4b0 + ci brings code
// 4b0 + ci's pair signs to bits 15 and 31 of each dword (bits the shift
// carries across the dword boundary land below bit 15 and are masked off).
// FIN: the low halves meet finite activations only (see sb_redo).
template <bool HI, bool FIN>
__device__ __forceinline__ void sb_mul(uint64_t S01, uint64_t S23, const SbShifts &sh,
                                       const u4 (&Dh)[4], const u4 (&Dl)[4], const u4 (&A)[16], int q,
                                       f4 &C) {
  const uint32_t SM = 0x80008000u;
#pragma unroll
  for (int ci = 0; ci < 4; ++ci) {
    const uint64_t c01 = S01 << sh.sg[ci], c23 = S23 << sh.sg[ci];
    const uint32_t m0 = (uint32_t)c01 & SM, m1 = (uint32_t)(c01 >> 32) & SM;
    const uint32_t m2 = (uint32_t)c23 & SM, m3 = (uint32_t)(c23 >> 32) & SM;
    const u4 wh = {Dh[ci][0] ^ m0, Dh[ci][1] ^ m1, Dh[ci][2] ^ m2, Dh[ci][3] ^ m3};
    const u4 wl = {Dl[ci][0] ^ m0, Dl[ci][1] ^ m1, Dl[ci][2] ^ m2, Dl[ci][3] ^ m3};  // HI: unused
    const h8 a = __builtin_bit_cast(h8, A[4 * ci + q]);
    C = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, __builtin_bit_cast(h8, wh), C, 0, 0, 0);
    if constexpr (!HI) {
      const h8 al = FIN ? __builtin_bit_cast(h8, sb_finite(A[4 * ci + q])) : a;
      C = __builtin_amdgcn_mfma_f32_16x16x32_f16(al, __builtin_bit_cast(h8, wl), C, 0, 0, 0);
    }
  }
}

// One unit of one row tile: the 16 codes of the lane, 16 MFMAs.
template <bool HI, int TAB = SB_OFF_XTAB, bool FIN = false>
__device__ __forceinline__ f4 sb_item(const SbCodes &c, const u4 (&A)[16], const SbShifts &sh) {
  f4 C0 = {0.f, 0.f, 0.f, 0.f}, C1 = {0.f, 0.f, 0.f, 0.f};
  u4 H0[4], L0[4], H1[4], L1[4];
  auto s01 = [&](int q) { return (uint64_t)c.S[q][0] | ((uint64_t)c.S[q][1] << 32); };
  auto s23 = [&](int q) { return (uint64_t)c.S[q][2] | ((uint64_t)c.S[q][3] << 32); };
  // the table reads of group q + 1 are in flight while group q is multiplied
  sb_reads<HI, TAB>(c.L[0], c.H[0], sh, H0, L0);
  sb_reads<HI, TAB>(c.L[1], c.H[1], sh, H1, L1);
  __builtin_amdgcn_sched_barrier(0);
  sb_mul<HI, FIN>(s01(0), s23(0), sh, H0, L0, A, 0, C0);
  __builtin_amdgcn_sched_barrier(0);
  sb_reads<HI, TAB>(c.L[2], c.H[2], sh, H0, L0);
  __builtin_amdgcn_sched_barrier(0);
  sb_mul<HI, FIN>(s01(1), s23(1), sh, H1, L1, A, 1, C1);
  __builtin_amdgcn_sched_barrier(0);
  sb_reads<HI, TAB>(c.L[3], c.H[3], sh, H1, L1);
  __builtin_amdgcn_sched_barrier(0);
  sb_mul<HI, FIN>(s01(2), s23(2), sh, H0, L0, A, 2, C0);
  __builtin_amdgcn_sched_barrier(0);
  sb_mul<HI, FIN>(s01(3), s23(3), sh, H1, L1, A, 3, C1);
  return C0 + C1;
}

typedef __attribute__((address_space(3))) u4 sb_lds_u4w_t;
typedef __attribute__((address_space(3))) float sb_lds_f_t;
typedef __attribute__((address_space(3))) int sb_lds_i_t;

__device__ __forceinline__ const uint8_t *sb_unit(const MatView &w, int t, int u) {
  return w.base + w.off_codes + ((size_t)t * w.units + u) * UNIT_BYTES;
}

// A unit that holds an infinity in some row has its scales stored negative.
__device__ __forceinline__ f4 sb_scales(const f4 &xs) {
  return (f4){fabsf(xs[0]), fabsf(xs[1]), fabsf(xs[2]), fabsf(xs[3])};
}
// A wave's run once more, for a run that met such a unit.  A code's weight is
// the sum of two halves, and an infinite activation times the low one is NaN
// (where it is zero) or of the wrong sign; here the low halves are multiplied
// by the finite activations alone (the infinity times the high half is the
// product's own value).  Items one at a time and not unrolled: run after the
// loop, which then carries nothing for it but the marks.  (As a branch in the
// unrolled loop, whose code it doubled, the seven matrices of a layer took
// 29.4 us at 16 rows, 28.1 this way.)  Same order of items: rows without an
// infinity get the sums they had.
template <int TAB>
__device__ __forceinline__ void sb_redo(const MatView &w, const uint8_t *xa_all, const float *xs, int t0, int u0,
                                        int tn, int i0, int nk, const SbOffs &offs, const SbShifts &sh,
                                        uint32_t slot0, int lane) {
#pragma unroll
  for (int t = 0; t < SB_TMAX; ++t) *(sb_lds_u4w_t *)(size_t)(slot0 + t * 1024) = (u4){0u, 0u, 0u, 0u};
#pragma unroll 1
  for (int i = i0; i < i0 + nk; ++i) {
    const int ui = i / tn, ti = i - ui * tn, u = u0 + ui;
    const u4 *xa = (const u4 *)(xa_all + (size_t)u * SB_XA_UNIT_BYTES) + lane;
    u4 A[16];
#pragma unroll
    for (int f = 0; f < 16; ++f) A[f] = xa[64 * f];
    const f4 xsc = sb_scales(*(const f4 *)(xs + (size_t)u * 16 + 4 * (lane >> 4)));
    const f4 C = sb_item<false, TAB, true>(sb_load_codes(sb_unit(w, t0 + ti, u), offs), A, sh) * xsc;
    sb_lds_u4w_t *sl = (sb_lds_u4w_t *)(size_t)(slot0 + ti * 1024);
    *sl = __builtin_bit_cast(u4, __builtin_bit_cast(f4, *sl) + C);
  }
}

// ea: nothing, the EpiArgs of a single matrix, or the PairArgs of a gated
// pair (jobs 0 and 1, equal plans): then every block leaves its sums, times
// its matrix's 2^-s, as a range of its own (the gate's ranges first), and the
// last of all to arrive finishes the pair.  (The body stands in the
// kernel itself: behind a function call the job records, indexed at run time,
// would be copied out of the kernel arguments.)
// HI: with the weights' high halves only (RNE_fp16, 2^-11 of a weight at most,
// an eighth of a bf16 output's own half step; for calls that round to bf16,
// whose relative error against 64 bits, 0.0017 in 2-norm for a gated pair of
// 13 rows of 9728 x 2560, is that of exact weights in fp32 too).
// Half the table reads, which bound the loop, and half the MFMAs.
template <bool HI, typename... EA>
__global__ __launch_bounds__(256) void sb_gemm_kernel(SbBatch b, EA... ea) {
  const auto epi = make_epi(ea...);
  const int jn = find_job(b.starts, b.count);
  const SbJob &J = b.job[jn];
  const MatView &w = J.w;
  const int lb = (int)blockIdx.x - J.block_begin;
  const int g = lb / J.splits, r = lb - g * J.splits;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int t0 = g * J.tiles, tn = min(J.tiles, w.n_tiles - t0);
  const int u0 = r * J.upr, ul = min(J.upr, w.units - u0);
  // this wave's run: items [i0, i0 + nk) of the block, item i = unit
  // u0 + i / tn, tile t0 + i % tn
  const int N = ul * tn;
  const int i0 = wv * N / SB_WAVES, nk = (wv + 1) * N / SB_WAVES - i0;
  const uint32_t s = lane >> 4, b0 = (lane >> 2) & 3, j = lane & 3;
  const uint32_t rec0 = 16 * s + j;
  const SbOffs offs = {16 * rec0, 16 * rec0 + 4 * b0, 4 * rec0};
  SbShifts sh;
#pragma unroll
  for (int ci = 0; ci < 4; ++ci) {
    sh.sg[ci] = 4 * b0 + ci;
    sh.hi[ci] = 8 * b0 + 2 * ci;
  }
  const uint32_t slot0 = SB_OFF_RED + wv * SB_TMAX * 1024 + 16 * lane;

  // the bf16 table (requested first), the activation fragments of the
  // run's first unit and the codes of its first two items
  constexpr int NBT = XTAB_BYTES / 4096 / (HI ? 2 : 1);
  u4 bt[NBT];
  const u4 *gbt = (const u4 *)(w.base + w.off_xtab);
#pragma unroll
  for (int i = 0; i < NBT; ++i) bt[i] = gbt[HI ? 2 * (tid + 256 * i) : tid + 256 * i];
  __builtin_amdgcn_sched_barrier(0);
  u4 A[16];
  f4 xsc;  // inverse activation scales of the lane's accumulator rows 4s..4s+3
  SbCodes cd[2];
  int ui = i0 / tn, ti = i0 - ui * tn;  // unit and tile of item k (relative)
  {
    // unconditional (a wave without items loads item i0 < N anyway), so
    // that only the table loads are waited for before the barrier
    const u4 *xa = (const u4 *)(J.xa + (size_t)(u0 + ui) * SB_XA_UNIT_BYTES) + lane;
#pragma unroll
    for (int f = 0; f < 16; ++f) A[f] = xa[64 * f];
    xsc = *(const f4 *)(J.xs + (size_t)(u0 + ui) * 16 + 4 * s);
    cd[0] = sb_load_codes(sb_unit(w, t0 + ti, u0 + ui), offs);
    const int i1 = min(i0 + 1, N - 1), u1 = i1 / tn;
    cd[1] = sb_load_codes(sb_unit(w, t0 + i1 - u1 * tn, u0 + u1), offs);
  }
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int t = 0; t < SB_TMAX; ++t)
    *(sb_lds_u4w_t *)(size_t)(slot0 + t * 1024) = (u4){0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < NBT; ++i)
    *(sb_lds_u4w_t *)(size_t)(SB_OFF_XTAB + 16 * (tid + 256 * i)) = bt[i];
  __syncthreads();

  int marks = 0;  // negative once a unit held an infinity
#pragma unroll
  for (int k = 0; k < SB_NMAX; ++k) {
    if (k >= nk) break;
    if (k > 0 && ti == 0) {
      // the run enters the next unit
      const u4 *xa = (const u4 *)(J.xa + (size_t)(u0 + ui) * SB_XA_UNIT_BYTES) + lane;
#pragma unroll
      for (int f = 0; f < 16; ++f) A[f] = xa[64 * f];
      xsc = *(const f4 *)(J.xs + (size_t)(u0 + ui) * 16 + 4 * s);
    }
    const f4 C = sb_item<HI>(cd[k & 1], A, sh) * sb_scales(xsc);
    if constexpr (!HI) marks |= __builtin_bit_cast(int, xsc[0]);
    if (k + 2 < nk) {
      const int i2 = i0 + k + 2, u2 = i2 / tn;
      cd[k & 1] = sb_load_codes(sb_unit(w, t0 + i2 - u2 * tn, u0 + u2), offs);
    }
    sb_lds_u4w_t *sl = (sb_lds_u4w_t *)(size_t)(slot0 + ti * 1024);
    *sl = __builtin_bit_cast(u4, __builtin_bit_cast(f4, *sl) + C);
    if (++ti == tn) {
      ti = 0;
      ++ui;
    }
  }
  if (!HI && __builtin_expect(__builtin_amdgcn_readfirstlane(marks) < 0, 0))
    sb_redo<SB_OFF_XTAB>(w, J.xa, J.xs, t0, u0, tn, i0, nk, offs, sh, slot0, lane);
  __syncthreads();

  // sum of the four waves' slots of each tile, in wave order.  Thread tid
  // takes output row n = tid & 15 of the tile for activation row
  // m = tid >> 4: accumulator element m & 3 of lane 16(m >> 2) + n.
  const int m = tid >> 4, nn = tid & 15;
  const uint32_t eoff = SB_OFF_RED + 256 * (m >> 2) + 16 * nn + 4 * (m & 3);
  float acc[SB_TMAX];
#pragma unroll
  for (int t = 0; t < SB_TMAX; ++t) {
    acc[t] = 0.f;
#pragma unroll
    for (int ww = 0; ww < SB_WAVES; ++ww)
      acc[t] += *(sb_lds_f_t *)(size_t)(eoff + (ww * SB_TMAX + t) * 1024);
  }
  constexpr bool pair = std::is_same_v<decltype(make_epi(ea...)), PairEpi>;
  if constexpr (pair) {
    const int total = 2 * J.splits, own = jn * J.splits + r;
    float *pt = epi.a.part + ((size_t)t0 * total + own) * 256 + tid;
#pragma unroll
    for (int t = 0; t < SB_TMAX; ++t)
      if (t < tn)
        __hip_atomic_store(pt + (size_t)t * total * 256, acc[t] * J.xinv, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (tid == 0) {
      const int prev = __hip_atomic_fetch_add(epi.a.cnt + g, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      *(sb_lds_i_t *)(size_t)SB_OFF_FLAG = prev == total - 1 ? 1 : 0;
    }
    __syncthreads();
    if (*(sb_lds_i_t *)(size_t)SB_OFF_FLAG == 0) return;
    const float *pa = epi.a.part + (size_t)t0 * total * 256 + tid;
    float up[SB_TMAX];
#pragma unroll
    for (int t = 0; t < SB_TMAX; ++t) acc[t] = up[t] = 0.f;
    for (int r0 = 0; r0 < J.splits; r0 += 4) {
      float vg[SB_TMAX][4], vu[SB_TMAX][4];
#pragma unroll
      for (int t = 0; t < SB_TMAX; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float *q = pa + ((size_t)min(t, tn - 1) * total + min(r0 + e, J.splits - 1)) * 256;
          vg[t][e] = __hip_atomic_load(q, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
          vu[t][e] = __hip_atomic_load(q + (size_t)J.splits * 256, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
#pragma unroll
      for (int t = 0; t < SB_TMAX; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (r0 + e < J.splits) {
            acc[t] += vg[t][e];
            up[t] += vu[t][e];
          }
    }
    if (m >= b.m) return;
#pragma unroll
    for (int t = 0; t < SB_TMAX; ++t) {
      const int n = (t0 + t) * UNIT_ROWS + nn;
      if (t < tn && n < w.n) store_out(J.y, (size_t)m * J.ldy + n, pair_value(epi.a, acc[t], up[t], n), b.ydt);
    }
    return;
  }
  if (J.splits > 1) {
    // Partial tiles for the range, then the arrival count of the group.
    // The partials are written and read as device-scope atomics (coherent
    // between the XCDs' L2 caches without writing back or invalidating
    // them, which a device-scope fence does), and every partial store has
    // completed (vmcnt 0, then the barrier) before the count is raised.
    float *pt = J.part + ((size_t)t0 * J.splits + r) * 256 + tid;
#pragma unroll
    for (int t = 0; t < SB_TMAX; ++t)
      if (t < tn)
        __hip_atomic_store(pt + (size_t)t * J.splits * 256, acc[t], __ATOMIC_RELAXED,
                           __HIP_MEMORY_SCOPE_AGENT);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (tid == 0) {
      const int prev = __hip_atomic_fetch_add(J.cnt + g, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      *(sb_lds_i_t *)(size_t)SB_OFF_FLAG = prev == J.splits - 1 ? 1 : 0;
    }
    __syncthreads();
    if (*(sb_lds_i_t *)(size_t)SB_OFF_FLAG == 0) return;
    // all partials of a batch of 8 ranges are requested before any is added
    const float *pa = J.part + (size_t)t0 * J.splits * 256 + tid;
#pragma unroll
    for (int t = 0; t < SB_TMAX; ++t) acc[t] = 0.f;
    for (int r0 = 0; r0 < J.splits; r0 += 8) {
      float v[SB_TMAX][8];
#pragma unroll
      for (int t = 0; t < SB_TMAX; ++t)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int rr = min(r0 + e, J.splits - 1), tt = min(t, tn - 1);
          v[t][e] = __hip_atomic_load(pa + ((size_t)tt * J.splits + rr) * 256, __ATOMIC_RELAXED,
                                      __HIP_MEMORY_SCOPE_AGENT);
        }
#pragma unroll
      for (int t = 0; t < SB_TMAX; ++t)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (r0 + e < J.splits) acc[t] += v[t][e];
    }
  }
  if (m >= b.m) return;
#pragma unroll
  for (int t = 0; t < SB_TMAX; ++t) {
    const int n = (t0 + t) * UNIT_ROWS + nn;
    if (t < tn && n < w.n) store_out(J.y, (size_t)m * J.ldy + n, epi(acc[t] * J.xinv, m, n), b.ydt);
  }
  (void)j;
}

// ---------------------------------------------------------------------------
// Gated pair without K ranges: both matrices of the same row tiles in one
// block of 8 waves, 0..3 on the gate's and 4..7 on the up matrix's, each half
// with its own table and partial sums in its part of LDS (what two blocks of
// the kernel above hold), so the pair meets in LDS.  (Through memory, as
// above, the exchange and its arrival cost 3 of 14 us.)
// ---------------------------------------------------------------------------
template <bool HI>
constexpr int sb_half_bytes() { return XTAB_BYTES / (HI ? 2 : 1) + SB_RED_BYTES; }

// One half's sums: thread (tid & 255) returns acc[t] of row tile t, activation
// row (tid & 255) >> 4, output row tid & 15, as the kernel above.
template <bool HI, int HB>
__device__ __forceinline__ void sb_pair_half(const SbJob &J, int g, float (&acc)[SB_TMAX]) {
  constexpr int OFF_TAB = HB, OFF_RED = HB + XTAB_BYTES / (HI ? 2 : 1), NBT = XTAB_BYTES / 4096 / (HI ? 2 : 1);
  const MatView &w = J.w;
  const int tid = threadIdx.x & 255, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int t0 = g * J.tiles, tn = min(J.tiles, w.n_tiles - t0);
  const int N = w.units * tn;
  const int i0 = wv * N / SB_WAVES, nk = (wv + 1) * N / SB_WAVES - i0;
  const uint32_t s = lane >> 4, b0 = (lane >> 2) & 3, j = lane & 3;
  const uint32_t rec0 = 16 * s + j;
  const SbOffs offs = {16 * rec0, 16 * rec0 + 4 * b0, 4 * rec0};
  SbShifts sh;
#pragma unroll
  for (int ci = 0; ci < 4; ++ci) {
    sh.sg[ci] = 4 * b0 + ci;
    sh.hi[ci] = 8 * b0 + 2 * ci;
  }
  const uint32_t slot0 = OFF_RED + wv * SB_TMAX * 1024 + 16 * lane;
  u4 bt[NBT];
  const u4 *gbt = (const u4 *)(w.base + w.off_xtab);
#pragma unroll
  for (int i = 0; i < NBT; ++i) bt[i] = gbt[HI ? 2 * (tid + 256 * i) : tid + 256 * i];
  __builtin_amdgcn_sched_barrier(0);
  u4 A[16];
  f4 xsc;
  SbCodes cd[2];
  int ui = i0 / tn, ti = i0 - ui * tn;
  auto load_unit = [&](int u) __attribute__((always_inline)) {
    const u4 *xa = (const u4 *)(J.xa + (size_t)u * SB_XA_UNIT_BYTES) + lane;
#pragma unroll
    for (int f = 0; f < 16; ++f) A[f] = xa[64 * f];
    xsc = *(const f4 *)(J.xs + (size_t)u * 16 + 4 * s);
  };
  auto codes_of = [&](int i) __attribute__((always_inline)) {
    const int u = i / tn;
    return sb_load_codes(sb_unit(w, t0 + i - u * tn, u), offs);
  };
  // unconditional (a wave without items loads item i0 < N anyway)
  load_unit(ui);
  cd[0] = codes_of(i0);
  cd[1] = codes_of(min(i0 + 1, N - 1));
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int t = 0; t < SB_TMAX; ++t) *(sb_lds_u4w_t *)(size_t)(slot0 + t * 1024) = (u4){0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < NBT; ++i) *(sb_lds_u4w_t *)(size_t)(OFF_TAB + 16 * (tid + 256 * i)) = bt[i];
  __syncthreads();
  int marks = 0;  // negative once a unit held an infinity
#pragma unroll
  for (int k = 0; k < SB_NMAX; ++k) {
    if (k >= nk) break;
    if (k > 0 && ti == 0) load_unit(ui);
    const f4 C = sb_item<HI, OFF_TAB>(cd[k & 1], A, sh) * sb_scales(xsc);
    if constexpr (!HI) marks |= __builtin_bit_cast(int, xsc[0]);
    if (k + 2 < nk) cd[k & 1] = codes_of(i0 + k + 2);
    sb_lds_u4w_t *sl = (sb_lds_u4w_t *)(size_t)(slot0 + ti * 1024);
    *sl = __builtin_bit_cast(u4, __builtin_bit_cast(f4, *sl) + C);
    if (++ti == tn) {
      ti = 0;
      ++ui;
    }
  }
  if (!HI && __builtin_expect(__builtin_amdgcn_readfirstlane(marks) < 0, 0))
    sb_redo<OFF_TAB>(w, J.xa, J.xs, t0, 0, tn, i0, nk, offs, sh, slot0, lane);
  __syncthreads();
  const int m = tid >> 4, nn = tid & 15;
  const uint32_t eoff = OFF_RED + 256 * (m >> 2) + 16 * nn + 4 * (m & 3);
#pragma unroll
  for (int t = 0; t < SB_TMAX; ++t) {
    acc[t] = 0.f;
#pragma unroll
    for (int ww = 0; ww < SB_WAVES; ++ww) acc[t] += *(sb_lds_f_t *)(size_t)(eoff + (ww * SB_TMAX + t) * 1024);
    acc[t] *= J.xinv;
  }
}

template <bool HI>
__global__ __launch_bounds__(512) void sb_pair_kernel(SbBatch b, PairArgs pa) {
  constexpr int HB = sb_half_bytes<HI>();
  const int g = blockIdx.x, tid = threadIdx.x & 255;
  float acc[SB_TMAX];
  const bool up = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 8) != 0;
  if (!up) sb_pair_half<HI, 0>(b.job[0], g, acc);
  else sb_pair_half<HI, HB>(b.job[1], g, acc);
  // the up half's sums to the gate's threads, over the up half's table (no
  // wave reads it any more)
  if (up) {
#pragma unroll
    for (int t = 0; t < SB_TMAX; ++t) *(sb_lds_f_t *)(size_t)(HB + (t * 256 + tid) * 4) = acc[t];
  }
  __syncthreads();
  const SbJob &J = b.job[0];
  const int m = tid >> 4, t0 = g * J.tiles, tn = min(J.tiles, J.w.n_tiles - t0);
  if (up || m >= b.m) return;
#pragma unroll
  for (int t = 0; t < SB_TMAX; ++t) {
    const int n = (t0 + t) * UNIT_ROWS + (tid & 15);
    if (t < tn && n < J.w.n)
      store_out(J.y, (size_t)m * J.ldy + n, pair_value(pa, acc[t], *(sb_lds_f_t *)(size_t)(HB + (t * 256 + tid) * 4), n),
                b.ydt);
  }
}
static_assert(2 * sb_half_bytes<false>() <= (int)GV_LDS_LIMIT, "both halves of a block in LDS");
static_assert(SB_TMAX * 256 * 4 <= XTAB_BYTES / 2, "the up sums fit over its table");

// Row maximum of the preps below over a block's waves: the lanes of one row
// (m, m + 16, m + 32, m + 48), then the waves.
template <bool AGAIN>
__device__ __forceinline__ float sb_row_max(float mx, float (&s_max)[4][16], int wv, int L) {
  mx = fmaxf(mx, __shfl_xor(mx, 16));
  mx = fmaxf(mx, __shfl_xor(mx, 32));
  if (AGAIN) __syncthreads();  // the first call's maxima are read
  if (L < 16) s_max[wv][L] = mx;
  __syncthreads();
  const int m = L & 15;
  return fmaxf(fmaxf(s_max[0][m], s_max[1][m]), fmaxf(s_max[2][m], s_max[3][m]));
}
// The lane's largest finite magnitude (the rare second look at a unit that
// holds an infinity).
__device__ __forceinline__ float sb_finite_max(const float (&v)[4][8]) {
  float mx = 0.f;
#pragma unroll
  for (int ff = 0; ff < 4; ++ff)
#pragma unroll
    for (int l = 0; l < 8; ++l) mx = fmaxf(mx, finite_mag(v[ff][l]));
  return mx;
}

// Prep: the permuted activations of every job in fragment order (see the
// file comment), rows >= m and slots >= k zero; block u of a job writes the
// 16 fragments of unit u, thread tid the 16-byte pieces of fragments
// 4 (tid >> 6) .. + 3 for lane tid & 63 (activation row tid & 15).  Each
// activation row's largest magnitude over the unit (512 slots) sets its
// power-of-two scale 2^e (max * 2^e in [2^14, 2^15)): a bf16 value of at
// least 2^-31 times the maximum is then exact in fp16.  2^-e goes to
// xs[16u + row].  The maximum is over the finite values: infinities and NaN
// keep theirs; a unit that holds an infinity in any row is marked by negative
// scales (see sb_redo).  The first block of a job also clears the
// job's arrival counters.
__global__ __launch_bounds__(256) void sb_prep_kernel(SbBatch b) {
  __shared__ float s_max[4][16];
  const int jn = find_job(b.prep_starts, b.count);
  const SbJob &J = b.job[jn];
  const MatView &w = J.w;
  const int u = (int)blockIdx.x - J.prep_begin;
  const int tid = threadIdx.x, wv = tid >> 6, L = tid & 63;
  if (u == 0 && J.cnt)
    for (int i = tid; i < J.groups; i += 256) J.cnt[i] = 0;
  const int m = L & 15, s = L >> 4;
  float v[4][8];
  float mx = 0.f;
#pragma unroll
  for (int ff = 0; ff < 4; ++ff) {
    const int f = 4 * wv + ff, ci = f >> 2, q = f & 3;
    const int p0 = u * UNIT_SLOTS + 8 * (16 * ci + 4 * s + q);
#pragma unroll
    for (int l = 0; l < 8; ++l) v[ff][l] = 0.f;
    if (m < b.m && p0 < w.k) {
      // perm is zero padded to the unit width, so every index is < k
      const u4 pv = *(const u4 *)(w.base + w.off_perm + 2 * (size_t)p0);
      const uint16_t *xr = J.x + (int64_t)m * J.ldx;
#pragma unroll
      for (int l = 0; l < 4; ++l) {
        const float lo = bf16_bits_to_f32(xr[pv[l] & 0xFFFFu]), hi = bf16_bits_to_f32(xr[pv[l] >> 16]);
        v[ff][2 * l] = p0 + 2 * l < w.k ? lo : 0.f;
        v[ff][2 * l + 1] = p0 + 2 * l + 1 < w.k ? hi : 0.f;
      }
    }
#pragma unroll
    for (int l = 0; l < 8; ++l) mx = fmaxf(mx, fabsf(v[ff][l]));
  }
  mx = sb_row_max<false>(mx, s_max, wv, L);
  const bool inf = __any(mx == __builtin_inff());  // of any row: the same in every wave
  if (__builtin_expect(inf, 0)) mx = sb_row_max<true>(sb_finite_max(v), s_max, wv, L);
  const int e = mx > 0.f ? 15 - __builtin_amdgcn_frexp_expf(mx) : 0;
#pragma unroll
  for (int ff = 0; ff < 4; ++ff) {
    const int f = 4 * wv + ff;
    u4 h;
#pragma unroll
    for (int l = 0; l < 4; ++l) {
      const _Float16 lo = (_Float16)ldexpf(v[ff][2 * l], e), hi = (_Float16)ldexpf(v[ff][2 * l + 1], e);
      h[l] = (uint32_t)__builtin_bit_cast(uint16_t, lo) | ((uint32_t)__builtin_bit_cast(uint16_t, hi) << 16);
    }
    *(u4 *)(J.xa + ((size_t)u * 16 + f) * 1024 + 16 * L) = h;
  }
  if (tid < 16) J.xs[(size_t)u * 16 + tid] = inf ? -ldexpf(1.f, -e) : ldexpf(1.f, -e);
}

// The same fragments and scales for the feed-forward calls, whose matrices
// share one x: four blocks per unit, each staging the rows whole in LDS with
// coalesced loads, gathering its unit there and writing one fragment in four.
// (Gathered from memory by one block per unit, the 2-byte loads of 64 lanes
// keep one compute unit's address path busy for 3 us.)
constexpr int SB_PREP_BATCH = 8;  // 16-byte loads in flight per thread
template <bool XVEC>
__global__ __launch_bounds__(256) void sb_prep_rows_kernel(SbBatch b, int32_t *cnt, int n_cnt) {
  extern __shared__ __attribute__((aligned(16))) uint16_t s_rows[];
  __shared__ float s_max[4][16];
  const int per = b.job[0].w.units * 4;
  const int jn = (int)blockIdx.x / per, lb = (int)blockIdx.x - jn * per, u = lb >> 2, part = lb & 3;
  const SbJob &J = b.job[jn];
  const MatView &w = J.w;
  const int tid = threadIdx.x, wv = tid >> 6, L = tid & 63, K = w.k, ks = K + 8;
  if (blockIdx.x == 0)
    for (int i = tid; i < n_cnt; i += 256) cnt[i] = 0;
  const int m = L & 15, s = L >> 4;
  u4 pv[4];
#pragma unroll
  for (int ff = 0; ff < 4; ++ff)  // perm is zero padded to the unit width
    pv[ff] = *(const u4 *)(w.base + w.off_perm + 2 * (size_t)(u * UNIT_SLOTS + 8 * (16 * wv + 4 * s + ff)));
  if (XVEC) {
    const int n8 = K / 8, tot = b.m * n8;
    for (int q0 = tid; q0 < tot; q0 += 256 * SB_PREP_BATCH) {
      u4 v[SB_PREP_BATCH];
#pragma unroll
      for (int i = 0; i < SB_PREP_BATCH; ++i) {
        const int q = min(q0 + 256 * i, tot - 1), rr = q / n8;
        v[i] = *(const u4 *)(J.x + (int64_t)rr * J.ldx + 8 * (q - rr * n8));
      }
#pragma unroll
      for (int i = 0; i < SB_PREP_BATCH; ++i) {
        const int q = q0 + 256 * i, rr = q / n8;
        if (q < tot) *(u4 *)(s_rows + (size_t)rr * ks + 8 * (q - rr * n8)) = v[i];
      }
    }
  } else {
    for (int rr = 0; rr < b.m; ++rr)
      for (int j = tid; j < K; j += 256) s_rows[(size_t)rr * ks + j] = J.x[(int64_t)rr * J.ldx + j];
  }
  __syncthreads();
  const uint16_t *row = s_rows + (size_t)min(m, b.m - 1) * ks;
  float v[4][8];
  float mx = 0.f;
#pragma unroll
  for (int ff = 0; ff < 4; ++ff) {
    // k is a multiple of 8, so eight slots are all inside k or all padding
    const bool on = m < b.m && u * UNIT_SLOTS + 8 * (16 * wv + 4 * s + ff) < K;
#pragma unroll
    for (int l = 0; l < 4; ++l) {
      const float lo = bf16_bits_to_f32(row[pv[ff][l] & 0xFFFFu]), hi = bf16_bits_to_f32(row[pv[ff][l] >> 16]);
      v[ff][2 * l] = on ? lo : 0.f;
      v[ff][2 * l + 1] = on ? hi : 0.f;
      mx = fmaxf(mx, fmaxf(fabsf(v[ff][2 * l]), fabsf(v[ff][2 * l + 1])));
    }
  }
  mx = sb_row_max<false>(mx, s_max, wv, L);
  const bool inf = __any(mx == __builtin_inff());  // of any row: the same in every wave
  if (__builtin_expect(inf, 0)) mx = sb_row_max<true>(sb_finite_max(v), s_max, wv, L);
  const int e = mx > 0.f ? 15 - __builtin_amdgcn_frexp_expf(mx) : 0;
#pragma unroll
  for (int ff = 0; ff < 4; ++ff) {
    if (ff != part) continue;
    u4 h;
#pragma unroll
    for (int l = 0; l < 4; ++l) {
      const _Float16 lo = (_Float16)ldexpf(v[ff][2 * l], e), hi = (_Float16)ldexpf(v[ff][2 * l + 1], e);
      h[l] = (uint32_t)__builtin_bit_cast(uint16_t, lo) | ((uint32_t)__builtin_bit_cast(uint16_t, hi) << 16);
    }
    *(u4 *)(J.xa + ((size_t)u * 16 + 4 * wv + ff) * 1024 + 16 * L) = h;
  }
  if (part == 0 && tid < 16) J.xs[(size_t)u * 16 + tid] = inf ? -ldexpf(1.f, -e) : ldexpf(1.f, -e);
}

static hipError_t launch_sb_prep_rows(SbBatch &b, hipStream_t s, bool *fits) {
  const size_t lds = (size_t)b.m * (b.job[0].w.k + 8) * 2;
  *fits = lds + 1024 <= GV_LDS_LIMIT;
  if (!*fits) return hipSuccess;
  const bool xvec = (((uintptr_t)b.job[0].x | ((uintptr_t)b.job[0].ldx * 2)) & 15) == 0;
  const hipError_t e = xvec ? allow_smem(sb_prep_rows_kernel<true>, lds) : allow_smem(sb_prep_rows_kernel<false>, lds);
  if (e != hipSuccess) return e;
  int32_t *cnt = b.pair ? b.pair->cnt : b.job[0].cnt;
  const int n_cnt = b.pair ? b.pair->n_cnt : (cnt ? b.job[0].groups : 0);
  const dim3 grid(b.count * b.job[0].w.units * 4);
  if (xvec)
    hipLaunchKernelGGL(sb_prep_rows_kernel<true>, grid, dim3(256), lds, s, b, cnt, n_cnt);
  else
    hipLaunchKernelGGL(sb_prep_rows_kernel<false>, grid, dim3(256), lds, s, b, cnt, n_cnt);
  return hipGetLastError();
}

hipError_t launch_sb(SbBatch &b, int prep_blocks, int blocks, hipStream_t s) {
  hipError_t e;
  bool rows = false;
  if (b.epi || b.pair) {
    e = launch_sb_prep_rows(b, s, &rows);
    if (e != hipSuccess) return e;
  }
  if (!rows) {
    hipLaunchKernelGGL(sb_prep_kernel, dim3(prep_blocks), dim3(256), 0, s, b);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const dim3 grid(blocks), block(256);
  const bool hi = b.ydt == 0;
  if (b.pair && b.job[0].splits == 1) {
    const size_t smem = 2 * (size_t)(hi ? sb_half_bytes<true>() : sb_half_bytes<false>());
    e = hi ? allow_smem(sb_pair_kernel<true>, smem) : allow_smem(sb_pair_kernel<false>, smem);
    if (e != hipSuccess) return e;
    if (hi) hipLaunchKernelGGL(sb_pair_kernel<true>, dim3(b.job[0].groups), dim3(512), smem, s, b, *b.pair);
    else hipLaunchKernelGGL(sb_pair_kernel<false>, dim3(b.job[0].groups), dim3(512), smem, s, b, *b.pair);
    return hipGetLastError();
  }
  if (b.pair && hi)
    hipLaunchKernelGGL((sb_gemm_kernel<true, PairArgs>), grid, block, SB_SMEM, s, b, *b.pair);
  else if (b.pair)
    hipLaunchKernelGGL((sb_gemm_kernel<false, PairArgs>), grid, block, SB_SMEM, s, b, *b.pair);
  else if (b.epi && hi)
    hipLaunchKernelGGL((sb_gemm_kernel<true, EpiArgs>), grid, block, SB_SMEM, s, b, *b.epi);
  else if (b.epi)
    hipLaunchKernelGGL((sb_gemm_kernel<false, EpiArgs>), grid, block, SB_SMEM, s, b, *b.epi);
  else
    hipLaunchKernelGGL(sb_gemm_kernel<false>, grid, block, SB_SMEM, s, b);
  return hipGetLastError();
}

}  // namespace svq
