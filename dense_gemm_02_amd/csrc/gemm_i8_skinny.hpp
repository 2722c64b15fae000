// Int8 product of a few rows (tokens of a decoding step) with many (a weight):
// time goes into reading the many rows once from HBM, so a workgroup takes a
// strip of 16 SF of them, splits K over its NW waves, which run independently
// until the end, and sums their integer results through LDS in wave order.
//
// Each wave copies its stages, 128 bytes of k of every row, straight into its
// own part of LDS, D stages in a ring, and multiplies them from there
// (v_mfma_i32_16x16x64_i8).  The copies cover whole 128-byte lines (8 rows of
// 128 bytes an instruction): loaded into registers in operand layout, 16
// rows of 64 bytes, the halves of a line were fetched twice as soon as more
// was in flight than the 32 KiB L1 holds.  Rows past the edge and chunks past K
// are pushed out of the descriptor's range and land as zeros; a chunk that
// straddles K is masked in the few rows' fragments (integers: zero times
// anything is zero).
//
// Memory bounds it while the few rows are few: 8192 x 16 x 8192 (67 MB) 12.1 us,
// 5.6 TB/s, over a few weights that the 256 MB cache behind the L2s holds, 14.2
// us, 4.7 TB/s, over twelve that it does not; then the copies, at about 40 GB/s
// per CU.
//
// Either operand may be the few: FEWP (D[p][q], p the contiguous direction of
// C) or not, and the few rows may come through a row index (grouped products).
#pragma once

#include "common.hpp"
#include "gemm_mfma.hpp"

namespace dg {

template <int SF, int FF, int NW_, int D>
struct SkinnyI8Cfg {
  static constexpr int NW = NW_, NT = 64 * NW_;
  static constexpr int SR = 16 * SF;                   // rows of the strip
  static constexpr int FR = 16 * FF;                   // few rows, at most
  static constexpr int BK = 128;                       // k (and bytes of a row) per stage
  static constexpr int STAGE = (SR + FR) * BK;         // strip, then few rows
  static constexpr int NDMA = 2 * (SF + FF);           // copies per stage
  static constexpr int RING = NW * D * STAGE;
  static constexpr int RED = NW * SF * FF * 64 * 16;   // the sums, in the same place
  static constexpr int LDS = RING > RED ? RING : RED;
  static_assert(LDS <= kLdsLimit && (D - 1) * NDMA <= 63, "LDS budget and vmcnt range");
};

template <class Op, int SF, int FF, int NW, int D, bool FEWP, bool GA>
__device__ __forceinline__ void gemm_i8_skinny_body(const GemmArgs& a, const Gather& gt) {
  using Cfg = SkinnyI8Cfg<SF, FF, NW, D>;
  constexpr int BK = Cfg::BK;
  __shared__ __attribute__((aligned(1024))) char smem[Cfg::LDS];

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t K = a.K;
  const uint32_t kbytes16 = (uint32_t)((K + 15) & ~(int64_t)15);
  const char* sbase = FEWP ? a.Q : a.P;
  const char* fbase = FEWP ? a.P : a.Q;
  const int64_t lds = FEWP ? a.ldq : a.ldp, ldf = FEWP ? a.ldp : a.ldq;
  const int64_t sn = FEWP ? a.Qn : a.Pn, fn = FEWP ? a.Pn : a.Qn;
  const int64_t srows = sn < Cfg::SR ? sn : Cfg::SR;
  const int64_t frows = GA ? gt.rows : (fn < Cfg::FR ? fn : Cfg::FR);
  const i32x4 rs = make_desc(sbase, (uint32_t)((srows - 1) * lds) + kbytes16);
  const i32x4 rf = make_desc(fbase, frows > 0 ? (uint32_t)((frows - 1) * ldf) + kbytes16 : 0u);

  // Copy s of an operand fills rows 8 s .. 8 s + 7: lane l lands at byte 16 l of
  // them, row l / 8, physical chunk l % 8, which holds logical chunk
  // (l % 8) ^ key(row), key(row) = (row / 2) mod 8.
  uint32_t soff[2 * SF], foff[2 * FF];
  const int crow = lane >> 3;
  auto chunk = [&](int s) { return ((lane & 7) ^ ((4 * s + (lane >> 4)) & 7)) * 16; };
#pragma unroll
  for (int s = 0; s < 2 * SF; ++s)
    soff[s] = 8 * s + crow < sn ? (uint32_t)((8 * s + crow) * lds + chunk(s)) : kOobOffset;
#pragma unroll
  for (int s = 0; s < 2 * FF; ++s) {
    if constexpr (GA) foff[s] = gather_row(gt, 8 * s + crow, fn, ldf, chunk(s));
    else foff[s] = 8 * s + crow < fn ? (uint32_t)((8 * s + crow) * ldf + chunk(s)) : kOobOffset;
  }

  // This wave's stages: every NW-th, from a place that differs between
  // workgroups, so that they do not all read the same part of the rows at once.
  const int nst = (int)((K + BK - 1) / BK);
  const int rot = nst > 0 ? (int)((blockIdx.x * 5u) % (uint32_t)nst) : 0;
  auto stage_of = [&](int i) {
    const int t = wave + i * NW + rot;
    return t < nst ? t : t - nst;
  };
  const int mine = (nst - wave + NW - 1) / NW;     // (0 or less: none)
  char* const ring = smem + wave * (D * Cfg::STAGE);
  auto copies = [&](int i, int slot) {
    const int t = stage_of(i);
    const uint32_t at = (uint32_t)t * BK;
    const int64_t left = i < mine ? K - at : 0;    // bytes of the row from the stage on
    char* dst = ring + slot * Cfg::STAGE;
#pragma unroll
    for (int s = 0; s < 2 * SF; ++s)
      copy16_lds(rs, (soff[s] + at) | (chunk(s) >= left ? kOobOffset : 0u), dst + s * 1024);
#pragma unroll
    for (int s = 0; s < 2 * FF; ++s)
      copy16_lds(rf, (foff[s] + at) | (chunk(s) >= left ? kOobOffset : 0u), dst + (2 * SF + s) * 1024);
  };

  i32x4 acc[SF][FF];
#pragma unroll
  for (int j = 0; j < SF; ++j)
#pragma unroll
    for (int f = 0; f < FF; ++f) acc[j][f] = i32x4{0, 0, 0, 0};
  const int r16 = lane & 15, kg = lane >> 4;
  auto consume = [&](int i, int slot) {
    const char* src = ring + slot * Cfg::STAGE + r16 * BK;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int at = ((4 * h + kg) ^ ((r16 >> 1) & 7)) * 16;
      i32x4 sv[SF], fv[FF];
#pragma unroll
      for (int j = 0; j < SF; ++j) sv[j] = *(const i32x4*)(src + 16 * j * BK + at);
#pragma unroll
      for (int f = 0; f < FF; ++f) fv[f] = *(const i32x4*)(src + (Cfg::SR + 16 * f) * BK + at);
      if (K % 16 != 0 && i < mine && stage_of(i) == nst - 1) {
        const int64_t vb = K - (int64_t)(nst - 1) * BK - (4 * h + kg) * 16;   // bytes of this chunk below K
#pragma unroll
        for (int f = 0; f < FF; ++f)
          fv[f] = __builtin_bit_cast(i32x4, mask_tail(__builtin_bit_cast(u32x4, fv[f]), vb < 0 ? 0 : (vb > 16 ? 16 : (int)vb)));
      }
#pragma unroll
      for (int j = 0; j < SF; ++j)
#pragma unroll
        for (int f = 0; f < FF; ++f)
          acc[j][f] = FEWP ? __builtin_amdgcn_mfma_i32_16x16x64_i8(fv[f], sv[j], acc[j][f], 0, 0, 0)
                           : __builtin_amdgcn_mfma_i32_16x16x64_i8(sv[j], fv[f], acc[j][f], 0, 0, 0);
    }
  };
  // Stage i lives in slot i mod D.  Every turn copies one stage (past the last:
  // zeros), so D - 1 later ones are in flight when one is multiplied.  The
  // copies are assembly the compiler does not see as LDS writes: the waits
  // here order them, and the multiplications, which need the fragments in
  // registers, come before the slot's next copy.
#pragma unroll
  for (int u = 0; u < D; ++u) copies(u, u);
  for (int i = 0; i < mine; i += D) {
#pragma unroll
    for (int u = 0; u < D; ++u) {
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_waitcnt(kWaitVmcntBase | vmcnt_bits((D - 1) * Cfg::NDMA));
      asm volatile("" ::: "memory");
      consume(i + u, u);
      __builtin_amdgcn_s_waitcnt(kWaitLgkmcnt0);
      __builtin_amdgcn_sched_barrier(0);
      copies(i + u + D, u);
    }
  }
  // No copy may land any more where the sums go.
  __builtin_amdgcn_s_waitcnt(kWaitVmcnt0);
  asm volatile("" ::: "memory");
  __syncthreads();

  // The waves' sums, tile by tile: lane l holds column l % 16 (q) and rows
  // 4 (l / 16) .. + 3 (p) of a 16 x 16 tile.
  i32x4* red = (i32x4*)smem;   // [NW][SF * FF][64]
#pragma unroll
  for (int j = 0; j < SF; ++j)
#pragma unroll
    for (int f = 0; f < FF; ++f) red[(wave * SF * FF + j * FF + f) * 64 + lane] = acc[j][f];
  __syncthreads();
  for (int u = wave; u < SF * FF; u += NW) {
    i32x4 s = i32x4{0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < NW; ++w) s += red[(w * SF * FF + u) * 64 + lane];
    const int j = u / FF, f = u % FF;
    const int64_t p = 16 * (FEWP ? f : j) + 4 * kg, q0 = 16 * (FEWP ? j : f);
    EpiScale<1, 16, GA> sc;
    sc.init(a, lane, q0, gt);
    float v0 = s[0], v1 = s[1], v2 = s[2], v3 = s[3];
    sc.apply(EpiScale<1, 16, GA>::p4(a, p), 0, v0, v1, v2, v3);
    if (q0 + r16 < a.Qn) store4<Op>(a, q0 + r16, p, v0, v1, v2, v3);
  }
}

// A dense product: one strip against at most FR of the few rows per workgroup.
template <class Op, int SF, int FF, int NW, int D, bool FEWP>
__global__ void __launch_bounds__(64 * NW) gemm_i8_skinny_kernel(const GemmArgs a) {
  using Cfg = SkinnyI8Cfg<SF, FF, NW, D>;
  const uint32_t tiles_p = (uint32_t)a.tiles_p;
  const int64_t tq = (uint32_t)__builtin_amdgcn_readfirstlane((int)(blockIdx.x / tiles_p));
  const int64_t p0 = (blockIdx.x - (uint32_t)tq * tiles_p) * (int64_t)(FEWP ? Cfg::FR : Cfg::SR);
  const int64_t q0 = tq * (FEWP ? Cfg::SR : Cfg::FR);
  GemmArgs g = a;
  g.P += p0 * a.ldp;
  g.Q += q0 * a.ldq;
  g.C = (char*)a.C + (q0 * a.ldc + p0) * Op::OE;
  g.Pn = a.Pn - p0;
  g.Qn = a.Qn - q0;
  if (a.sp_row) g.sp += p0;
  if (a.sq_row) g.sq += q0;
  gemm_i8_skinny_body<Op, SF, FF, NW, D, FEWP, false>(g, Gather{});
}

}  // namespace dg
