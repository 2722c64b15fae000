// Int8 product with row-major B (NN) of few rows, or of so few tiles that the
// block kernel leaves CUs idle: the skinny kernel's plan (gemm_i8_skinny.hpp)
// for an operand whose k runs down its rows.
//
// D[p][q] = sum_k P(k, p) Q(q, k): P = B, rows of k with p contiguous; Q = A.
// A workgroup computes SP x 16 FF of D; its NW waves take every NW-th stage of
// 128 k each, copy it straight into their own part of LDS and multiply from
// there, independently until their integer sums meet in LDS.
//
// P's fragments come from transposing LDS reads (ds_read_b64_tr_b8: in a group
// of 16 lanes, lane s addresses 8 consecutive p of row k0 + s / 2 and lane i
// receives 8 consecutive k of p0 + i).  Rows of SP bytes of P are XOR-swizzled
// in 16-byte chunks so that the 8 rows of a lane group, and those of the next
// group 16 rows on, meet different banks.  Rows of k at and past K land as
// zeros, so nothing of Q needs masking: what lies behind K in its rows
// meets zeros.  Workgroups next to each other along p run on one XCD at the
// same time: a 128-byte line of B that two narrow strips share is fetched once.
// The latency of rows a pitch apart bounds it: 16 x 8192 x 8192 28 us, 2.4 TB/s
// (with B in the caches 20), against 12.4 for a B contiguous along K.
#pragma once

#include "common.hpp"
#include "gemm_mfma.hpp"

namespace dg {

template <int SP_, int FF_, int NW_>
struct SkinnyNnCfg {
  static constexpr int SP = SP_, FF = FF_, NW = NW_, NT = 64 * NW_;
  static constexpr int FR = 16 * FF;
  static constexpr int BK = 128;                        // k per stage
  static constexpr int P_LDS = BK * SP, Q_LDS = FR * BK;
  static constexpr int STAGE = P_LDS + Q_LDS;
  static constexpr int CPR = SP / 16;                   // chunks per row of P
  static constexpr int RPC = 64 / CPR;                  // rows of P per copy
  static constexpr int RPB = 16 / CPR;                  // rows of P per 256 bytes (all banks)
  static constexpr int TP = SP / 16;
  static constexpr int RED = NW * TP * FF * 64 * 16;
  static constexpr int LDS = NW * STAGE > RED ? NW * STAGE : RED;
  static_assert(LDS <= kLdsLimit, "LDS budget");
  // Swizzle key of row k of P: what of k the banks do not tell apart.
  __device__ static constexpr int key(int k) {
    if constexpr (RPB >= 8) return CPR > 1 ? (k >> 4) & 1 : 0;
    else return ((k / RPB) & (8 / RPB - 1)) | (((k >> 4) & 1) * (8 / RPB));
  }
};

template <class Op, int SP, int FF, int NW>
__global__ void __launch_bounds__(64 * NW) gemm_i8_skinny_nn_kernel(const GemmArgs a) {
  using Cfg = SkinnyNnCfg<SP, FF, NW>;
  constexpr int BK = Cfg::BK, CPR = Cfg::CPR, TP = Cfg::TP;
  __shared__ __attribute__((aligned(1024))) char smem[Cfg::LDS];

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  // Tile: consecutive ones along p, contiguous ranges per XCD (see tile_map).
  const uint32_t total = gridDim.x, per = total / kXcds, extra = total % kXcds;
  const uint32_t xcd = blockIdx.x % kXcds, local = blockIdx.x / kXcds;
  const uint32_t lid = (xcd < extra ? xcd * (per + 1) : extra * (per + 1) + (xcd - extra) * per) + local;
  const uint32_t tiles_p = (uint32_t)a.tiles_p;
  const uint32_t tq = (uint32_t)__builtin_amdgcn_readfirstlane((int)(lid / tiles_p));
  const int64_t p0 = (int64_t)(lid - tq * tiles_p) * SP, q0 = (int64_t)tq * Cfg::FR;

  const int64_t K = a.K;
  const uint32_t kbytes16 = (uint32_t)((K + 15) & ~(int64_t)15);
  const int64_t pcols = a.Pn - p0 < SP ? a.Pn - p0 : SP;
  const int64_t qrows = a.Qn - q0 < Cfg::FR ? a.Qn - q0 : Cfg::FR;
  const i32x4 rp = make_desc(a.P + p0, K > 0 ? (uint32_t)((K - 1) * a.ldp) + (uint32_t)((pcols + 15) & ~(int64_t)15) : 0u);
  const i32x4 rq = make_desc(a.Q + q0 * a.ldq, (uint32_t)((qrows - 1) * a.ldq) + kbytes16);

  // Copy s of P fills rows RPC s .. of its stage: lane l lands in row l / CPR,
  // physical chunk l % CPR.  Copy s of Q fills rows 8 s .. 8 s + 7 as in the
  // other kernels.
  constexpr int NP = BK / Cfg::RPC, NQ = 2 * FF;
  uint32_t poff[NP], qoff[NQ];
#pragma unroll
  for (int s = 0; s < NP; ++s) {
    const int k = Cfg::RPC * s + lane / CPR;
    const int c = 16 * ((lane % CPR) ^ Cfg::key(k));
    poff[s] = c < pcols ? (uint32_t)(k * a.ldp + c) : kOobOffset;
  }
  const int crow = lane >> 3;
  auto chunk = [&](int s) { return ((lane & 7) ^ ((4 * s + (lane >> 4)) & 7)) * 16; };
#pragma unroll
  for (int s = 0; s < NQ; ++s)
    qoff[s] = 8 * s + crow < qrows ? (uint32_t)((8 * s + crow) * a.ldq + chunk(s)) : kOobOffset;

  const int nst = (int)((K + BK - 1) / BK);
  char* const mine = smem + wave * Cfg::STAGE;
  i32x4 acc[TP][FF];
#pragma unroll
  for (int j = 0; j < TP; ++j)
#pragma unroll
    for (int f = 0; f < FF; ++f) acc[j][f] = i32x4{0, 0, 0, 0};
  const int r16 = lane & 15, kg = lane >> 4;
  // Workgroups start at different stages, so that they do not all read the
  // same rows of B and columns of A at once.
  const int rot = nst > 0 ? (int)((lid * 5u) % (uint32_t)nst) : 0;
  // One stage in LDS at a time: a second in flight gained nothing (16 rows,
  // strips of 32: 8192 x 8192 28.7 us with one and 31.7 with two, 4096 x 4096
  // 10.0 and 9.9), the other waves' copies fill the time.
  for (int i = wave; i < nst; i += NW) {
    const int t = i + rot < nst ? i + rot : i + rot - nst;
    const int64_t at = (int64_t)t * BK, left = K - at;   // k from the stage on
    const uint32_t pat = (uint32_t)(at * a.ldp);
#pragma unroll
    for (int s = 0; s < NP; ++s)
      copy16_lds(rp, (poff[s] + pat) | (Cfg::RPC * s + lane / CPR >= left ? kOobOffset : 0u), mine + s * 1024);
#pragma unroll
    for (int s = 0; s < NQ; ++s)
      copy16_lds(rq, (qoff[s] + (uint32_t)at) | (chunk(s) >= left ? kOobOffset : 0u), mine + Cfg::P_LDS + s * 1024);
    __builtin_amdgcn_s_waitcnt(kWaitVmcnt0);
    asm volatile("" ::: "memory");
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      i32x4 pv[TP], qv[FF];
#pragma unroll
      for (int f = 0; f < FF; ++f)
        qv[f] = *(const i32x4*)(mine + Cfg::P_LDS + (16 * f + r16) * BK + (((4 * h + kg) ^ ((r16 >> 1) & 7)) * 16));
#pragma unroll
      for (int j = 0; j < TP; ++j)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int k = 64 * h + 16 * kg + 8 * half + r16 / 2;
          const char* src = mine + k * SP + ((j ^ Cfg::key(k)) * 16) + (r16 % 2) * 8;
          typedef int i32x2v __attribute__((ext_vector_type(2)));
          const i32x2v v = __builtin_amdgcn_ds_read_tr8_b64_v2i32((__attribute__((address_space(3))) i32x2v*)src);
          pv[j][2 * half] = v[0];
          pv[j][2 * half + 1] = v[1];
        }
#pragma unroll
      for (int j = 0; j < TP; ++j)
#pragma unroll
        for (int f = 0; f < FF; ++f)
          acc[j][f] = __builtin_amdgcn_mfma_i32_16x16x64_i8(pv[j], qv[f], acc[j][f], 0, 0, 0);
    }
    // The next copies overwrite what has been read.
    __builtin_amdgcn_s_waitcnt(kWaitLgkmcnt0);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  }
  __syncthreads();

  // The waves' sums (as in gemm_i8_skinny.hpp).
  GemmArgs g = a;
  g.C = (char*)a.C + (q0 * a.ldc + p0) * Op::OE;
  g.Pn = a.Pn - p0;
  g.Qn = a.Qn - q0;
  if (a.sp_row) g.sp += p0;
  if (a.sq_row) g.sq += q0;
  i32x4* red = (i32x4*)smem;   // [NW][TP * FF][64]
#pragma unroll
  for (int j = 0; j < TP; ++j)
#pragma unroll
    for (int f = 0; f < FF; ++f) red[(wave * TP * FF + j * FF + f) * 64 + lane] = acc[j][f];
  __syncthreads();
  for (int u = wave; u < TP * FF; u += NW) {
    i32x4 s = i32x4{0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < NW; ++w) s += red[(w * TP * FF + u) * 64 + lane];
    const int64_t p = 16 * (u / FF) + 4 * kg, q = 16 * (u % FF);
    EpiScale<1, 16> sc;
    sc.init(g, lane, q, Gather{});
    float v0 = s[0], v1 = s[1], v2 = s[2], v3 = s[3];
    sc.apply(EpiScale<1, 16>::p4(g, p), 0, v0, v1, v2, v3);
    if (q + r16 < g.Qn) store4<Op>(g, q + r16, p, v0, v1, v2, v3);
  }
}

}  // namespace dg
