// Grouped products (mixture of experts): the block kernels run over the
// tiles of every group in one launch, with the groups' row ranges read on the
// device, so the host waits for nothing.
//
// The host launches as many workgroups as the groups could need at most;
// each wave sums the groups' tile counts with one scan (lane e, expert e),
// finds its own group, and patches the arguments so that the block kernel
// sees a product of one tile: P = the group's weights (p along N), Q = its rows
// of A, C row-major.  Surplus workgroups end there.  Tiles are ordered group
// by group, spread over the XCDs in contiguous ranges and walked eight along
// p, as tile_map does for one product, so the workgroups of one XCD share
// one group's weights and rows in its L2.
#pragma once

#include "common.hpp"

namespace dg {

struct GroupedArgs {
  GemmArgs g;               // P, sp: of group 0; Q, C, sq: of row 0
  const int32_t* offsets;   // groups + 1 row numbers
  int64_t groups, rows;
  int64_t pstride;          // bytes between the groups' P
  Gather gt;                // row index of Q (index: of row 0), or none
};

// This lane's group e: its rows, clamped to the matrix.
__device__ __forceinline__ void group_rows(const GroupedArgs& A, int64_t e, int* lo, int* hi) {
  const int rows = (int)A.rows;
  int a = 0, b = 0;
  if (e < A.groups) {
    a = A.offsets[e];
    b = A.offsets[e + 1];
  }
  a = a < 0 ? 0 : (a > rows ? rows : a);
  b = b < a ? a : (b > rows ? rows : b);
  *lo = a;
  *hi = b;
}

// Inclusive sum over the lanes of a wave.
__device__ __forceinline__ int64_t wave_scan(int64_t v) {
  const int lane = lane_id();
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int64_t o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// A value of lane `src` in scalar registers.
__device__ __forceinline__ int64_t lane_value(int64_t v, int src) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, src);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)((uint64_t)v >> 32), src);
  return (int64_t)((uint64_t)hi << 32 | lo);
}

// The tile of workgroup blockIdx.x: false if there is none, else *g holds the
// arguments of its product (one tile, at most BP x BQ of it valid) and *gt its
// row index.
template <int BP, int BQ, int OE>
__device__ __forceinline__ bool group_tile(const GroupedArgs& A, GemmArgs* g, Gather* gt) {
  const int lane = lane_id();
  const int64_t tiles_p = A.g.tiles_p;
  int64_t mtiles = 0;
  for (int64_t e0 = 0; e0 < A.groups; e0 += 64) {
    int lo, hi;
    group_rows(A, e0 + lane, &lo, &hi);
    mtiles += lane_value(wave_scan((hi - lo + BQ - 1) / BQ), 63);
  }
  const int64_t total = mtiles * tiles_p, pid = blockIdx.x;
  if (pid >= total) return false;
  // XCD spread over the tiles there are (see tile_map).
  const int64_t per = total / kXcds, extra = total % kXcds;
  const int64_t xcd = pid % kXcds, local = pid / kXcds;
  const int64_t lid = (xcd < extra ? xcd * (per + 1) : extra * (per + 1) + (xcd - extra) * per) + local;
  const int64_t m = lid / tiles_p;
  int64_t before = 0;
  for (int64_t e0 = 0; e0 < A.groups; e0 += 64) {
    int lo, hi;
    group_rows(A, e0 + lane, &lo, &hi);
    const int64_t mine = (hi - lo + BQ - 1) / BQ;
    const int64_t end = before + wave_scan(mine);
    const uint64_t past = __ballot(end > m);
    if (past == 0) {
      before = lane_value(end, 63);
      continue;
    }
    const int src = __builtin_ctzll(past);
    const int64_t e = e0 + src;
    const int64_t mt = lane_value(mine, src);
    const int64_t in = lid - (lane_value(end, src) - mt) * tiles_p;   // tile within the group
    const int64_t r0 = __builtin_amdgcn_readlane(lo, src), r1 = __builtin_amdgcn_readlane(hi, src);
    const int64_t width = A.g.group * mt;
    const int64_t grp = in / width, first = grp * A.g.group;
    const int64_t gsz = tiles_p - first < A.g.group ? tiles_p - first : A.g.group;
    const int64_t rest = in - grp * width;
    const int64_t p0 = (first + rest % gsz) * BP, q0 = r0 + rest / gsz * BQ;
    *g = A.g;
    g->P += e * A.pstride + p0 * A.g.ldp;
    g->C = (char*)A.g.C + (q0 * A.g.ldc + p0) * OE;
    if (A.g.sp_row) g->sp += e * A.g.Pn + p0;
    g->Pn = A.g.Pn - p0;
    g->Qn = r1 - q0;
    g->tiles_p = g->tiles_q = g->group = 1;
    *gt = A.gt;
    if (A.gt.index != nullptr) {
      gt->index += q0;
    } else {
      g->Q += q0 * A.g.ldq;
      if (A.g.sq_row) g->sq += q0;
    }
    return true;
  }
  return false;
}

}  // namespace dg
