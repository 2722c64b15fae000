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
// one group's weights and rows in its L2.  32768 rows in one group take as
// long as the dense product (442 us against 440, N = K = 4096), in 32 groups
// 7% longer, and 5% on top through an index.
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
__device__ __forceinline__ int wave_scan(int v) {
  const int lane = lane_id();
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// The tile of workgroup blockIdx.x: false if there is none, else *g holds the
// arguments of its product (one tile, at most BP x BQ of it valid) and *gt its
// row index.  (Tiles and rows are counted in 32 bits: the grid is below 2^31.)
template <int BP, int BQ, int OE>
__device__ __forceinline__ bool group_tile(const GroupedArgs& A, GemmArgs* g, Gather* gt) {
  const int lane = lane_id();
  const uint32_t tiles_p = (uint32_t)A.g.tiles_p;
  const int groups = (int)A.groups;
  // Lanes' groups e0 + lane: rows, tiles along q and their sum up to here.
  // One load of the offsets serves both the total and the search where there
  // are at most 64 groups.
  int e0 = 0, lo, hi, end;
  auto look = [&](int e, int before) {
    e0 = e;
    group_rows(A, e + lane, &lo, &hi);
    end = before + wave_scan((hi - lo + BQ - 1) / BQ);
    return __builtin_amdgcn_readlane(end, 63);
  };
  int mtiles = look(0, 0);
  for (int e = 64; e < groups; e += 64) mtiles = look(e, mtiles);
  const uint32_t total = (uint32_t)mtiles * tiles_p, pid = blockIdx.x;
  if (pid >= total) return false;
  // XCD spread over the tiles there are (see tile_map).
  const uint32_t per = total / kXcds, extra = total % kXcds;
  const uint32_t xcd = pid % kXcds, local = pid / kXcds;
  const uint32_t lid = (xcd < extra ? xcd * (per + 1) : extra * (per + 1) + (xcd - extra) * per) + local;
  const int m = (int)(lid / tiles_p);
  int before = 0;
  if (groups > 64) {
    before = look(0, 0);
    while (before <= m && e0 + 64 < groups) before = look(e0 + 64, before);
  }
  const uint64_t past = __ballot(end > m);
  if (past == 0) return false;   // (offsets that do not ascend can add up to anything)
  const int src = __builtin_amdgcn_readfirstlane(__builtin_ctzll(past));
  const int e = e0 + src;
  const int r0 = __builtin_amdgcn_readlane(lo, src), r1 = __builtin_amdgcn_readlane(hi, src);
  const uint32_t mt = (uint32_t)((r1 - r0 + BQ - 1) / BQ);
  const uint32_t in = lid - ((uint32_t)__builtin_amdgcn_readlane(end, src) - mt) * tiles_p;   // tile within the group
  const uint32_t width = (uint32_t)A.g.group * mt;
  const uint32_t grp = in / width, first = grp * (uint32_t)A.g.group;
  const uint32_t gsz = tiles_p - first < (uint32_t)A.g.group ? tiles_p - first : (uint32_t)A.g.group;
  const uint32_t rest = in - grp * width;
  // (The divisions run in vector registers; brought back, everything derived
  // from them is scalar, and the copies' descriptors need no per-lane loops.)
  auto scalar = [](uint32_t v) { return (int64_t)__builtin_amdgcn_readfirstlane((int)v); };
  const int64_t p0 = scalar(first + rest % gsz) * BP, q0 = r0 + scalar(rest / gsz) * BQ;
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

}  // namespace dg
