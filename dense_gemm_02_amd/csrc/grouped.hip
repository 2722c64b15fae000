// gemm_i8_grouped: argument checks, kernel choice and launch.
#include <math.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "dgemm.h"
#include "gemm_grouped.hpp"
#include "gemm_i8_skinny.hpp"
#include "gemm_pp.hpp"
#include "gemm_tn.hpp"
#include "launch.hpp"

namespace dg {
namespace {

// The block kernels and the skinny kernel over the groups' tiles.
template <class Op, int BP, int BQ, int NS, bool KT, bool GA>
__global__ void __launch_bounds__(256)
__attribute__((amdgpu_waves_per_eu(TnCfg<Op, false, BP, BQ, NS>::WPE, TnCfg<Op, false, BP, BQ, NS>::WPE)))
grouped_kernel(const GroupedArgs A) {
  GemmArgs g;
  Gather gt;
  if (!group_tile<BP, BQ, Op::OE>(A, &g, &gt)) return;
  gemm_tn_body<Op, false, BP, BQ, NS, KT, OneTile, GA>(g, OneTile{}, gt);
}

template <class Op, bool KT, bool GA>
__global__ void __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2)))
grouped_pp(const GroupedArgs A) {
  GemmArgs g;
  Gather gt;
  if (!group_tile<256, 256, Op::OE>(A, &g, &gt)) return;
  gemm_pp_body<Op, KT, OneTile, GA>(g, OneTile{}, gt);
}

template <class Op, int SF, int FF, int D, bool GA>
__global__ void __launch_bounds__(512) grouped_skinny(const GroupedArgs A) {
  GemmArgs g;
  Gather gt;
  if (!group_tile<16 * SF, 16 * FF, Op::OE>(A, &g, &gt)) return;
  gemm_i8_skinny_body<Op, SF, FF, 8, D, false, GA>(g, gt);
}

template <class Op, int BP, int BQ, int NS, bool GA>
Launch four_wave(const char* name, bool kt) {
  using Cfg = TnCfg<Op, false, BP, BQ, NS>;
  return Launch{kt ? (const void*)&grouped_kernel<Op, BP, BQ, NS, true, GA>
                   : (const void*)&grouped_kernel<Op, BP, BQ, NS, false, GA>,
                name, BP, BQ, Cfg::NT, Cfg::LDS, false};
}

template <class Op, int SF, int FF, bool GA>
Launch skinny(const char* name) {
  using Cfg = SkinnyI8Cfg<SF, FF, 8, 1>;
  return Launch{(const void*)&grouped_skinny<Op, SF, FF, 1, GA>, name, Cfg::SR, Cfg::FR, Cfg::NT, Cfg::LDS, false};
}

enum Kind { kPingPong, kFourWave, kFourStages, kNarrow, kSkinny16, kSkinny32, kSkinny64, kKinds };
const char* const kNames[kKinds] = {"i8_grouped_256x256_pp", "i8_grouped_128x128_w4", "i8_grouped_128x128_w4_s4",
                                    "i8_grouped_128x64_w4_s4", "i8_grouped_skinny16",
                                    "i8_grouped_skinny32", "i8_grouped_skinny64"};

template <class Op, bool GA>
Launch launch_of(int kind, bool kt) {
  switch (kind) {
    case kPingPong: {
      using Cfg = PpCfg<Op>;
      return Launch{kt ? (const void*)&grouped_pp<Op, true, GA> : (const void*)&grouped_pp<Op, false, GA>,
                    kNames[kind], 256, 256, Cfg::NT, Cfg::LDS, false};
    }
    case kFourWave: return four_wave<Op, 128, 128, 2, GA>(kNames[kind], kt);
    case kFourStages: return four_wave<Op, 128, 128, 4, GA>(kNames[kind], kt);
    case kNarrow: return four_wave<Op, 128, 64, 4, GA>(kNames[kind], kt);
    case kSkinny16: return skinny<Op, 2, 1, GA>(kNames[kind]);
    case kSkinny32: return skinny<Op, 2, 2, GA>(kNames[kind]);
    default: return skinny<Op, 2, 4, GA>(kNames[kind]);
  }
}

template <bool GA>
Launch launch_for(int c_type, int kind, bool kt) {
  switch (c_type) {
    case DGEMM_F32: return launch_of<OpI8F, GA>(kind, kt);
    case DGEMM_F16: return launch_of<OpI8H, GA>(kind, kt);
    default: return launch_of<OpI8B, GA>(kind, kt);
  }
}

// The kernel for `rows` rows spread over `groups` groups, whose sizes only the
// device knows: every group that can have rows is taken to have some, with a
// part-filled last tile half the time.  Estimated time in us: the larger of
// what the kernel's tiles cost and of what reading the groups' weights costs it,
//   256 x 256 (ping-pong, one per CU)   a round 12.5 us and 10.25 ns per k; weights at 4.0 TB/s
//   128 x 128 (two stages, two per CU)  a round 8.3 us and 7.7 ns per k; weights at 3.9 TB/s
//   128 x 128 (four stages, one)        a round 8 us and 6.4 ns per k; weights at 4.9 TB/s
//   128 x 64 (four stages, one)         a round 5.3 us and 3.7 ns per k; weights at 4.3 TB/s
//   skinny of `few` rows                a tile 54 ns * few and (32 + few) * K at 40 GB/s per CU; weights at 4.9 TB/s
// Measured (us; 256 x 256 / 128 x 128 / the same with four stages / 128 x 64 /
// skinny of 16 / of 32), sizes uneven as a router's:
//   512 rows, 64 groups, N 2048, K 4096    123 / 114 / 129 / 115 /   87 /   97
//   1024                                   136 / 130 / 137 / 120 /  121 /  122
//   2048                                   143 / 157 / 152 / 131 /  164 /  155
//   8192                                   179 / 180 / 207 / 215 /  420 /  347
//   256 rows, 8 groups, N 4096, K 14336    145 / 118 /  95 / 126 /  131 /  108
//   512                                    152 / 126 / 101 / 129 /  207 /  158
//   1024                                   156 / 157 / 170 / 182 /  369 /  270
//   2006                                   169 / 261 (four stages and narrow not measured)
//   32768 rows, 32 groups, N 4096, K 4096  518 / 707
//   30788 rows, 5 groups, N 2990, K 68      76 / 100 / 187 / 250 /  753 /  599
//   30788 rows, 5 groups, N 2990, K 1024   127 / 159 / 292 / 376 / 1014 /  758
//   12054 rows, 79 groups, N 1021, K 445    41 /  37 /  57 /  64 /  184 /  133
//   4096 rows, 8 groups, N 4096, K 128      16 /  20 /  34 /  43 /  140 /  109
//   512 rows, 64 groups, N 2048, K 256      22 /  14 /  24 /  21 /   23 /   32
// The skinny kernel of 64 is estimated fastest where one tile a CU covers all
// rows; there it runs within a tenth of that of 32 (256 x 256 / 128 x 128 / four
// stages / 128 x 64 / skinny of 16 / of 32 / of 64):
//   256 rows, 2 groups, N 2048, K 4096       42 / 35 / 31 / 21 / 19 / 17 / 18
//   512 rows, 4 groups, N 1024, K 4096       42 / 36 / 31 / 21 / 21 / 17 / 18
//   128 rows, 2 groups, N 4096, K 8192       74 / 63 / 52 / 36 / 35 / 32 / 35
//   1024 rows, 16 groups, N 512, K 8192      76 / 66 / 53 / 36 / 36 / 32 / 34
//   512 rows, 5 groups, N 1024, K 1024       17 / 13 / 15 / 12 / 12 / 12 / 12
int choose_kind(int64_t groups, int64_t rows, int64_t N, int64_t K) {
  const double cus = 256.0;
  const double some = (double)(groups < rows ? groups : rows);
  const double weights = some * (double)N * (double)K;   // bytes
  auto tiles = [&](int bq) {
    const double t = (double)rows / bq + 0.5 * some;
    return t > some ? t : some;
  };
  auto rounds = [&](int bp, int bq, int per_cu) {
    return ceil(tiles(bq) * (double)((N + bp - 1) / bp) / (cus * per_cu));
  };
  auto larger = [](double x, double y) { return x > y ? x : y; };
  double t[kKinds];
  t[kPingPong] = larger(rounds(256, 256, 1) * (12.5 + (double)K * 10.25e-3), weights / 4.0e6);
  t[kFourWave] = larger(rounds(128, 128, 2) * (8.3 + (double)K * 7.7e-3), weights / 3.9e6);
  t[kFourStages] = larger(rounds(128, 128, 1) * (8.0 + (double)K * 6.4e-3), weights / 4.9e6);
  t[kNarrow] = larger(rounds(128, 64, 1) * (5.3 + (double)K * 3.7e-3), weights / 4.3e6);
  for (int kind = kSkinny16; kind <= kSkinny64; ++kind) {
    const int few = 16 << (kind - kSkinny16);
    const double wgs = tiles(few) * (double)((N + 31) / 32) / cus;
    t[kind] = larger((wgs > 1 ? wgs : 1) * ((32 + few) * (double)K / 40e3 + 0.054 * few), weights / 4.9e6);
  }
  // (Sweeps and tests: DGEMM_CONFIG=<kernel name> forces a kernel, as for gemm_*.)
  if (const char* want = getenv("DGEMM_CONFIG"))
    for (int kind = 0; kind < kKinds; ++kind)
      if (strcmp(want, kNames[kind]) == 0) return kind;
  int best = 0;
  for (int kind = 1; kind < kKinds; ++kind)
    if (t[kind] < t[best]) best = kind;
  return best;
}

struct GroupedPlan {
  Launch L;
  int64_t tiles_p, tiles_q;
};

// The kernel and its workgroups: for the most row tiles that `rows` rows in
// `groups` groups can have, every group with rows may end in a part-filled
// one.  False if no launch holds them.
bool plan_grouped(int64_t groups, int64_t rows, int64_t N, int64_t K, int c_type, bool gather, GroupedPlan* pl) {
  const int kind = choose_kind(groups, rows, N, K);
  const bool kt = K % 128 != 0;
  pl->L = gather ? launch_for<true>(c_type, kind, kt) : launch_for<false>(c_type, kind, kt);
  pl->tiles_p = (N + pl->L.bp - 1) / pl->L.bp;
  const int64_t some = groups < rows ? groups : rows;
  pl->tiles_q = (rows + some * (pl->L.bq - 1)) / pl->L.bq;
  return launchable(pl->tiles_p * pl->tiles_q, pl->L.threads);
}

// Every wave looks through the groups 64 at a time (gemm_grouped.hpp, whose
// counter of groups has 32 bits): 2^14 steps at this many.
constexpr int64_t kMaxGroups = int64_t(1) << 20;

}  // namespace
}  // namespace dg

extern "C" {

int gemm_i8_grouped(int64_t groups, int64_t rows, int64_t N, int64_t K, const int8_t* A, int64_t rows_a, int64_t lda,
                    const int32_t* row_index, const int8_t* B, int64_t ldb, int64_t group_b, void* C, int64_t ldc,
                    int c_type, const float* scale_a, int64_t n_scale_a, const float* scale_b, int64_t n_scale_b,
                    const int32_t* offsets, void* stream) {
  using namespace dg;
  if (c_type < DGEMM_F32 || c_type > DGEMM_BF16) return DGEMM_ERR_INVALID_TYPE;
  if (groups < 0 || rows < 0 || N < 0 || K < 0 || rows_a < 0 || group_b < 0) return DGEMM_ERR_INVALID_DIM;
  if (groups > kMaxGroups || N > kMaxCount || groups * N > kMaxCount) return DGEMM_ERR_UNSUPPORTED;
  if ((n_scale_a != 1 && n_scale_a != rows_a) || (n_scale_b != 1 && n_scale_b != groups * N))
    return DGEMM_ERR_INVALID_DIM;
  if (row_index == nullptr && rows_a < rows) return DGEMM_ERR_INVALID_DIM;
  if (rows == 0 || N == 0 || groups == 0) return DGEMM_OK;
  if ((K > 0 && ((A == nullptr && rows_a > 0) || B == nullptr)) || C == nullptr ||
      (scale_a == nullptr && rows_a > 0) || scale_b == nullptr ||
      offsets == nullptr)
    return DGEMM_ERR_NULL_POINTER;
  const int64_t min_ld = K > 0 ? K : 1;
  if (lda < min_ld || ldb < min_ld || ldc < N) return DGEMM_ERR_INVALID_LD;
  const int oe = c_type == DGEMM_F32 ? 4 : 2;
  if (K > 0 && (!aligned_to(A, 16) || !aligned_to(B, 16) || lda % 16 != 0 || ldb % 16 != 0 || group_b % 16 != 0))
    return DGEMM_ERR_MISALIGNED;
  if (!aligned_to(C, oe) || !aligned_to(scale_a, 4) || !aligned_to(scale_b, 4) || !aligned_to(offsets, 4) ||
      !aligned_to(row_index, 4))
    return DGEMM_ERR_MISALIGNED;
  if (K > kMaxI8K || lda > kMaxDescBytes / 256 || ldb > kMaxDescBytes / 256) return DGEMM_ERR_UNSUPPORTED;
  // The factors of a group and of the rows, and with an index all rows of A
  // and their index, are addressed through one descriptor each.
  if (rows_a > kMaxDescBytes / 4 || N > kMaxDescBytes / 4 || rows > kMaxDescBytes / 4) return DGEMM_ERR_UNSUPPORTED;
  if (row_index != nullptr && rows_a > 0 && lda > kMaxDescBytes / rows_a) return DGEMM_ERR_UNSUPPORTED;

  // An index over no rows: every row counts as zeros, as with K == 0.
  if (rows_a == 0) K = 0;

  GroupedPlan pl;
  if (!plan_grouped(groups, rows, N, K, c_type, row_index != nullptr, &pl)) return DGEMM_ERR_UNSUPPORTED;
  GroupedArgs a{};
  GemmArgs& g = a.g;
  g.P = (const char*)B; g.ldp = ldb; g.Pn = N;
  g.Q = (const char*)A; g.ldq = lda; g.Qn = rows;
  g.C = C; g.ldc = ldc; g.K = K;
  g.group = 8;
  g.sp = scale_b; g.sp_row = n_scale_b > 1 ? 1 : 0;
  g.sq = scale_a; g.sq_row = n_scale_a > 1 ? 1 : 0;
  a.offsets = offsets; a.groups = groups; a.rows = rows; a.pstride = group_b;
  a.gt.index = row_index; a.gt.rows = rows_a;
  g.tiles_p = pl.tiles_p;
  g.tiles_q = pl.tiles_q;
  return launch_kernel(pl.L.fn, pl.tiles_p * pl.tiles_q, pl.L.threads, &a, stream);
}

int dgemm_grouped_config(int c_type, int gather, int64_t groups, int64_t rows, int64_t N, int64_t K, char* buf,
                         int64_t len) {
  using namespace dg;
  if (c_type < DGEMM_F32 || c_type > DGEMM_BF16) return DGEMM_ERR_INVALID_TYPE;
  if (groups < 0 || rows < 0 || N < 0 || K < 0) return DGEMM_ERR_INVALID_DIM;
  if (groups > kMaxGroups || N > kMaxCount || groups * N > kMaxCount) return DGEMM_ERR_UNSUPPORTED;
  if (rows > kMaxDescBytes / 4 || N > kMaxDescBytes / 4 || K > kMaxI8K) return DGEMM_ERR_UNSUPPORTED;
  GroupedPlan pl{};
  const bool none = rows == 0 || N == 0 || groups == 0;
  if (!none && !plan_grouped(groups, rows, N, K, c_type, gather != 0, &pl)) return DGEMM_ERR_UNSUPPORTED;
  if (buf != nullptr && len > 0) {
    if (none)
      snprintf(buf, (size_t)len, "none (empty output)");
    else
      snprintf(buf, (size_t)len, "%s tile=%dx%d threads=%d lds=%d grid=%lld tiles=%lldx%lld", pl.L.name, pl.L.bp,
               pl.L.bq, pl.L.threads, pl.L.lds, (long long)(pl.tiles_p * pl.tiles_q), (long long)pl.tiles_p,
               (long long)pl.tiles_q);
  }
  return DGEMM_OK;
}

}  // extern "C"
