// gemm_i8_grouped: argument checks, kernel choice and launch.
#include "dgemm.h"
#include "gemm_grouped.hpp"
#include "gemm_tn.hpp"
#include "launch.hpp"

namespace dg {
namespace {

// The four-wave kernel over the groups' tiles (K-tail masks in any case).
template <class Op, int BP, int BQ, bool GA>
__global__ void __launch_bounds__(256)
__attribute__((amdgpu_waves_per_eu(TnCfg<Op, false, BP, BQ, 2>::WPE, TnCfg<Op, false, BP, BQ, 2>::WPE)))
grouped_kernel(const GroupedArgs A) {
  GemmArgs g;
  Gather gt;
  if (!group_tile<BP, BQ, Op::OE>(A, &g, &gt)) return;
  gemm_tn_body<Op, false, BP, BQ, 2, true, OneTile, GA>(g, OneTile{}, gt);
}

template <class Op, int BP, int BQ>
Launch four_wave(bool ga) {
  using Cfg = TnCfg<Op, false, BP, BQ, 2>;
  return Launch{ga ? (const void*)&grouped_kernel<Op, BP, BQ, true> : (const void*)&grouped_kernel<Op, BP, BQ, false>,
                "i8_grouped", BP, BQ, Cfg::NT, Cfg::LDS, false};
}

Launch select(int c_type, bool ga) {
  switch (c_type) {
    case DGEMM_F32: return four_wave<OpI8F, 128, 128>(ga);
    case DGEMM_F16: return four_wave<OpI8H, 128, 128>(ga);
    default: return four_wave<OpI8B, 128, 128>(ga);
  }
}

constexpr int64_t kMaxCount = 0x7fffffff;

bool aligned(const void* p, int64_t n) { return ((uintptr_t)p) % (uintptr_t)n == 0; }

}  // namespace
}  // namespace dg

extern "C" int gemm_i8_grouped(int64_t groups, int64_t rows, int64_t N, int64_t K, const int8_t* A, int64_t rows_a,
                               int64_t lda, const int32_t* row_index, const int8_t* B, int64_t ldb, int64_t group_b,
                               void* C, int64_t ldc, int c_type, const float* scale_a, int64_t n_scale_a,
                               const float* scale_b, int64_t n_scale_b, const int32_t* offsets, void* stream) {
  using namespace dg;
  if (c_type < DGEMM_F32 || c_type > DGEMM_BF16) return DGEMM_ERR_INVALID_TYPE;
  if (groups < 0 || rows < 0 || N < 0 || K < 0 || rows_a < 0 || group_b < 0) return DGEMM_ERR_INVALID_DIM;
  if (groups > kMaxCount || N > kMaxCount || groups * N > kMaxCount) return DGEMM_ERR_UNSUPPORTED;
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
  if (K > 0 && (!aligned(A, 16) || !aligned(B, 16) || lda % 16 != 0 || ldb % 16 != 0 || group_b % 16 != 0))
    return DGEMM_ERR_MISALIGNED;
  if (!aligned(C, oe) || !aligned(scale_a, 4) || !aligned(scale_b, 4) || !aligned(offsets, 4) ||
      !aligned(row_index, 4))
    return DGEMM_ERR_MISALIGNED;
  if (K > kMaxI8K || lda > kMaxDescBytes / 256 || ldb > kMaxDescBytes / 256) return DGEMM_ERR_UNSUPPORTED;
  // The factors of a group and of the rows, and with an index all rows of A
  // and their index, are addressed through one descriptor each.
  if (rows_a > kMaxDescBytes / 4 || N > kMaxDescBytes / 4 || rows > kMaxDescBytes / 4) return DGEMM_ERR_UNSUPPORTED;
  if (row_index != nullptr && rows_a > 0 && lda > kMaxDescBytes / rows_a) return DGEMM_ERR_UNSUPPORTED;

  // An index over no rows: every row counts as zeros, as with K == 0.
  if (rows_a == 0) K = 0;

  const Launch L = select(c_type, row_index != nullptr);
  GroupedArgs a{};
  GemmArgs& g = a.g;
  g.P = (const char*)B; g.ldp = ldb; g.Pn = N;
  g.Q = (const char*)A; g.ldq = lda; g.Qn = rows;
  g.C = C; g.ldc = ldc; g.K = K;
  g.group = 8;
  g.vec_store = aligned(C, 4 * oe) && ldc % 4 == 0;
  g.vec16 = aligned(C, 16) && (ldc * oe) % 16 == 0;
  g.sp = scale_b; g.sp_row = n_scale_b > 1 ? 1 : 0;
  g.sq = scale_a; g.sq_row = n_scale_a > 1 ? 1 : 0;
  a.offsets = offsets; a.groups = groups; a.rows = rows; a.pstride = group_b;
  a.gt.index = row_index; a.gt.rows = rows_a;
  // Workgroups for the most row tiles that `rows` rows in `groups` groups
  // can have: every group with rows may end in a part-filled one.
  g.tiles_p = (N + L.bp - 1) / L.bp;
  const int64_t some = groups < rows ? groups : rows;
  g.tiles_q = (rows + some * (L.bq - 1)) / L.bq;
  const int64_t grid = g.tiles_p * g.tiles_q;
  if (grid > kMaxCount) return DGEMM_ERR_UNSUPPORTED;
  return launch_kernel(L.fn, grid, L.threads, &a, stream);
}
