// gemm_fp8_block and gemm_fp8_grouped: argument checks, kernel choice and launch.
#include <math.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "dgemm.h"
#include "elementwise.hpp"
#include "fp8_block.hpp"
#include "gemm_grouped.hpp"

namespace dg {
namespace {

constexpr int kBlock = 128;
constexpr double kCus = 256.0;

int64_t blocks_of(int64_t n) { return n / kBlock + (n % kBlock != 0); }
double tiles_of(int64_t n, int b) { return (double)((n + b - 1) / b); }

// The factors of one operand, and whether they can be addressed: `n` of them
// along the rows (or groups of 128) within one descriptor.
struct Factors {
  const float* at;
  int rows;         // rows of the operand to a factor: 1 or 128
  int64_t r, k;     // elements between factors of neighbouring rows and blocks
  int shift() const { return rows == 1 ? 0 : 7; }
};

bool valid_rows(int rows) { return rows == 1 || rows == kBlock; }
bool addressable(const Factors& f, int64_t rows) {
  const int64_t n = f.rows == 1 ? rows : blocks_of(rows);
  return n <= kMaxDescBytes / 4 && f.r <= kMaxDescBytes / 4 / (n > 0 ? n : 1) && f.k <= (int64_t(1) << 40);
}

Launch tn_launch(int c_type, int tile, bool rows, bool kt) {
  return c_type == DGEMM_F32 ? b8_tn_f32(tile, rows, kt)
                             : (c_type == DGEMM_F16 ? b8_tn_f16(tile, rows, kt) : b8_tn_bf16(tile, rows, kt));
}
Launch nn_launch(int c_type, int tile, bool rows, bool kt) {
  return c_type == DGEMM_F32 ? b8_nn_f32(tile, rows, kt)
                             : (c_type == DGEMM_F16 ? b8_nn_f16(tile, rows, kt) : b8_nn_bf16(tile, rows, kt));
}
Launch nn_skinny_launch(int c_type, int sp, int fr) {
  return c_type == DGEMM_F32 ? b8_nn_skinny_f32(sp, fr)
                             : (c_type == DGEMM_F16 ? b8_nn_skinny_f16(sp, fr) : b8_nn_skinny_bf16(sp, fr));
}
Launch skinny_launch(int c_type, int sf, int ff, bool few_p, bool two) {
  return c_type == DGEMM_F32 ? b8_skinny_f32(sf, ff, few_p, two)
                             : (c_type == DGEMM_F16 ? b8_skinny_f16(sf, ff, few_p, two)
                                                    : b8_skinny_bf16(sf, ff, few_p, two));
}
Launch grouped_launch(int c_type, int kind, bool gather, bool kt) {
  return c_type == DGEMM_F32 ? b8_grouped_f32(kind, gather, kt)
                             : (c_type == DGEMM_F16 ? b8_grouped_f16(kind, gather, kt)
                                                    : b8_grouped_bf16(kind, gather, kt));
}

// The TN strip that DGEMM_CONFIG names (sweeps and tests): its kernel's name with its
// rows, few rows and stages in flight behind, "b8bf16_tn_skinny_a:32x16x2".
bool forced_strip(const char* want, int c_type, int64_t Pn, int64_t Qn, Launch* L) {
  for (int sf = 1; sf <= 2; ++sf)
    for (int ff = 1; ff <= 4; ff *= 2)
      for (int stages = 1; stages <= 2; ++stages)
        for (int few_p = 0; few_p < 2; ++few_p) {
          if (ff == 4 && (sf == 1 || stages == 2)) continue;   // (not built)
          *L = skinny_launch(c_type, sf, ff, few_p != 0, stages == 2);
          char name[64];
          snprintf(name, sizeof name, "%s:%dx%dx%d", L->name, 16 * sf, 16 * ff, stages);
          if (strcmp(name, want) == 0)
            return tiles_of(Pn, L->bp) * tiles_of(Qn, L->bq) <= (double)(0xffffffffll / L->threads);
        }
  return false;
}

// The kernel of a TN product of Pn x Qn x K; `rows`: P has a factor for each row.
Launch choose_tn(int c_type, int64_t Pn, int64_t Qn, int64_t K, bool rows) {
  const char* want = getenv("DGEMM_CONFIG");
  const bool kt = K % kBlock != 0;
  if (want != nullptr && *want != 0) {
    Launch L;
    if (forced_strip(want, c_type, Pn, Qn, &L)) return L;
    for (int tile = 0; tile < kB8TnTiles; ++tile) {
      L = tn_launch(c_type, tile, rows, kt);
      if (strcmp(L.name, want) == 0) return L;
    }
  }
  // Strips, as for int8 (i8.hip): time in rows fetched per CU.
  const bool few_p = Pn <= Qn;
  const int64_t few = few_p ? Pn : Qn, many = few_p ? Qn : Pn;
  int sf = 2, ff = 4;
  double strips = 0.0, wgs = 0.0;
  for (int s = 1; s <= 2; ++s)
    for (int f = 1; f <= 4; f *= 2) {
      if (s == 1 && f > 2) continue;
      const double n = tiles_of(many, 16 * s) * tiles_of(few, 16 * f);
      const double rounds = f >= 4 ? ceil(n / kCus) : (n > kCus ? n / kCus : 1.0);
      const double t = rounds * (16 * s + 16 * f);
      if (strips == 0.0 || t < strips) {
        strips = t;
        sf = s;
        ff = f;
        wgs = n;
      }
    }
  // Block tiles in the same unit, a round of workgroups each.  (us, 256 x 256 / 128 x
  // 128 / with four stages / 64 x 128 / with four, P's factors one for 128 rows, bf16
  // results: 8192^3 410 / 557 / 724 / 813 / 961, 4096 x 4096 x 8192 105 / 137 / 180 /
  // 178 / 241, 8192 x 1024 x 8192 74 / 70 / 92 / 91 / 125, 8192 x 512 x 8192 72 / 49 / 47 /
  // 46 / 62, 8192 x 256 x 8192 71 / 47 / 45 / 42 / 32, 4096 x 1024 x 4096 41 / 29 / 27 /
  // 26 / 36; one for each row: 4096 x 4096 x 8192 134 / 158 / 209 / 190 / 267, 8192 x 1024 x
  // 8192 114 / 83 / 106 / 102 / 132, 8192 x 256 x 8192 112 / 49 / 52 / 43 / 36.  Strips:
  // 8192 x 64 x 8192 16, 300 x 300 x 8192 15, 1536 x 700 x 2048 15.)
  const double cost[kB8TnTiles] = {410.0, 308.0, 308.0, 230.0, 185.0};
  const int bp[kB8TnTiles] = {256, 128, 128, 64, 64}, bq[kB8TnTiles] = {256, 128, 128, 128, 128};
  const int per_cu[kB8TnTiles] = {1, 2, 1, 2, 1};
  int best = -1;
  double time = 0.0;
  for (int tile = 0; tile < kB8TnTiles; ++tile) {
    const double n = tiles_of(Pn, bp[tile]) * tiles_of(Qn, bq[tile]);
    if ((tile == kB8Square4 || tile == kB8Narrow4) && n > kCus) continue;   // (one round only)
    const double t = ceil(n / (kCus * per_cu[tile])) * cost[tile];
    if (best < 0 || t < time) {
      best = tile;
      time = t;
    }
  }
  if ((few <= 32 || strips < time) && launchable((int64_t)wgs, 512))
    return skinny_launch(c_type, sf, ff, few_p, wgs <= kCus && K >= 2048);
  return tn_launch(c_type, best, rows, kt);
}

// (ldp: the ping-pong kernel addresses 128 rows of P in 31 bits.)
Launch choose_nn(int c_type, int64_t Pn, int64_t Qn, int64_t K, int64_t ldp, bool rows) {
  const char* want = getenv("DGEMM_CONFIG");
  const bool kt = K % kBlock != 0, pp = !rows && ldp <= kMaxDescBytes / kBlock;
  auto strip = [&](int sp, int fr) { return launchable(((Pn + sp - 1) / sp) * ((Qn + fr - 1) / fr), 512); };
  if (want != nullptr && *want != 0)
    for (int s = 16; s <= 128; s *= 2)
      for (int f = 16; f <= 128; f *= 2)
        if (nn_strip_fits(s, f) && strip(s, f) && strcmp(nn_skinny_launch(c_type, s, f).name, want) == 0)
          return nn_skinny_launch(c_type, s, f);
  if (want != nullptr && *want != 0)
    for (int tile = pp ? 0 : kB8Nn128; tile < kB8NnTiles; ++tile) {
      const Launch L = nn_launch(c_type, tile, rows, kt);
      if (strcmp(L.name, want) == 0) return L;
    }
  // Block tiles: rounds of a fixed time and one per 1000 k (us).  (256 x 256 / 256 x 192 /
  // 256 x 128 / 256 x 64: 4096^3 59 / 86 / 87 / 120, 8192^3 426 / 521 / 637 / 1032, 2047 x
  // 4099 x 4111 54 / 49 / 90 / 110, 2048 x 4096 x 4096 44 / 42 / 44 / 62, 3000 x 3000 x 4096
  // 48 / 46 / 87 / 96, 512 x 4096 x 4096 41 / 40 / 42 / 32, 300 x 300 x 1000 20 / 18 / 20 / 14.
  // In TN, whose copies and reads are the lighter, 256 x 192 took as long as 256 x 256:
  // 8192 x 1024 x 8192 75 and 74.)
  const double k = (double)K * 1e-3;
  const double round_us[kB8NnTiles] = {9.0 + 7.8 * k, 8.7 + 7.6 * k, 9.0 + 8.1 * k, 7.0 + 6.0 * k};
  const int bq[kB8NnTiles] = {256, 192, 128, 64};
  int best = -1;
  double time = 0.0;
  for (int tile = pp ? 0 : kB8Nn128; tile < kB8NnTiles; ++tile) {
    const double t = ceil(tiles_of(Pn, 256) * tiles_of(Qn, bq[tile]) / kCus) * round_us[tile];
    if (best < 0 || t < time) {
      best = tile;
      time = t;
    }
  }
  // Strips of few rows: 1 us and rounds (each after the first four fifths) of a fixed
  // time and one per 1000 k, the latter a third more with four waves.  (Best block tile /
  // strips of 32 x 16 / 32 x 32 / 64 x 64 / 128 x 64, us: 16 x 8192 x 8192 55 / 22, 16 x 4096 x
  // 4096 29 / 10, 64 x 4096 x 4096 30 / 25 / 16 / 15 / 31, 256 x 4096 x 4096 32 / 87 / 43 / 22 /
  // 33, 512 x 4096 x 4096 32 / 175 / 72 / 37 / 37, 128 x 8192 x 8192 57 / 200 / 89 / 39 / 57,
  // 1024 x 1024 x 8192 56 / 120 / 68 / 39 / 56, 300 x 300 x 1000 13.7 / 4.5 / 4.6 / 6.4 / 11, 4096 x
  // 16 x 4096 31 / 6.7 / 8.1, 2007 x 2295 x 221 15 / - / - / 24, 159 x 6915 x 191 - / - / - / 10.5 / 8.4.)
  int sp = 0, fr = 0;
  double strips = 0.0;
  for (int s = 16; s <= 128; s *= 2)
    for (int f = 16; f <= 128; f *= 2) {
      if (!nn_strip_fits(s, f)) continue;
      const double n = tiles_of(Pn, s) * tiles_of(Qn, f) / kCus;
      const bool four = s * f > 64 * 64;   // waves
      const double round = 0.8 + s * f * (four ? 0.48e-3 : 0.66e-3) +
                           (110.0 + 1.6 * s + 0.55 * f) * (four ? 23e-3 : 17e-3) * k;
      const double t = 1.0 + round * (n > 1.0 ? 1.0 + 0.8 * ceil(n - 1.0) : 1.0);
      if (strips == 0.0 || t < strips) {
        strips = t;
        sp = s;
        fr = f;
      }
    }
  if (strips < time && strip(sp, fr)) return nn_skinny_launch(c_type, sp, fr);
  return nn_launch(c_type, best, rows, kt);
}

struct B8Plan {
  Launch L;
  GemmArgs g;
  int64_t grid;   // 0: nothing to do
};

int plan_block(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const void* B, int64_t ldb, void* C,
               int64_t ldc, int c_type, const Factors& fa, const Factors& fb, int layout, bool pointers, B8Plan* out) {
  if (layout != DGEMM_NN && layout != DGEMM_TN) return DGEMM_ERR_INVALID_LAYOUT;
  if (!valid_type(c_type)) return DGEMM_ERR_INVALID_TYPE;
  if (M < 0 || N < 0 || K < 0 || !valid_rows(fa.rows) || !valid_rows(fb.rows)) return DGEMM_ERR_INVALID_DIM;
  out->grid = 0;
  if (M == 0 || N == 0) return DGEMM_OK;
  if (pointers && ((K > 0 && (A == nullptr || B == nullptr || fa.at == nullptr || fb.at == nullptr)) || C == nullptr))
    return DGEMM_ERR_NULL_POINTER;
  const bool nn = layout == DGEMM_NN;
  const int64_t min_k = K > 0 ? K : 1;
  if (lda < min_k || ldb < (nn ? N : min_k) || ldc < (nn ? N : M)) return DGEMM_ERR_INVALID_LD;
  if (fa.r < 0 || fa.k < 0 || fb.r < 0 || fb.k < 0) return DGEMM_ERR_INVALID_LD;
  if (pointers && K > 0 && (!aligned_to(A, 16) || !aligned_to(B, 16) || lda % 16 != 0 || ldb % 16 != 0))
    return DGEMM_ERR_MISALIGNED;
  if (!aligned_to(C, type_bytes(c_type)) || !aligned_to(fa.at, 4) || !aligned_to(fb.at, 4)) return DGEMM_ERR_MISALIGNED;
  if (!addressable(fa, M) || !addressable(fb, N)) return DGEMM_ERR_UNSUPPORTED;
  GemmArgs g{};
  const Factors &p = nn ? fb : fa, &q = nn ? fa : fb;
  g.P = (const char*)(nn ? B : A); g.ldp = nn ? ldb : lda; g.Pn = nn ? N : M;
  g.Q = (const char*)(nn ? A : B); g.ldq = nn ? lda : ldb; g.Qn = nn ? M : N;
  g.C = C; g.ldc = ldc; g.K = K; g.group = 8;
  g.sp = p.at; g.sp_r = p.r; g.sp_k = p.k; g.sp_shift = p.shift();
  g.sq = q.at; g.sq_r = q.r; g.sq_k = q.k; g.sq_shift = q.shift();
  // Descriptor ranges stay below 2^31 bytes.
  if (K > kMaxDescBytes || g.ldq > kMaxDescBytes / 256) return DGEMM_ERR_UNSUPPORTED;
  if (nn ? K > 0 && g.ldp > kMaxDescBytes / K : g.ldp > kMaxDescBytes / 256) return DGEMM_ERR_UNSUPPORTED;
  if (g.Pn > (int64_t(1) << 40) || g.Qn > (int64_t(1) << 40)) return DGEMM_ERR_UNSUPPORTED;
  const Launch L = nn ? choose_nn(c_type, g.Pn, g.Qn, K, g.ldp, p.rows == 1)
                      : choose_tn(c_type, g.Pn, g.Qn, K, p.rows == 1);
  g.tiles_p = (g.Pn + L.bp - 1) / L.bp;
  g.tiles_q = (g.Qn + L.bq - 1) / L.bq;
  if (g.tiles_p > 0xffffffffll / g.tiles_q || !launchable(g.tiles_p * g.tiles_q, L.threads))
    return DGEMM_ERR_UNSUPPORTED;
  out->L = L;
  out->g = g;
  out->grid = g.tiles_p * g.tiles_q;
  return DGEMM_OK;
}

// The kernel for `rows` rows spread over `groups` groups, by estimated time (us) as for
// int8 (grouped.hip): every group that can have rows is taken to have some.  Block
// tiles take a round a fixed time and one per 1000 k; a skinny workgroup fetches 55
// GB/s per CU and costs 1.35, 1.9 or 4 us besides (16, 32, 64 rows).  Over 100 draws of
// sizes the choice took 1% longer than the best of the seven.  Measured (us, bf16 results, rows through
// an index, 256 x 256 / 128 x 128 / the same with four stages / 128 x 64 / skinny of
// 16 / of 32 / of 64):
//   128 rows, 64 groups, N 2048, K 4096     95 /  84 /  80 /  74 /   54 /   59 /   94
//   512                                    115 / 106 / 106 / 101 /   86 /   89 /  137
//   1024                                   120 / 113 / 118 / 105 /  116 /  110 /  159
//   2048                                   129 / 124 / 125 / 119 /  168 /  152 /  196
//   8192                                   181 / 183 / 196 / 214 /  441 /  362 /  421
//   256 rows, 8 groups, N 4096, K 14336    153 / 120 /  88 / 110 /  143 /  121 /  138
//   1024                                   160 / 155 / 164 / 181 /  402 /  290 /  270
//   2006                                   176 / 266 / 239 / 278 /  679 /  531 /  466
//   30788 rows, 5 groups, N 2990, K 1024   146 / 174 / 257 / 339 / 1178 /  870 /  941
//   12054 rows, 79 groups, N 1021, K 445    41 /  36 /  53 /  62 /  187 /  148 /  166
//   7508 rows, 10 groups, N 3613, K 3612   127 / 168 / 216 / 269
//   238 rows, 43 groups, N 2400, K 89       17 /  11 /  18 /  15 /   19
//   512 rows, 64 groups, N 2048, K 256      20 /  14 /  21 /  19 /   26 /   32 /   57
//   128 rows, 2 groups, N 4096, K 8192      81 /  46 /  44 /  31 /   25 /   22 /   22
int choose_group(int64_t groups, int64_t rows, int64_t N, int64_t K) {
  const double some = (double)(groups < rows ? groups : rows);
  const double weights = some * (double)N * (double)K;   // bytes
  auto tiles = [&](int bq) {
    const double t = (double)rows / bq + 0.5 * some;
    return t > some ? t : some;
  };
  // (The tiles are an estimate, so past the first round part of one more, not whole ones.)
  auto rounds = [&](int bp, int bq, int per_cu, double more) {
    const double n = tiles(bq) * (double)((N + bp - 1) / bp) / (kCus * per_cu);
    return n > 1.0 ? n + more : 1.0;
  };
  auto larger = [](double x, double y) { return x > y ? x : y; };
  double t[kB8GroupKinds];
  t[kB8GroupPp] = larger(rounds(256, 256, 1, 0.75) * (12.5 + (double)K * 10.25e-3), weights / 4.0e6);
  const double full = (double)rows / (128.0 * tiles(128));   // (few rows: less to copy and to store)
  t[kB8GroupSquare] = larger(3.0 + rounds(128, 128, 2, 0.4) * (4.0 + 4.3 * full + (double)K * (4.5e-3 + 3.2e-3 * full)),
                             weights / 3.9e6);
  t[kB8GroupSquare4] = larger(1.0 + rounds(128, 128, 1, 0.5) * (8.0 + (double)K * 6.4e-3), weights / 4.9e6);
  t[kB8GroupThin4] = larger(1.0 + rounds(128, 64, 1, 0.5) * (5.3 + (double)K * 3.7e-3), weights / 4.3e6);
  for (int kind = kB8GroupSkinny16; kind <= kB8GroupSkinny64; ++kind) {
    const int few = 16 << (kind - kB8GroupSkinny16);
    const double wgs = tiles(few) * (double)((N + 31) / 32) / kCus;
    const double fixed = few == 16 ? 1.35 : (few == 32 ? 1.9 : 4.0);
    t[kind] = larger((wgs > 1 ? wgs : 1) * ((32 + few) * (double)K / 55e3 + fixed), weights / 4.9e6) + 3.0;
  }
  // (Sweeps and tests: DGEMM_CONFIG=<kernel name> forces a kernel, as for gemm_*.)
  if (const char* want = getenv("DGEMM_CONFIG"))
    for (int kind = 0; kind < kB8GroupKinds; ++kind)
      for (int c = DGEMM_F32; c <= DGEMM_BF16; ++c)
        if (strcmp(want, grouped_launch(c, kind, false, false).name) == 0) return kind;
  int best = 0;
  for (int kind = 1; kind < kB8GroupKinds; ++kind)
    if (t[kind] < t[best]) best = kind;
  return best;
}

struct GroupPlan {
  Launch L;
  int64_t tiles_p, tiles_q;
};

bool plan_group(int64_t groups, int64_t rows, int64_t N, int64_t K, int c_type, bool gather, GroupPlan* pl) {
  pl->L = grouped_launch(c_type, choose_group(groups, rows, N, K), gather, K % kBlock != 0);
  pl->tiles_p = (N + pl->L.bp - 1) / pl->L.bp;
  const int64_t some = groups < rows ? groups : rows;
  pl->tiles_q = (rows + some * (pl->L.bq - 1)) / pl->L.bq;
  return launchable(pl->tiles_p * pl->tiles_q, pl->L.threads);
}

constexpr int64_t kMaxGroups = int64_t(1) << 20;   // (as gemm_i8_grouped)

int describe(const Launch& L, int64_t tiles_p, int64_t tiles_q, bool none, char* buf, int64_t len) {
  if (buf == nullptr || len <= 0) return DGEMM_OK;
  if (none)
    snprintf(buf, (size_t)len, "none (empty output)");
  else
    snprintf(buf, (size_t)len, "%s tile=%dx%d threads=%d lds=%d grid=%lld tiles=%lldx%lld", L.name, L.bp, L.bq,
             L.threads, L.lds, (long long)(tiles_p * tiles_q), (long long)tiles_p, (long long)tiles_q);
  return DGEMM_OK;
}

}  // namespace
}  // namespace dg

extern "C" {

int gemm_fp8_block(int64_t M, int64_t N, int64_t K, const uint8_t* A, int64_t lda, const uint8_t* B, int64_t ldb,
                   void* C, int64_t ldc, int c_type, const float* scale_a, int rows_a, int64_t scale_a_row,
                   int64_t scale_a_block, const float* scale_b, int rows_b, int64_t scale_b_row, int64_t scale_b_block,
                   int layout, void* stream) {
  using namespace dg;
  B8Plan pl;
  const int st = plan_block(M, N, K, A, lda, B, ldb, C, ldc, c_type, {scale_a, rows_a, scale_a_row, scale_a_block},
                            {scale_b, rows_b, scale_b_row, scale_b_block}, layout, true, &pl);
  if (st != DGEMM_OK || pl.grid == 0) return st;
  return launch_kernel(pl.L.fn, pl.grid, pl.L.threads, &pl.g, stream);
}

int dgemm_fp8_block_config(int c_type, int layout, int rows_a, int rows_b, int64_t M, int64_t N, int64_t K, char* buf,
                           int64_t len) {
  using namespace dg;
  const bool nn = layout == DGEMM_NN;
  auto up = [](int64_t n) { return n > 0 && n < (int64_t(1) << 60) ? (n + 15) / 16 * 16 : (n > 0 ? n : 1); };
  B8Plan pl{};
  const int st = plan_block(M, N, K, nullptr, up(K), nullptr, nn ? up(N) : up(K), nullptr, nn ? N : M, c_type,
                            {nullptr, rows_a, 1, 0}, {nullptr, rows_b, 1, 0}, layout, false, &pl);
  if (st != DGEMM_OK) return st;
  return describe(pl.L, pl.g.tiles_p, pl.g.tiles_q, pl.grid == 0, buf, len);
}

int gemm_fp8_grouped(int64_t groups, int64_t rows, int64_t N, int64_t K, const uint8_t* A, int64_t rows_a, int64_t lda,
                     const int32_t* row_index, const uint8_t* B, int64_t ldb, int64_t group_b, void* C, int64_t ldc,
                     int c_type, const float* scale_a, int64_t scale_a_row, int64_t scale_a_block, const float* scale_b,
                     int64_t scale_b_group, int64_t scale_b_row, int64_t scale_b_block, const int32_t* offsets,
                     void* stream) {
  using namespace dg;
  if (!valid_type(c_type)) return DGEMM_ERR_INVALID_TYPE;
  if (groups < 0 || rows < 0 || N < 0 || K < 0 || rows_a < 0 || group_b < 0) return DGEMM_ERR_INVALID_DIM;
  if (groups > kMaxGroups || N > kMaxCount || groups * N > kMaxCount) return DGEMM_ERR_UNSUPPORTED;
  if (row_index == nullptr && rows_a < rows) return DGEMM_ERR_INVALID_DIM;
  if (rows == 0 || N == 0 || groups == 0) return DGEMM_OK;
  if ((K > 0 && (((A == nullptr || scale_a == nullptr) && rows_a > 0) || B == nullptr || scale_b == nullptr)) ||
      C == nullptr || offsets == nullptr)
    return DGEMM_ERR_NULL_POINTER;
  const int64_t min_ld = K > 0 ? K : 1;
  if (lda < min_ld || ldb < min_ld || ldc < N) return DGEMM_ERR_INVALID_LD;
  if (scale_a_row < 0 || scale_a_block < 0 || scale_b_group < 0 || scale_b_row < 0 || scale_b_block < 0)
    return DGEMM_ERR_INVALID_LD;
  if (K > 0 && (!aligned_to(A, 16) || !aligned_to(B, 16) || lda % 16 != 0 || ldb % 16 != 0 || group_b % 16 != 0))
    return DGEMM_ERR_MISALIGNED;
  if (!aligned_to(C, type_bytes(c_type)) || !aligned_to(scale_a, 4) || !aligned_to(scale_b, 4) ||
      !aligned_to(offsets, 4) || !aligned_to(row_index, 4))
    return DGEMM_ERR_MISALIGNED;
  const Factors fa{scale_a, 1, scale_a_row, scale_a_block}, fb{scale_b, kBlock, scale_b_row, scale_b_block};
  if (!addressable(fa, rows_a) || !addressable(fb, N) || scale_b_group > (int64_t(1) << 40))
    return DGEMM_ERR_UNSUPPORTED;
  if (K > kMaxDescBytes || lda > kMaxDescBytes / 256 || ldb > kMaxDescBytes / 256) return DGEMM_ERR_UNSUPPORTED;
  // With an index all rows of A, and the index itself, go through one descriptor.
  if (rows_a > kMaxDescBytes / 4 || rows > kMaxDescBytes / 4 || N > kMaxDescBytes / 4) return DGEMM_ERR_UNSUPPORTED;
  if (row_index != nullptr && rows_a > 0 && lda > kMaxDescBytes / rows_a) return DGEMM_ERR_UNSUPPORTED;

  // An index over no rows: every row counts as zeros, as with K == 0.
  if (rows_a == 0) K = 0;

  GroupPlan pl;
  if (!plan_group(groups, rows, N, K, c_type, row_index != nullptr, &pl)) return DGEMM_ERR_UNSUPPORTED;
  GroupedArgs a{};
  GemmArgs& g = a.g;
  g.P = (const char*)B; g.ldp = ldb; g.Pn = N;
  g.Q = (const char*)A; g.ldq = lda; g.Qn = rows;
  g.C = C; g.ldc = ldc; g.K = K;
  g.group = 8;
  g.sp = fb.at; g.sp_r = fb.r; g.sp_k = fb.k; g.sp_shift = 7;
  g.sq = fa.at; g.sq_r = fa.r; g.sq_k = fa.k; g.sq_shift = 0;
  a.offsets = offsets; a.groups = groups; a.rows = rows; a.pstride = group_b; a.sp_group = scale_b_group;
  a.gt.index = row_index; a.gt.rows = rows_a;
  g.tiles_p = pl.tiles_p;
  g.tiles_q = pl.tiles_q;
  return launch_kernel(pl.L.fn, pl.tiles_p * pl.tiles_q, pl.L.threads, &a, stream);
}

int dgemm_fp8_grouped_config(int c_type, int gather, int64_t groups, int64_t rows, int64_t N, int64_t K, char* buf,
                             int64_t len) {
  using namespace dg;
  if (!valid_type(c_type)) return DGEMM_ERR_INVALID_TYPE;
  if (groups < 0 || rows < 0 || N < 0 || K < 0) return DGEMM_ERR_INVALID_DIM;
  if (groups > kMaxGroups || N > kMaxCount || groups * N > kMaxCount) return DGEMM_ERR_UNSUPPORTED;
  if (rows > kMaxDescBytes / 4 || N > kMaxDescBytes / 4 || K > kMaxDescBytes / 256) return DGEMM_ERR_UNSUPPORTED;
  GroupPlan pl{};
  const bool none = rows == 0 || N == 0 || groups == 0;
  if (!none && !plan_group(groups, rows, N, K, c_type, gather != 0, &pl)) return DGEMM_ERR_UNSUPPORTED;
  return describe(pl.L, pl.tiles_p, pl.tiles_q, none, buf, len);
}

}  // extern "C"
