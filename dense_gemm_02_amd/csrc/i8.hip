// Int8 instantiations, FP32, FP16 and BF16 results: the eight-wave ping-pong
// kernel (gemm_pp.hpp; TN, 256 x 256, with and without K-tail masks; 8192^3
// in 372-392 us, 2.8-2.95 POPS, bound by the chip's power limit as FP8 is) and
// the skinny kernel (gemm_i8_skinny.hpp; TN).
#include <math.h>

#include "dgemm.h"
#include "gemm_i8_skinny.hpp"
#include "gemm_pp.hpp"
#include "launch.hpp"

namespace dg {
namespace {

template <class Op, bool KT>
__global__ void __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2)))
gemm_i8_pp(const GemmArgs a) {
  gemm_pp_body<Op, KT>(a, GridTile{});
}

template <class Op>
Launch pp_launch(const char* name, bool kt) {
  using Cfg = PpCfg<Op>;
  const void* fn = kt ? (const void*)&gemm_i8_pp<Op, true> : (const void*)&gemm_i8_pp<Op, false>;
  return Launch{fn, name, Cfg::BP, Cfg::BQ, Cfg::NT, Cfg::LDS, false};
}

template <class Op, int SF, int FF, int NW, int D>
Launch skinny_launch(bool few_p) {
  using Cfg = SkinnyI8Cfg<SF, FF, NW, D>;
  // (bp x bq: a strip of the one operand, few rows of the other)
  if (few_p)
    return Launch{(const void*)&gemm_i8_skinny_kernel<Op, SF, FF, NW, D, true>, "i8_tn_skinny_a", Cfg::FR, Cfg::SR,
                  Cfg::NT, Cfg::LDS, false};
  return Launch{(const void*)&gemm_i8_skinny_kernel<Op, SF, FF, NW, D, false>, "i8_tn_skinny_b", Cfg::SR, Cfg::FR,
                Cfg::NT, Cfg::LDS, false};
}

template <class Op, int SF>
Launch skinny(bool few_p, int ff, bool two) {
  // Two stages of copies in flight where a CU has one workgroup and the waves
  // more than a stage each, else one (bf16 results, 16 rows: 8192 x 8192 14.7
  // us with two and 15.5 with one; 28672 x 8192 48.4 and 45.4; 5120 x 1040 5.1
  // and 4.3; more than 32 few rows leave LDS for one).
  switch (ff) {
    case 1: return two ? skinny_launch<Op, SF, 1, 8, 2>(few_p) : skinny_launch<Op, SF, 1, 8, 1>(few_p);
    case 2: return two ? skinny_launch<Op, SF, 2, 8, 2>(few_p) : skinny_launch<Op, SF, 2, 8, 1>(few_p);
    case 4: return skinny_launch<Op, 2, 4, 8, 1>(few_p);
    default: return skinny_launch<Op, 2, 8, 8, 1>(few_p);
  }
}

}  // namespace

// A workgroup of the skinny kernel fetches (strip + few) rows of K bytes at
// about 40 GB/s per CU, whatever the rest does: its time is counted in rows per
// CU, with fewer workgroups than CUs taking as long as one each.  The block
// kernels in the same unit: 64 x 128 tiles 185 rows while there is at most one
// per CU and 230 with two, 128 x 128 tiles 308 per two per CU, 256 x 256 tiles
// 410 a round.  Up to 32 rows on one side the stream of the other bounds the
// skinny kernel, and it always won.  (us, bf16 results, skinny / the best
// block kernel: 8192 x 64 x 8192 20.5 / 32, 8192 x 128 x 8192 29.2 / 33, 8192 x
// 160 x 8192 57 / 32, 4096 x 256 x 4096 13.6 / 18.1, 1024 x 1024 x 4096 15.2 /
// 18.2, 1536 x 700 x 2048 15.6 / 12.6, 28672 x 64 x 8192 68 / 57, 57344 x 32 x
// 4096 50.5 / 53.6.)
bool skinny_i8_tn(int out, int64_t Pn, int64_t Qn, int64_t K, Launch* L) {
  constexpr double kCus = 256.0;
  auto tiles = [](int64_t n, int64_t b) { return (double)((n + b - 1) / b); };
  const bool few_p = Pn <= Qn;
  const int64_t few = few_p ? Pn : Qn, many = few_p ? Qn : Pn;
  int sf = 2, ff = 8;
  double best = 0.0, wgs = 0.0;
  for (int s = 1; s <= 2; ++s)
    for (int f = 1; f <= 8; f *= 2) {
      if (s == 1 && f > 2) continue;   // (as many workgroups as half the few rows and strips of 32, more to fetch)
      const double n = tiles(many, 16 * s) * tiles(few, 16 * f);
      // (From 64 few rows on a CU's LDS holds one workgroup, so rounds are whole.)
      const double rounds = f >= 4 ? ceil(n / kCus) : (n > kCus ? n / kCus : 1.0);
      const double t = rounds * (16 * s + 16 * f);
      if (best == 0.0 || t < best) {
        best = t;
        sf = s;
        ff = f;
        wgs = n;
      }
    }
  const double t64 = tiles(Pn, 64) * tiles(Qn, 128), t128 = tiles(Pn, 128) * tiles(Qn, 128);
  const double t256 = tiles(Pn, 256) * tiles(Qn, 256);
  const double small = t64 <= kCus ? 185.0 : (t64 <= 2 * kCus ? 230.0 : 308.0 * ceil(t128 / (2 * kCus)));
  const double large = 410.0 * ceil(t256 / kCus);
  if (few > 32 && best > (small < large ? small : large)) return false;
  if (!launchable((int64_t)wgs, 512)) return false;   // (2^28 rows of 16 bytes; the block tiles take these)
  const bool two = wgs <= kCus && K >= 2048;
  auto pick = [&](auto op) {
    using Op = decltype(op);
    return sf == 1 ? skinny<Op, 1>(few_p, ff, two) : skinny<Op, 2>(few_p, ff, two);
  };
  *L = out == DGEMM_F32 ? pick(OpI8F{}) : (out == DGEMM_F16 ? pick(OpI8H{}) : pick(OpI8B{}));
  return true;
}

Launch ping_pong_i8_tn(int out, bool kt) {
  switch (out) {
    case DGEMM_F32: return pp_launch<OpI8F>("i8f_tn_256x256_pp", kt);
    case DGEMM_F16: return pp_launch<OpI8H>("i8h_tn_256x256_pp", kt);
    default: return pp_launch<OpI8B>("i8b_tn_256x256_pp", kt);
  }
}

}  // namespace dg
