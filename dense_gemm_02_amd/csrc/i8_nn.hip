// Int8 NN instantiations of the skinny kernel (gemm_i8_skinny_nn.hpp), FP32,
// FP16 and BF16 results, and the rule that picks one.
#include <math.h>

#include "dgemm.h"
#include "gemm_i8_skinny_nn.hpp"
#include "launch.hpp"

namespace dg {
namespace {

template <class Op, int SP, int FF, int NW>
Launch launch() {
  using Cfg = SkinnyNnCfg<SP, FF, NW>;
  return Launch{(const void*)&gemm_i8_skinny_nn_kernel<Op, SP, FF, NW>, "i8_nn_skinny", SP, Cfg::FR, Cfg::NT, Cfg::LDS,
                true};
}

// (Four waves where eight waves' stages do not fit the LDS.)
template <class Op>
Launch pick(int sp, int fr) {
  switch (sp) {
    case 16: return fr == 16 ? launch<Op, 16, 1, 8>() : launch<Op, 16, 2, 8>();
    case 32:
      if (fr <= 32) return fr == 16 ? launch<Op, 32, 1, 8>() : launch<Op, 32, 2, 8>();
      return fr == 64 ? launch<Op, 32, 4, 8>() : launch<Op, 32, 8, 8>();
    case 64:
      if (fr <= 32) return fr == 16 ? launch<Op, 64, 1, 8>() : launch<Op, 64, 2, 8>();
      return fr == 64 ? launch<Op, 64, 4, 8>() : launch<Op, 64, 8, 4>();
    default:
      if (fr <= 32) return fr == 16 ? launch<Op, 128, 1, 8>() : launch<Op, 128, 2, 8>();
      return launch<Op, 128, 4, 4>();
  }
}

}  // namespace

// Estimated times in a unit of 20 ns per 1000 k: a round of workgroups of SP x FR
// costs 110 + 1.6 SP + 0.55 FR (a tenth more with four waves), further ones
// four fifths of that each; the block kernels 497 a round of 256 x 128 tiles and
// 760 of 256 x 256.  Measured (us, bf16 results; skinny / block): 16 x 8192 x
// 8192 28.5 / 92, 16 x 4096 x 4096 10.2 / 43, 16 x 28672 x 8192 54 / 98, 128 x
// 8192 x 8192 37 / 93, 8192 x 16 x 8192 12.7 / 84, 300 x 300 x 1000 4.5 / 30,
// 1024 x 1024 x 8192 35.5 / 81, 700 x 2000 x 3000 23.7 / 41.7.
bool skinny_i8_nn(int out, int64_t Pn, int64_t Qn, Launch* L) {
  constexpr double kCus = 256.0;
  auto tiles = [](int64_t n, int64_t b) { return (double)((n + b - 1) / b); };
  int sp = 0, fr = 0;
  double best = 0.0;
  for (int s = 16; s <= 128; s *= 2)
    for (int f = 16; f <= 128; f *= 2) {
      if ((s == 16 && f > 32) || (s == 128 && f > 64)) continue;
      const double n = tiles(Pn, s) * tiles(Qn, f) / kCus;
      double t = (110.0 + 1.6 * s + 0.55 * f) * (n > 1.0 ? 1.0 + 0.8 * (n - 1.0) : 1.0);
      if (s * f > 64 * 64) t *= 1.1;
      if (best == 0.0 || t < best) {
        best = t;
        sp = s;
        fr = f;
      }
    }
  const double narrow = 497.0 * ceil(tiles(Pn, 256) * tiles(Qn, 128) / kCus);
  const double square = 760.0 * ceil(tiles(Pn, 256) * tiles(Qn, 256) / kCus);
  if (best > (narrow < square ? narrow : square)) return false;
  if (!launchable(((Pn + sp - 1) / sp) * ((Qn + fr - 1) / fr), 512)) return false;   // (2^30 rows; as in TN)
  *L = out == DGEMM_F32 ? pick<OpI8F>(sp, fr) : (out == DGEMM_F16 ? pick<OpI8H>(sp, fr) : pick<OpI8B>(sp, fr));
  return true;
}

}  // namespace dg
