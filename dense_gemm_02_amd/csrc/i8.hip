// Int8 instantiations, FP32, FP16 and BF16 results: the eight-wave ping-pong
// kernel (gemm_pp.hpp; TN, 256 x 256, with and without K-tail masks) and the
// skinny kernel (gemm_i8_skinny.hpp; TN).
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
  // (bp x bq: a strip of the one operand, all rows of the other)
  if (few_p)
    return Launch{(const void*)&gemm_i8_skinny_kernel<Op, SF, FF, NW, D, true>, "i8_tn_skinny_a", Cfg::FR, Cfg::SR,
                  Cfg::NT, Cfg::LDS, false};
  return Launch{(const void*)&gemm_i8_skinny_kernel<Op, SF, FF, NW, D, false>, "i8_tn_skinny_b", Cfg::SR, Cfg::FR,
                Cfg::NT, Cfg::LDS, false};
}

template <class Op, int FF>
Launch skinny_few(bool few_p, int64_t many, int64_t K) {
  if (i8_strip(many) == 32) {
    // A second stage of copies in flight where a CU has one workgroup and the
    // waves more than a stage each (bf16 results, 16 rows: 8192 x 8192 14.7
    // us with two and 15.5 with one; 28672 x 8192 48.4 and 45.4; 5120 x 1040
    // 5.1 and 4.3).
    if constexpr (FF <= 2)
      if (many <= 32 * 256 && K >= 2048) return skinny_launch<Op, 2, FF, 8, 2>(few_p);
    return skinny_launch<Op, 2, FF, 8, 1>(few_p);
  }
  if constexpr (FF <= 2)
    if (K >= 2048) return skinny_launch<Op, 1, FF, 8, 2>(few_p);
  return skinny_launch<Op, 1, FF, 8, 1>(few_p);
}

template <class Op>
Launch skinny(bool few_p, int64_t few, int64_t many, int64_t K) {
  if (few <= 16) return skinny_few<Op, 1>(few_p, many, K);
  if (few <= 32) return skinny_few<Op, 2>(few_p, many, K);
  if (few <= 64) return skinny_few<Op, 4>(few_p, many, K);
  return skinny_few<Op, 8>(few_p, many, K);
}

}  // namespace

Launch skinny_i8_tn(int out, bool few_p, int64_t few, int64_t many, int64_t K) {
  switch (out) {
    case DGEMM_F32: return skinny<OpI8F>(few_p, few, many, K);
    case DGEMM_F16: return skinny<OpI8H>(few_p, few, many, K);
    default: return skinny<OpI8B>(few_p, few, many, K);
  }
}

Launch ping_pong_i8_tn(int out, bool kt) {
  switch (out) {
    case DGEMM_F32: return pp_launch<OpI8F>("i8f_tn_256x256_pp", kt);
    case DGEMM_F16: return pp_launch<OpI8H>("i8h_tn_256x256_pp", kt);
    default: return pp_launch<OpI8B>("i8b_tn_256x256_pp", kt);
  }
}

}  // namespace dg
