// Int8 instantiations of the eight-wave ping-pong kernel (gemm_pp.hpp): TN,
// 256 x 256, FP32, FP16 and BF16 results, with and without K-tail masks.
#include "dgemm.h"
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

}  // namespace

Launch ping_pong_i8_tn(int out, bool kt) {
  switch (out) {
    case DGEMM_F32: return pp_launch<OpI8F>("i8f_tn_256x256_pp", kt);
    case DGEMM_F16: return pp_launch<OpI8H>("i8h_tn_256x256_pp", kt);
    default: return pp_launch<OpI8B>("i8b_tn_256x256_pp", kt);
  }
}

}  // namespace dg
