// quantize_i8: rows to int8 with one factor per row.
//
//   s = fl(max_k |x_k| / 127),  q_k = rne(x_k / s)
//
// The quotient is rounded once, as if computed exactly: n = rint(x * fl(1/s))
// can be off by one only next to the middle between two integers, and the
// remainder x - n s (exact there: a multiple of the operands' last place that
// is no larger than s) tells.
#include "elementwise.hpp"
#include "launch.hpp"

namespace dg {
namespace {

struct QuantArgs {
  const void* X;
  int64_t ldx;
  int8_t* Q;
  int64_t ldq;
  float* scale;
  int64_t rows, K;
};

// What turns a row's maximum (as bits of |x|; NaN above infinity above all
// numbers) into its quantisation: the stored scale, and the scale and its
// reciprocal after the exact factor `up` that keeps tiny rows away from
// subnormal reciprocals.
struct RowScale {
  float scale, s, inv, up;
};

__device__ __forceinline__ RowScale row_scale(uint32_t max_bits) {
  RowScale r;
  const float m = __builtin_bit_cast(float, max_bits);
  r.scale = m / 127.0f;
  r.up = r.scale < 0x1p-60f ? 0x1p80f : 1.0f;
  r.s = r.scale * r.up;
  // 0 where nothing is left to quantise: a scale of 0, infinity or NaN.
  r.inv = (max_bits < 0x7f800000u && r.scale > 0.0f) ? 1.0f / r.s : 0.0f;
  return r;
}

__device__ __forceinline__ int quantize_one(float x, const RowScale& r) {
  if (r.inv == 0.0f) return 0;
  const float v = x * r.up;
  float n = __builtin_rintf(v * r.inv);
  const float rest = __builtin_fmaf(-n, r.s, v), half = 0.5f * r.s;
  // Off the nearest integer, or on the middle but on the odd side.
  const bool odd = ((int)n & 1) != 0;
  if (rest > half || (rest == half && odd)) n += 1.0f;
  else if (rest < -half || (rest == -half && odd)) n -= 1.0f;
  n = n > 127.0f ? 127.0f : (n < -127.0f ? -127.0f : n);
  return (int)n;
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
  for (int d = 32; d > 0; d /= 2) {
    const uint32_t o = (uint32_t)__shfl_xor((int)v, d);
    v = o > v ? o : v;
  }
  return v;
}

template <class T>
__global__ void __launch_bounds__(256) quantize_kernel(const QuantArgs a) {
  __shared__ uint32_t part[4];
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = (const T*)a.X + row * a.ldx;
    int8_t* q = a.Q + row * a.ldq;
    uint32_t m = 0;
    for (int64_t k = threadIdx.x; k < a.K; k += 256) {
      const uint32_t b = __builtin_bit_cast(uint32_t, (float)x[k]) & 0x7fffffffu;
      m = b > m ? b : m;
    }
    m = wave_max(m);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 4; ++w) m = part[w] > m ? part[w] : m;
    const RowScale r = row_scale(m);
    if (threadIdx.x == 0) a.scale[row] = r.scale;
    for (int64_t k = threadIdx.x; k < a.K; k += 256) q[k] = (int8_t)quantize_one((float)x[k], r);
  }
}

}  // namespace
}  // namespace dg

extern "C" int quantize_i8(int64_t rows, int64_t K, const void* X, int64_t ldx, int x_type, int8_t* Q, int64_t ldq,
                           float* scale, void* stream) {
  using namespace dg;
  if (!valid_type(x_type)) return DGEMM_ERR_INVALID_TYPE;
  if (rows < 0 || K < 0) return DGEMM_ERR_INVALID_DIM;
  if (rows == 0) return DGEMM_OK;
  if ((K > 0 && (X == nullptr || Q == nullptr)) || scale == nullptr) return DGEMM_ERR_NULL_POINTER;
  if (ldx < K || ldq < K) return DGEMM_ERR_INVALID_LD;
  if (!aligned_to(X, type_bytes(x_type)) || !aligned_to(scale, 4)) return DGEMM_ERR_MISALIGNED;
  if (rows > 0x7fffffff) return DGEMM_ERR_UNSUPPORTED;
  QuantArgs a{X, ldx, Q, ldq, scale, rows, K};
  return with_type(x_type, [&](auto t) {
    return launch_kernel((const void*)&quantize_kernel<decltype(t)>, rows, 256, &a, stream);
  });
}
