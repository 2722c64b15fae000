// quantize_i8: rows to int8 with one factor per row.
//
//   s = fl(max_k |x_k| / 127),  q_k = rne(x_k / s)
//
// The quotient is rounded once, as if computed exactly: n = rint(x * fl(1/s))
// can be off by one only next to the middle between two integers, and the
// remainder x - n s (exact there: a multiple of the operands' last place that
// is no larger than s) tells.
//
// HBM bounds it: e + 1 bytes an element, with about eight vector
// instructions between (one for the maximum, seven to round, check and pack).
// 16384 x 8192 bf16 (403 MB): 61.5 us, 6.5 TB/s; 16 rows of 8192, where the
// latency of one row counts: 3.8 us.
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

// Integers near 0 in the last bits of a float: x + kMagic rounds x to the
// nearest-even integer n, whose low byte is that of the sum.
constexpr float kMagic = 0x1.8p23f;

// Four values to four bytes.  Nearly always every |x - n s| is below s / 2
// and n is right; else, and in rows so small that s is subnormal and a
// quotient can pass 127, the lane goes through the values one by one.
__device__ __forceinline__ uint32_t quantize4(const float* f, const RowScale& r) {
  uint32_t t[4];
  float worst = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float v = f[i], u = __builtin_fmaf(v, r.inv, kMagic);
    const float rest = __builtin_fmaf(-(u - kMagic), r.s, v);
    worst = __builtin_fmaxf(worst, __builtin_fabsf(rest));
    t[i] = __builtin_bit_cast(uint32_t, u);
  }
  if (worst >= 0.5f * r.s || r.up != 1.0f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float v = f[i] * r.up;
      float n = __builtin_rintf(v * r.inv);
      const float rest = __builtin_fmaf(-n, r.s, v), half = 0.5f * r.s;
      // Off the nearest integer, or on the middle but on the odd side.
      const bool odd = ((int)n & 1) != 0;
      if (rest > half || (rest == half && odd)) n += 1.0f;
      else if (rest < -half || (rest == -half && odd)) n -= 1.0f;
      t[i] = (uint32_t)(int)__builtin_fminf(__builtin_fmaxf(n, -127.0f), 127.0f);
    }
  }
  // Low bytes of t[0 .. 3], in order.
  const uint32_t lo = __builtin_amdgcn_perm(t[1], t[0], 0x0c0c0400u);
  const uint32_t hi = __builtin_amdgcn_perm(t[3], t[2], 0x0c0c0400u);
  return lo | hi << 16;
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
  for (int d = 32; d > 0; d /= 2) {
    const uint32_t o = (uint32_t)__shfl_xor((int)v, d);
    v = o > v ? o : v;
  }
  return v;
}

// The maximum of a row over its WPR waves.
template <int WPR>
__device__ __forceinline__ uint32_t row_max(uint32_t m, uint32_t* part, int wave) {
  m = wave_max(m);
  if constexpr (WPR == 1) return m;
  if (lane_id() == 0) part[wave] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < WPR; ++w) m = part[w] > m ? part[w] : m;
  return m;
}

// The running maximum of |x| over packs: of the bits of 16-bit values two at
// a time, or of FP32 values, ordered as their magnitudes in either case (NaN
// highest).
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

template <class T>
__device__ __forceinline__ uint32_t max_pack(u32x4 v, uint32_t m) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 2) {
      const u16x2 b = __builtin_bit_cast(u16x2, v[i] & 0x7fff7fffu);
      m = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, m), b));
    } else {
      const uint32_t b = v[i] & 0x7fffffffu;
      m = b > m ? b : m;
    }
  }
  return m;
}

// ... as the bits of one FP32 value.
template <class T>
__device__ __forceinline__ uint32_t max_value(uint32_t m) {
  if constexpr (sizeof(T) == 4) {
    return m;
  } else {
    const uint16_t b = (uint16_t)((m & 0xffffu) > (m >> 16) ? m & 0xffffu : m >> 16);
    return __builtin_bit_cast(uint32_t, (float)__builtin_bit_cast(T, b));
  }
}

// Quantised values of one pack to q[k ..].
template <class T>
__device__ __forceinline__ void store_quantized(int8_t* q, int64_t k, int64_t K, const float (&f)[Pack<T>::N],
                                                const RowScale& r) {
  constexpr int N = Pack<T>::N;
  uint32_t d[N / 4];
#pragma unroll
  for (int i = 0; i < N / 4; ++i) d[i] = r.inv == 0.0f ? 0u : quantize4(f + 4 * i, r);
  if (k + N <= K) {
    __builtin_memcpy(q + k, d, N);
    return;
  }
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (k + i < K) q[k + i] = (int8_t)(d[i / 4] >> (8 * (i % 4)));
}

// WPR waves of a workgroup of four take a row and hold all of it in
// registers, NP packs of 16 bytes a lane: the row is read once.
template <class T, bool STREAM, int WPR, int NP>
__global__ void __launch_bounds__(256) quantize_kernel(const QuantArgs a) {
  using P = Pack<T>;
  __shared__ uint32_t part[4];
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int64_t row = (int64_t)blockIdx.x * (4 / WPR) + wave / WPR;
  if (WPR < 4 && row >= a.rows) return;   // (WPR 4: every workgroup has a row)
  const T* x = (const T*)a.X + row * a.ldx;
  const int64_t k0 = (wave % WPR * 64 + lane_id()) * P::N;
  u32x4 v[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) v[i] = load_pack<T, STREAM>(x, k0 + i * (WPR * 64 * P::N), a.K);
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < NP; ++i) m = max_pack<T>(v[i], m);
  const RowScale r = row_scale(row_max<WPR>(max_value<T>(m), part, wave));
  if (wave % WPR == 0 && lane_id() == 0) a.scale[row] = r.scale;
  int8_t* q = a.Q + row * a.ldq;
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    float f[P::N];
    P::unpack(v[i], f);
    store_quantized<T>(q, k0 + i * (WPR * 64 * P::N), a.K, f, r);
  }
}

// Rows longer than the registers hold: read twice (the second time mostly
// from the caches), 1024 threads a row.
template <class T>
__global__ void __launch_bounds__(1024) quantize_long_kernel(const QuantArgs a) {
  using P = Pack<T>;
  __shared__ uint32_t part[16];
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int64_t row = blockIdx.x;
  const T* x = (const T*)a.X + row * a.ldx;
  uint32_t m = 0;
  for (int64_t k = (int64_t)threadIdx.x * P::N; k < a.K; k += 1024 * P::N)
    m = max_pack<T>(load_pack<T, false>(x, k, a.K), m);
  const RowScale r = row_scale(row_max<16>(max_value<T>(m), part, wave));
  if (threadIdx.x == 0) a.scale[row] = r.scale;
  for (int64_t k = (int64_t)threadIdx.x * P::N; k < a.K; k += 1024 * P::N) {
    float f[P::N];
    P::unpack(load_pack<T, false>(x, k, a.K), f);
    store_quantized<T>(a.Q + row * a.ldq, k, a.K, f, r);
  }
}

// The kernel for rows of K elements and the rows per workgroup of 256 (0: the
// long one, a row per workgroup of 1024): the fewest registers that hold the
// row, a wave for up to two packs a lane.
template <class T, bool STREAM>
const void* quantize_choice(int64_t K, int* rows) {
  const int64_t packs = (K + Pack<T>::N - 1) / Pack<T>::N;
  *rows = packs <= 128 ? 4 : (packs <= 256 * 8 ? 1 : 0);
  if (packs <= 64) return (const void*)&quantize_kernel<T, STREAM, 1, 1>;
  if (packs <= 128) return (const void*)&quantize_kernel<T, STREAM, 1, 2>;
  if (packs <= 256) return (const void*)&quantize_kernel<T, STREAM, 4, 1>;
  if (packs <= 512) return (const void*)&quantize_kernel<T, STREAM, 4, 2>;
  if (packs <= 1024) return (const void*)&quantize_kernel<T, STREAM, 4, 4>;
  if (packs <= 2048) return (const void*)&quantize_kernel<T, STREAM, 4, 8>;
  return (const void*)&quantize_long_kernel<T>;
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
  if (rows > 0x7fffffff || K > 0x7fffffff) return DGEMM_ERR_UNSUPPORTED;
  QuantArgs a{X, ldx, Q, ldq, scale, rows, K};
  int per = 0;
  const bool stream_rows = rows * K >= kStreamBytes / type_bytes(x_type);
  const void* fn = with_type(x_type, [&](auto t) {
    using T = decltype(t);
    return stream_rows ? quantize_choice<T, true>(K, &per) : quantize_choice<T, false>(K, &per);
  });
  const int threads = per > 0 ? 256 : 1024;
  if (per == 0) per = 1;
  const int64_t step = kMaxRowBlocks * per;
  for (int64_t at = 0; at < rows; at += step) {
    QuantArgs part = a;
    if (K > 0) {   // (else both may be null)
      part.X = (const char*)X + at * ldx * type_bytes(x_type);
      part.Q = Q + at * ldq;
    }
    part.scale = scale + at;
    part.rows = rows - at < step ? rows - at : step;
    if (const int st = launch_kernel(fn, (part.rows + per - 1) / per, threads, &part, stream)) return st;
  }
  return DGEMM_OK;
}
