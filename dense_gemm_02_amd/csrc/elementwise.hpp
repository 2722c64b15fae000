// Row operators' shared pieces: element types and their conversions.
#pragma once

#include <type_traits>

#include "common.hpp"
#include "dgemm.h"

namespace dg {

inline int type_bytes(int type) { return type == DGEMM_F32 ? 4 : 2; }
inline bool valid_type(int type) { return type >= DGEMM_F32 && type <= DGEMM_BF16; }

// Row matrices of this many bytes and more are read once and written past the
// caches (nontemporal).  Measured on tokens dispatched to eight rows of 8 KiB
// each, a copy of the rows, and combined: 64 MiB of rows 56 us through the
// caches, 62 past them; 128 MiB 129 and 114; 256 MiB 247 and 229.  256 MiB
// of rows quantised: 77 and 66.
constexpr int64_t kStreamBytes = 96ll << 20;

// f(T{}) with the element type of a dgemm_type.
template <class F>
auto with_type(int type, F f) {
  if (type == DGEMM_F32) return f(float{});
  if (type == DGEMM_F16) return f(_Float16{});
  return f(__bf16{});
}

// Sixteen bytes of a row as FP32 values and back (rounded to nearest-even).
template <class T>
struct Pack {
  static constexpr int N = 16 / (int)sizeof(T);
  typedef T vec __attribute__((ext_vector_type(N)));
  __device__ static void unpack(u32x4 v, float (&f)[N]) {
    const vec t = __builtin_bit_cast(vec, v);
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = (float)t[i];
  }
  __device__ static u32x4 pack(const float (&f)[N]) {
    vec t;
#pragma unroll
    for (int i = 0; i < N; ++i) t[i] = (T)f[i];
    return __builtin_bit_cast(u32x4, t);
  }
};

// Sixteen bytes at the alignment of T.  (gfx950 serves global accesses of any
// alignment; 16-byte ones of aligned and unaligned rows are the same
// instruction.)
typedef u32x4 u32x4_at4 __attribute__((aligned(4)));
template <class T>
struct Unaligned {
  typedef std::conditional_t<sizeof(T) == 2, u32x4_at2, u32x4_at4> type;
};

// Elements h .. h + N - 1 of a row of H, zeros past its end, in one access
// where all of them are there.  STREAM: past the caches (nontemporal).
template <class T, bool STREAM>
__device__ __forceinline__ u32x4 load_pack(const T* row, int64_t h, int64_t H) {
  if (h + Pack<T>::N <= H) {
    const typename Unaligned<T>::type* p = (const typename Unaligned<T>::type*)(row + h);
    if constexpr (STREAM) return __builtin_nontemporal_load(p);
    else return *p;
  }
  typename Pack<T>::vec t;
#pragma unroll
  for (int i = 0; i < Pack<T>::N; ++i) t[i] = h + i < H ? row[h + i] : (T)0.0f;
  return __builtin_bit_cast(u32x4, t);
}

template <class T, bool STREAM>
__device__ __forceinline__ void store_pack(T* row, int64_t h, int64_t H, u32x4 v) {
  if (h + Pack<T>::N <= H) {
    typename Unaligned<T>::type* p = (typename Unaligned<T>::type*)(row + h);
    if constexpr (STREAM) __builtin_nontemporal_store(v, p);
    else *p = v;
    return;
  }
  const typename Pack<T>::vec t = __builtin_bit_cast(typename Pack<T>::vec, v);
#pragma unroll
  for (int i = 0; i < Pack<T>::N; ++i)
    if (h + i < H) row[h + i] = t[i];
}

}  // namespace dg
