// Row operators' shared pieces: element types and their conversions.
#pragma once

#include "common.hpp"
#include "dgemm.h"

namespace dg {

inline int type_bytes(int type) { return type == DGEMM_F32 ? 4 : 2; }
inline bool valid_type(int type) { return type >= DGEMM_F32 && type <= DGEMM_BF16; }
inline bool aligned_to(const void* p, int64_t n) { return ((uintptr_t)p) % (uintptr_t)n == 0; }

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

// How rows are accessed: element by element; 16 bytes at once (rows 16-byte
// aligned, h a multiple of a pack); or that and past the caches (nontemporal),
// for matrices larger than they are.
enum RowAccess { kScalar = 0, kVector = 1, kStream = 2 };

// Elements h .. h + N - 1 of a row of H, zeros past its end.  One 16-byte
// access where all of them are there.
template <class T, int A>
__device__ __forceinline__ u32x4 load_pack(const T* row, int64_t h, int64_t H) {
  if (A != kScalar && h + Pack<T>::N <= H) {
    if constexpr (A == kStream) return __builtin_nontemporal_load((const u32x4*)(row + h));
    else return *(const u32x4*)(row + h);
  }
  typename Pack<T>::vec t;
#pragma unroll
  for (int i = 0; i < Pack<T>::N; ++i) t[i] = h + i < H ? row[h + i] : (T)0.0f;
  return __builtin_bit_cast(u32x4, t);
}

template <class T, int A>
__device__ __forceinline__ void store_pack(T* row, int64_t h, int64_t H, u32x4 v) {
  if (A != kScalar && h + Pack<T>::N <= H) {
    if constexpr (A == kStream) __builtin_nontemporal_store(v, (u32x4*)(row + h));
    else *(u32x4*)(row + h) = v;
    return;
  }
  const typename Pack<T>::vec t = __builtin_bit_cast(typename Pack<T>::vec, v);
#pragma unroll
  for (int i = 0; i < Pack<T>::N; ++i)
    if (h + i < H) row[h + i] = t[i];
}

}  // namespace dg
