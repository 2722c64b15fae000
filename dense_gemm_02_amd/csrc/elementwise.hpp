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

}  // namespace dg
