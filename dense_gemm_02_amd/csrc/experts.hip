// Tokens sorted by expert and back (mixture of experts): expert_sort,
// expert_dispatch, expert_combine and expert_combine_grad.
#include "elementwise.hpp"
#include "launch.hpp"

namespace dg {
namespace {

constexpr int kMaxExperts = 1024;
constexpr int64_t kMaxCount = 0x7fffffff;

// ---- sort -------------------------------------------------------------------------

struct SortArgs {
  const void* ids;
  int32_t* offsets;
  int32_t* slot;
  int32_t* pair;
  int32_t* token;
  int64_t n;
  int k;
  int experts;
};

template <class Id>
__device__ __forceinline__ int expert_of(const SortArgs& a, int64_t i) {
  if (i >= a.n) return -1;
  const Id id = ((const Id*)a.ids)[i];
  return id >= 0 && id < (Id)a.experts ? (int)id : -1;
}

// One workgroup: counts, their prefix sums, then the pairs in order, 1024 at
// a time; a pair's place among those of its expert is found wave by wave.
template <class Id>
__global__ void __launch_bounds__(1024) sort_kernel(const SortArgs a) {
  __shared__ int32_t base[kMaxExperts + 1];
  const int tid = threadIdx.x;
  for (int e = tid; e <= a.experts; e += 1024) base[e] = 0;
  __syncthreads();
  for (int64_t i = tid; i < a.n; i += 1024) {
    const int e = expert_of<Id>(a, i);
    if (e >= 0) atomicAdd(&base[e], 1);
  }
  __syncthreads();
  if (tid == 0) {
    int32_t sum = 0;
    for (int e = 0; e <= a.experts; ++e) {
      const int32_t c = base[e];
      base[e] = sum;
      a.offsets[e] = sum;
      sum += c;
    }
  }
  __syncthreads();
  const int32_t kept = base[a.experts];
  for (int64_t i0 = 0; i0 < a.n; i0 += 1024) {
    const int64_t i = i0 + tid;
    const int e = expert_of<Id>(a, i);
    for (int w = 0; w < 16; ++w) {
      if (w == tid >> 6) {
        uint64_t same = __ballot(e >= 0);
        for (int b = 1; b < kMaxExperts; b *= 2) {
          const uint64_t m = __ballot((e & b) != 0);
          same &= (e & b) != 0 ? m : ~m;
        }
        const int rank = __popcll(same & ((1ull << (tid & 63)) - 1ull));
        int32_t at = -1;
        if (e >= 0) at = base[e] + rank;
        if (i < a.n) a.slot[i] = at;
        if (e >= 0) {
          a.pair[at] = (int32_t)i;
          if (a.token != nullptr) a.token[at] = (int32_t)i / a.k;
          if (rank == 0) base[e] += __popcll(same);
        }
      }
      __syncthreads();
    }
  }
  for (int64_t n = kept + tid; n < a.n; n += 1024) {
    a.pair[n] = -1;
    if (a.token != nullptr) a.token[n] = -1;
  }
}

// ---- rows -------------------------------------------------------------------------

struct RowArgs {
  const void* x;      // rows by token, in
  int64_t ldx;
  const void* y;      // sorted rows, in
  int64_t ldy;
  void* out;          // rows by token (combine) or sorted rows, out
  int64_t ldo;
  const int32_t* slot;
  const float* w;
  float* dw;
  int64_t tokens, k, H, rows;
};

__device__ __forceinline__ int64_t slot_of(const RowArgs& a, int64_t pair) {
  const int64_t s = a.slot[pair];
  return s >= 0 && s < a.rows ? s : -1;
}

template <class T>
__global__ void __launch_bounds__(256) dispatch_kernel(const RowArgs a) {
  for (int64_t t = blockIdx.x; t < a.tokens; t += gridDim.x) {
    const T* x = (const T*)a.x + t * a.ldx;
    for (int64_t j = 0; j < a.k; ++j) {
      const int64_t s = slot_of(a, t * a.k + j);
      if (s < 0) continue;
      for (int64_t h = threadIdx.x; h < a.H; h += 256) ((T*)a.out)[s * a.ldo + h] = x[h];
    }
  }
}

template <class T>
__global__ void __launch_bounds__(256) combine_kernel(const RowArgs a) {
  for (int64_t t = blockIdx.x; t < a.tokens; t += gridDim.x) {
    for (int64_t h = threadIdx.x; h < a.H; h += 256) {
      float sum = 0.0f;
      for (int64_t j = 0; j < a.k; ++j) {
        const int64_t s = slot_of(a, t * a.k + j);
        if (s < 0) continue;
        const float y = (float)((const T*)a.y)[s * a.ldy + h];
        sum = a.w != nullptr ? __builtin_fmaf(a.w[t * a.k + j], y, sum) : sum + y;
      }
      ((T*)a.out)[t * a.ldo + h] = (T)sum;
    }
  }
}

template <class T>
__global__ void __launch_bounds__(256) combine_grad_kernel(const RowArgs a) {
  __shared__ float part[4];
  for (int64_t t = blockIdx.x; t < a.tokens; t += gridDim.x) {
    const T* d = (const T*)a.x + t * a.ldx;
    for (int64_t j = 0; j < a.k; ++j) {
      const int64_t s = slot_of(a, t * a.k + j);
      const float w = a.w != nullptr ? a.w[t * a.k + j] : 1.0f;
      float dot = 0.0f;
      if (s >= 0) {
        for (int64_t h = threadIdx.x; h < a.H; h += 256) {
          const float g = (float)d[h];
          if (a.dw != nullptr) dot = __builtin_fmaf(g, (float)((const T*)a.y)[s * a.ldy + h], dot);
          if (a.out != nullptr) ((T*)a.out)[s * a.ldo + h] = (T)(w * g);
        }
      }
      if (a.dw == nullptr) continue;
#pragma unroll
      for (int o = 32; o > 0; o /= 2) dot += __shfl_xor(dot, o);
      __syncthreads();
      if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = dot;
      __syncthreads();
      if (threadIdx.x == 0) a.dw[t * a.k + j] = (part[0] + part[1]) + (part[2] + part[3]);
    }
  }
}

// The checks the three row operators share, up to the limits.
int check_rows(int64_t tokens, int64_t k, int64_t H, int64_t rows, int type) {
  if (!valid_type(type)) return DGEMM_ERR_INVALID_TYPE;
  if (tokens < 0 || k < 0 || H < 0 || rows < 0) return DGEMM_ERR_INVALID_DIM;
  return DGEMM_OK;
}

bool too_many(int64_t tokens, int64_t k, int64_t rows) {
  return tokens > kMaxCount || k > kMaxCount || tokens * k > kMaxCount || rows > kMaxCount;
}

}  // namespace
}  // namespace dg

extern "C" {

int64_t expert_sort_workspace(int64_t tokens, int64_t k, int64_t experts) {
  using namespace dg;
  if (tokens < 0 || k < 0 || experts < 0 || experts > kMaxExperts || too_many(tokens, k, 0)) return -1;
  return 0;
}

int expert_sort(int64_t tokens, int64_t k, int64_t experts, const void* ids, int id_bytes, int32_t* offsets,
                int32_t* slot, int32_t* pair, int32_t* token, void* workspace, int64_t workspace_bytes,
                void* stream) {
  using namespace dg;
  if (id_bytes != 4 && id_bytes != 8) return DGEMM_ERR_INVALID_TYPE;
  if (tokens < 0 || k < 0 || experts < 0) return DGEMM_ERR_INVALID_DIM;
  const int64_t need = expert_sort_workspace(tokens, k, experts);
  if (need < 0) return DGEMM_ERR_UNSUPPORTED;
  if (workspace_bytes < need) return DGEMM_ERR_INVALID_DIM;
  const int64_t n = tokens * k;
  if (offsets == nullptr || (n > 0 && (ids == nullptr || slot == nullptr || pair == nullptr)) ||
      (need > 0 && workspace == nullptr))
    return DGEMM_ERR_NULL_POINTER;
  if (!aligned_to(ids, id_bytes) || !aligned_to(offsets, 4) || !aligned_to(slot, 4) || !aligned_to(pair, 4) ||
      !aligned_to(token, 4) ||
      (need > 0 && !aligned_to(workspace, 4)))
    return DGEMM_ERR_MISALIGNED;
  SortArgs a{ids, offsets, slot, pair, token, n, (int)k, (int)experts};
  const void* fn = id_bytes == 8 ? (const void*)&sort_kernel<int64_t> : (const void*)&sort_kernel<int32_t>;
  return launch_kernel(fn, 1, 1024, &a, stream);
}

int expert_dispatch(int64_t tokens, int64_t k, int64_t H, int type, const void* X, int64_t ldx, const int32_t* slot,
                    void* Y, int64_t rows, int64_t ldy, void* stream) {
  using namespace dg;
  if (const int st = check_rows(tokens, k, H, rows, type)) return st;
  if (tokens == 0 || k == 0 || H == 0 || rows == 0) return DGEMM_OK;
  if (X == nullptr || slot == nullptr || Y == nullptr) return DGEMM_ERR_NULL_POINTER;
  if (ldx < H || ldy < H) return DGEMM_ERR_INVALID_LD;
  const int e = type_bytes(type);
  if (!aligned_to(X, e) || !aligned_to(Y, e) || !aligned_to(slot, 4)) return DGEMM_ERR_MISALIGNED;
  if (too_many(tokens, k, rows)) return DGEMM_ERR_UNSUPPORTED;
  RowArgs a{X, ldx, nullptr, 0, Y, ldy, slot, nullptr, nullptr, tokens, k, H, rows};
  return with_type(type, [&](auto t) {
    return launch_kernel((const void*)&dispatch_kernel<decltype(t)>, tokens, 256, &a, stream);
  });
}

int expert_combine(int64_t tokens, int64_t k, int64_t H, int type, const void* Y, int64_t rows, int64_t ldy,
                   const int32_t* slot, const float* weights, void* O, int64_t ldo, void* stream) {
  using namespace dg;
  if (const int st = check_rows(tokens, k, H, rows, type)) return st;
  if (tokens == 0 || H == 0) return DGEMM_OK;
  if (O == nullptr || (k > 0 && slot == nullptr) || (k > 0 && rows > 0 && Y == nullptr))
    return DGEMM_ERR_NULL_POINTER;
  if (ldo < H || ldy < H) return DGEMM_ERR_INVALID_LD;
  const int e = type_bytes(type);
  if (!aligned_to(Y, e) || !aligned_to(O, e) || !aligned_to(slot, 4) || !aligned_to(weights, 4))
    return DGEMM_ERR_MISALIGNED;
  if (too_many(tokens, k, rows)) return DGEMM_ERR_UNSUPPORTED;
  RowArgs a{nullptr, 0, Y, ldy, O, ldo, slot, weights, nullptr, tokens, k, H, rows};
  return with_type(type, [&](auto t) {
    return launch_kernel((const void*)&combine_kernel<decltype(t)>, tokens, 256, &a, stream);
  });
}

int expert_combine_grad(int64_t tokens, int64_t k, int64_t H, int type, const void* dO, int64_t ldo, const void* Y,
                        int64_t rows, int64_t ldy, const int32_t* slot, const float* weights, void* dY, int64_t lddy,
                        float* dW, void* stream) {
  using namespace dg;
  if (const int st = check_rows(tokens, k, H, rows, type)) return st;
  if (tokens == 0 || k == 0 || (dY == nullptr && dW == nullptr)) return DGEMM_OK;
  const bool some = H > 0 && rows > 0;
  if (slot == nullptr || (some && (dO == nullptr || (dW != nullptr && Y == nullptr)))) return DGEMM_ERR_NULL_POINTER;
  if (ldo < H || (dW != nullptr && ldy < H) || (dY != nullptr && lddy < H)) return DGEMM_ERR_INVALID_LD;
  const int e = type_bytes(type);
  if (!aligned_to(dO, e) || !aligned_to(Y, e) || !aligned_to(dY, e) || !aligned_to(slot, 4) ||
      !aligned_to(weights, 4) || !aligned_to(dW, 4))
    return DGEMM_ERR_MISALIGNED;
  if (too_many(tokens, k, rows)) return DGEMM_ERR_UNSUPPORTED;
  RowArgs a{dO, ldo, Y, ldy, dY, lddy, slot, weights, dW, tokens, k, H, rows};
  return with_type(type, [&](auto t) {
    return launch_kernel((const void*)&combine_grad_kernel<decltype(t)>, tokens, 256, &a, stream);
  });
}

}  // extern "C"
