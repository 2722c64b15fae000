// Tokens sorted by expert and back (mixture of experts): expert_sort,
// expert_dispatch, expert_combine and expert_combine_grad.
#include "elementwise.hpp"
#include "launch.hpp"

namespace dg {
namespace {

constexpr int kMaxExperts = 1024;

// ---- sort -------------------------------------------------------------------------
//
// A stable counting sort.  The pairs are cut into one contiguous chunk per
// workgroup and that into one per wave; a pair's place is
//   pairs of lower experts + pairs of its expert in earlier chunks (of
//   workgroups, then waves) + those before it in its own wave's chunk.
// Up to kChunk pairs one workgroup does it alone; beyond, a first launch
// leaves every chunk's counts in the workspace and each workgroup of the
// second sums the columns it needs (chunks x experts words from the L2, at
// most kBlocks x 1024; no third launch for the prefix sums, no atomics across
// workgroups, so the order never depends on timing).
//
// Latency bounds it, not bytes: 131072 pairs of 128 experts take 4.8 + 6.4 us
// (one workgroup alone, 1024 pairs a turn, took 700), 128 pairs 4.1.

constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;
constexpr int kChunk = 2048;     // pairs per workgroup, until there are kBlocks of them
constexpr int kBlocks = 256;     // one per CU

struct SortArgs {
  const void* ids;
  int32_t* offsets;
  int32_t* slot;
  int32_t* pair;
  int32_t* token;
  int32_t* counts;    // [blocks][experts], with more than one block
  int64_t n, chunk;   // pairs in all and per workgroup
  int k, experts, blocks;
};

// The chunk of a workgroup: a whole number of waves' 64-pair steps.
inline int64_t sort_chunk(int64_t n) {
  const int64_t c = (n + kBlocks - 1) / kBlocks;
  return c <= kChunk ? kChunk : (c + kSortThreads - 1) / kSortThreads * kSortThreads;
}

template <class Id>
__device__ __forceinline__ int expert_of(const SortArgs& a, int64_t i, int64_t end) {
  if (i >= end) return -1;
  const Id id = ((const Id*)a.ids)[i];
  return id >= 0 && id < (Id)a.experts ? (int)id : -1;
}

// First launch: the experts' counts in each chunk.
template <class Id>
__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(const SortArgs a) {
  __shared__ int32_t count[kMaxExperts];
  const int tid = threadIdx.x;
  if (tid < a.experts) count[tid] = 0;
  __syncthreads();
  const int64_t i0 = blockIdx.x * a.chunk, end = i0 + a.chunk < a.n ? i0 + a.chunk : a.n;
  for (int64_t i = i0 + tid; i < end; i += kSortThreads) {
    const int e = expert_of<Id>(a, i, end);
    if (e >= 0) atomicAdd(&count[e], 1);
  }
  __syncthreads();
  if (tid < a.experts) a.counts[(int64_t)blockIdx.x * a.experts + tid] = count[tid];
}

// The places of a chunk's pairs; workgroup 0 also stores the offsets.
template <class Id>
__global__ void __launch_bounds__(kSortThreads) sort_place_kernel(const SortArgs a) {
  __shared__ int32_t place[kSortWaves][kMaxExperts];   // counts of each wave's pairs, then their next places
  __shared__ int32_t part[2][kSortThreads];
  __shared__ int32_t wave_sum[kSortWaves];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int E = a.experts;
  const int64_t i0 = blockIdx.x * a.chunk, end = i0 + a.chunk < a.n ? i0 + a.chunk : a.n;
  const int64_t per = a.chunk / kSortWaves;            // pairs per wave
  const int64_t w0 = i0 + wave * per, w1 = w0 + per < end ? w0 + per : end;

  for (int e = lane; e < E; e += 64) place[wave][e] = 0;
  // (A wave counts into its own row only.)
  for (int64_t i = w0 + lane; i < w1; i += 64) {
    const int e = expert_of<Id>(a, i, w1);
    if (e >= 0) atomicAdd(&place[wave][e], 1);
  }
  // Columns of the counts: thread (g, e) sums chunks g, g + G, ... of expert e.
  const int width = E <= 64 ? 64 : (E <= 128 ? 128 : (E <= 256 ? 256 : (E <= 512 ? 512 : 1024)));
  const int groups = kSortThreads / width, g = tid / width, ge = tid % width;
  int32_t before = 0, all = 0;
  if (a.blocks > 1) {
    if (ge < E) {
#pragma unroll 4
      for (int b = g; b < a.blocks; b += groups) {
        const int32_t c = a.counts[(int64_t)b * E + ge];
        all += c;
        before += b < (int)blockIdx.x ? c : 0;
      }
    }
    part[0][tid] = before;
    part[1][tid] = all;
  }
  __syncthreads();
  before = all = 0;
  if (tid < E) {
    if (a.blocks > 1) {
      for (int q = 0; q < groups; ++q) {
        before += part[0][q * width + tid];
        all += part[1][q * width + tid];
      }
    } else {
#pragma unroll
      for (int w = 0; w < kSortWaves; ++w) all += place[w][tid];
    }
  }
  // Pairs of lower experts: an exclusive sum over the threads.
  int32_t sum = all;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int32_t o = __shfl_up(sum, d);
    if (lane >= d) sum += o;
  }
  if (lane == 63) wave_sum[wave] = sum;
  __syncthreads();
  int32_t kept = 0, first = sum - all;
#pragma unroll
  for (int w = 0; w < kSortWaves; ++w) {
    const int32_t s = wave_sum[w];
    first += w < wave ? s : 0;
    kept += s;
  }
  if (blockIdx.x == 0) {
    if (tid < E) a.offsets[tid] = first;
    if (tid == 0) a.offsets[E] = kept;
  }
  if (tid < E) {
    int32_t at = first + before;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      const int32_t c = place[w][tid];
      place[w][tid] = at;
      at += c;
    }
  }
  __syncthreads();
  // Each wave places its pairs in order, 64 at a time: a lane's rank is the
  // number of lower lanes with its expert, found bit by bit of the expert.
  int bits = 0;
  while ((1 << bits) < E) ++bits;
  for (int64_t j = w0; j < w1; j += 64) {
    const int64_t i = j + lane;
    const int e = expert_of<Id>(a, i, w1);
    uint64_t same = __ballot(e >= 0);
    for (int b = 0; b < bits; ++b) {
      const uint64_t m = __ballot((e >> b) & 1);
      same &= (e >> b) & 1 ? m : ~m;
    }
    const int rank = __popcll(same & ((1ull << lane) - 1ull));
    int32_t at = -1;
    if (e >= 0) at = place[wave][e] + rank;
    if (i < w1) a.slot[i] = at;
    if (e >= 0) {
      a.pair[at] = (int32_t)i;
      if (a.token != nullptr) a.token[at] = (int32_t)i / a.k;
      if (rank == 0) place[wave][e] += __popcll(same);
    }
  }
  // No pairs behind the last place (each workgroup its share).
  for (int64_t n = (kept > i0 ? kept : i0) + tid; n < end; n += kSortThreads) {
    a.pair[n] = -1;
    if (a.token != nullptr) a.token[n] = -1;
  }
}

// ---- rows -------------------------------------------------------------------------
//
// All three move rows and little else: HBM bounds them.  WPT waves of a
// workgroup of four take a token: all four where a row is longer than the
// 1 KiB one wave covers, else one each.  (8191 tokens x 8 rows of 8 KiB,
// combined: 123 us with four waves on a token, 176 with one, whose 8 x 1 KiB
// pieces lie further apart; past the caches, see kStreamBytes, 105.)  A lane takes 16 bytes of the row at a time, of kBatch pairs at once,
// so that kBatch loads per lane are in flight.  A token's slots are the same
// for the whole wave and sit in scalar registers: a dropped pair costs a
// branch and no traffic.  Now: dispatch of 16384 x 8 rows (1.2 GB) 223 us, 5.4
// TB/s; combine of 8191 x 8 (604 MB) 105 us, 5.7 TB/s; gradients of 16384 x 2
// (671 MB) 120 us, 5.6 TB/s; a large copy reaches 4.9.

constexpr int kBatch = 8;       // combine
constexpr int kGradBatch = 4;   // combine_grad, which holds more per pair (8 parked scalars in vector registers)

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

// The token of this wave, -1 behind the last, and its part of the row.
template <int WPT>
__device__ __forceinline__ int64_t token_of(const RowArgs& a, int* part) {
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  *part = wave % WPT;
  const int64_t t = (int64_t)blockIdx.x * (4 / WPT) + wave / WPT;
  return t < a.tokens ? t : -1;
}

// Slots of pairs j0 .. of token t, all loaded at once; -1 past the last.
template <int N>
__device__ __forceinline__ void slots_of(const RowArgs& a, int64_t t, int64_t j0, int32_t (&s)[N]) {
#pragma unroll
  for (int j = 0; j < N; ++j) s[j] = a.slot[t * a.k + (j0 + j < a.k ? j0 + j : a.k - 1)];
#pragma unroll
  for (int j = 0; j < N; ++j) s[j] = j0 + j < a.k && (uint32_t)s[j] < (uint32_t)a.rows ? s[j] : -1;
}

template <class T, bool STREAM, int WPT>
__global__ void __launch_bounds__(256) dispatch_kernel(const RowArgs a) {
  using P = Pack<T>;
  int part;
  const int64_t t = token_of<WPT>(a, &part);
  if (t < 0) return;
  const T* x = (const T*)a.x + t * a.ldx;
  for (int64_t j0 = 0; j0 < a.k; j0 += kBatch) {
    int32_t s[kBatch];
    slots_of(a, t, j0, s);
    for (int64_t h = (part * 64 + lane_id()) * P::N; h < a.H; h += WPT * 64 * P::N) {
      const u32x4 v = load_pack<T, false>(x, h, a.H);
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (s[j] >= 0) store_pack<T, STREAM>((T*)a.out + s[j] * a.ldo, h, a.H, v);
    }
  }
}

template <class T, bool STREAM, int WPT>
__global__ void __launch_bounds__(256) combine_kernel(const RowArgs a) {
  using P = Pack<T>;
  int part;
  const int64_t t = token_of<WPT>(a, &part);
  if (t < 0) return;
  // The first batch's slots and weights, and mostly the only one's, are kept.
  int32_t s[kBatch];
  float w[kBatch];
  auto batch = [&](int64_t j0) {
    slots_of(a, t, j0, s);
#pragma unroll
    for (int j = 0; j < kBatch; ++j) w[j] = s[j] < 0 ? 0.0f : (a.w != nullptr ? a.w[t * a.k + j0 + j] : 1.0f);
  };
  if (a.k > 0) batch(0);
  for (int64_t h = (part * 64 + lane_id()) * P::N; h < a.H; h += WPT * 64 * P::N) {
    float sum[P::N] = {};
    for (int64_t j0 = 0; j0 < a.k; j0 += kBatch) {
      if (a.k > kBatch) batch(j0);
      u32x4 y[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        // (A pair past the last, or dropped, adds 0 * 0.)
        y[j] = u32x4{0, 0, 0, 0};
        if (s[j] >= 0) y[j] = load_pack<T, STREAM>((const T*)a.y + s[j] * a.ldy, h, a.H);
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        float f[P::N];
        P::unpack(y[j], f);
#pragma unroll
        for (int i = 0; i < P::N; ++i) sum[i] = __builtin_fmaf(w[j], f[i], sum[i]);
      }
    }
    store_pack<T, STREAM>((T*)a.out + t * a.ldo, h, a.H, P::pack(sum));
  }
}

template <class T, bool STREAM, int WPT>
__global__ void __launch_bounds__(256) combine_grad_kernel(const RowArgs a) {
  using P = Pack<T>;
  __shared__ float sums[4][kGradBatch];
  int part;
  const int64_t t = token_of<WPT>(a, &part);
  if (WPT == 1 && t < 0) return;   // (WPT 4: every workgroup has a token)
  const T* x = (const T*)a.x + t * a.ldx;
  for (int64_t j0 = 0; j0 < a.k; j0 += kGradBatch) {
    int32_t s[kGradBatch];
    float w[kGradBatch], dot[kGradBatch];
    slots_of(a, t, j0, s);
#pragma unroll
    for (int j = 0; j < kGradBatch; ++j) {
      w[j] = s[j] >= 0 && a.w != nullptr ? a.w[t * a.k + j0 + j] : 1.0f;
      dot[j] = 0.0f;
    }
    for (int64_t h = (part * 64 + lane_id()) * P::N; h < a.H; h += WPT * 64 * P::N) {
      float d[P::N];
      P::unpack(load_pack<T, false>(x, h, a.H), d);
      u32x4 y[kGradBatch];
#pragma unroll
      for (int j = 0; j < kGradBatch; ++j)
        if (s[j] >= 0 && a.dw != nullptr) y[j] = load_pack<T, STREAM>((const T*)a.y + s[j] * a.ldy, h, a.H);
#pragma unroll
      for (int j = 0; j < kGradBatch; ++j) {
        if (s[j] < 0) continue;
        if (a.out != nullptr) {
          float g[P::N];
#pragma unroll
          for (int i = 0; i < P::N; ++i) g[i] = w[j] * d[i];
          store_pack<T, STREAM>((T*)a.out + s[j] * a.ldo, h, a.H, P::pack(g));
        }
        if (a.dw != nullptr) {
          float f[P::N];
          P::unpack(y[j], f);
#pragma unroll
          for (int i = 0; i < P::N; ++i) dot[j] = __builtin_fmaf(d[i], f[i], dot[j]);
        }
      }
    }
    if (a.dw == nullptr) continue;
    float mine = 0.0f;
#pragma unroll
    for (int j = 0; j < kGradBatch; ++j) {
#pragma unroll
      for (int o = 32; o > 0; o /= 2) dot[j] += __shfl_xor(dot[j], o);
      mine = lane_id() == j ? dot[j] : mine;
    }
    if constexpr (WPT > 1) {
      __syncthreads();
      if (lane_id() < kGradBatch) sums[part][lane_id()] = mine;
      __syncthreads();
      if (lane_id() < kGradBatch)
        mine = (sums[0][lane_id()] + sums[1][lane_id()]) + (sums[2][lane_id()] + sums[3][lane_id()]);
    }
    if (part == 0 && lane_id() < kGradBatch && j0 + lane_id() < a.k) a.dw[t * a.k + j0 + lane_id()] = mine;
  }
}

// A row operator's launch: the kernel for the type, the rows' length and how
// many bytes they are.
enum RowOp { kDispatch, kCombine, kCombineGrad };

template <class T, bool STREAM, int WPT>
const void* row_kernel(RowOp op) {
  if (op == kDispatch) return (const void*)&dispatch_kernel<T, STREAM, WPT>;
  if (op == kCombine) return (const void*)&combine_kernel<T, STREAM, WPT>;
  return (const void*)&combine_grad_kernel<T, STREAM, WPT>;
}

int launch_rows(RowOp op, int type, RowArgs a, void* stream) {
  const int64_t e = type_bytes(type);
  const bool stream_rows = a.tokens * a.k * a.H >= kStreamBytes / e;
  const bool one = (a.H * e + 15) / 16 <= 64;   // one wave's width
  const void* fn = with_type(type, [&](auto t) {
    using T = decltype(t);
    if (stream_rows) return one ? row_kernel<T, true, 1>(op) : row_kernel<T, true, 4>(op);
    return one ? row_kernel<T, false, 1>(op) : row_kernel<T, false, 4>(op);
  });
  const int64_t per = one ? 4 : 1, step = kMaxRowBlocks * per;
  for (int64_t at = 0; at < a.tokens; at += step) {
    // Tokens at .. of the matrices by token and of the slots and weights; the
    // sorted rows stay whole.
    RowArgs part = a;
    part.tokens = a.tokens - at < step ? a.tokens - at : step;
    if (a.x != nullptr) part.x = (const char*)a.x + at * a.ldx * e;
    if (op == kCombine) part.out = (char*)a.out + at * a.ldo * e;
    if (a.slot != nullptr) part.slot = a.slot + at * a.k;
    if (a.w != nullptr) part.w = a.w + at * a.k;
    if (a.dw != nullptr) part.dw = a.dw + at * a.k;
    if (const int st = launch_kernel(fn, (part.tokens + per - 1) / per, 256, &part, stream)) return st;
  }
  return DGEMM_OK;
}

// The checks the three row operators share, up to the limits.
int check_rows(int64_t tokens, int64_t k, int64_t H, int64_t rows, int type) {
  if (!valid_type(type)) return DGEMM_ERR_INVALID_TYPE;
  if (tokens < 0 || k < 0 || H < 0 || rows < 0) return DGEMM_ERR_INVALID_DIM;
  return DGEMM_OK;
}

bool too_many(int64_t tokens, int64_t k, int64_t rows, int64_t H = 0) {
  return tokens > kMaxCount || k > kMaxCount || tokens * k > kMaxCount || rows > kMaxCount || H > kMaxCount;
}

}  // namespace
}  // namespace dg

extern "C" {

int64_t expert_sort_workspace(int64_t tokens, int64_t k, int64_t experts) {
  using namespace dg;
  if (tokens < 0 || k < 0 || experts < 0 || experts > kMaxExperts || too_many(tokens, k, 0)) return -1;
  const int64_t n = tokens * k, blocks = (n + sort_chunk(n) - 1) / sort_chunk(n);
  return blocks > 1 ? 4 * blocks * experts : 0;
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
  SortArgs a{ids, offsets, slot, pair, token, (int32_t*)workspace, n, sort_chunk(n), (int)k, (int)experts, 1};
  if (n > a.chunk) a.blocks = (int)((n + a.chunk - 1) / a.chunk);
  const bool wide = id_bytes == 8;
  if (a.blocks > 1 && experts > 0) {
    const void* fn = wide ? (const void*)&sort_count_kernel<int64_t> : (const void*)&sort_count_kernel<int32_t>;
    if (const int st = launch_kernel(fn, a.blocks, kSortThreads, &a, stream)) return st;
  }
  const void* fn = wide ? (const void*)&sort_place_kernel<int64_t> : (const void*)&sort_place_kernel<int32_t>;
  return launch_kernel(fn, a.blocks, kSortThreads, &a, stream);
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
  if (too_many(tokens, k, rows, H)) return DGEMM_ERR_UNSUPPORTED;
  RowArgs a{X, ldx, nullptr, 0, Y, ldy, slot, nullptr, nullptr, tokens, k, H, rows};
  return launch_rows(kDispatch, type, a, stream);
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
  if (too_many(tokens, k, rows, H)) return DGEMM_ERR_UNSUPPORTED;
  RowArgs a{nullptr, 0, Y, ldy, O, ldo, slot, weights, nullptr, tokens, k, H, rows};
  return launch_rows(kCombine, type, a, stream);
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
  if (too_many(tokens, k, rows, H)) return DGEMM_ERR_UNSUPPORTED;
  // No sorted rows: every pair is dropped and dW is zeros.  dO may be NULL then,
  // so the kernel is given rows of no elements (it loads dO whatever the slots are).
  RowArgs a{dO, ldo, Y, ldy, dY, lddy, slot, weights, dW, tokens, k, some ? H : 0, rows};
  return launch_rows(kCombineGrad, type, a, stream);
}

}  // extern "C"
