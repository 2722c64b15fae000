// expert_route and expert_route_grad: a router's logits to each token's experts
// and weights, and the weights' gradient back to the logits.
//
//   s = softmax(l) or 1 / (1 + exp(-l)),  v = s + bias
//   groups of E / G experts: their value the sum of their best one or two v;
//   the best top_groups of them stay, of their experts the best k by v are
//   chosen (ties: the lowest index), with w = f s or f s / sum of the chosen s
//
// Which experts are chosen is decided by values in 64 bits: values next to each
// other in 32 bits may stand the other way round.  Sixteen lanes take a token
// (route_row) and choose in 32 bits, with a margin; tokens where two values that
// matter are within it, a few in a thousand, are then done over in 64 bits by the
// whole wave (route_wave), as is every token of a router that does not fit
// sixteen lanes.
//
// Instructions bound it, a pick most of all: 16384 tokens, 8 of 256 experts in 8 groups
// (17 MB of logits, 19 in all) 14.3 us, their gradient (26 MB) 5.4; 8191 tokens, 6 of 61
// experts by softmax in bf16 5.8 and 3.6; 16 tokens 6.7 us, one token's steps.  Without
// groups 8 of 256 take 10 us, 12 of them 11, 15 19, 16 (route_wave) 46.
#include "elementwise.hpp"
#include "launch.hpp"

namespace dg {
namespace {

constexpr int kMaxExperts = 1024;
constexpr int kMaxChoices = 64;   // a lane each

struct RouteArgs {
  const void* logits;
  int64_t ldl;
  const float* bias;
  const int32_t* ids_in;     // gradient
  const float* dw;
  void* dl;
  int64_t lddl;
  int32_t* ids;
  float* weights;
  int64_t tokens;
  int experts, k, sigmoid, groups, top_groups, group_best, renormalize;
  float factor;
  int group_size, lanes_per_group, per_lane;   // sixteen lanes a token: lanes of a group, experts of a lane
};

constexpr float kInf = __builtin_inff();
constexpr float kMax = 3.402823466e38f;

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int d = 32; d > 0; d /= 2) v = __builtin_fmaxf(v, __shfl_xor(v, d));
  return v;
}
template <class F>
__device__ __forceinline__ F wave_sum(F v) {
#pragma unroll
  for (int d = 32; d > 0; d /= 2) v += __shfl_xor(v, d);
  return v;
}

// What the lanes of a wave have written to its part of the LDS is there.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

template <int N>
__device__ __forceinline__ uint32_t row_ror(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x120 + N, 0xf, 0xf, true);
}
template <int N>
__device__ __forceinline__ float row_ror(float v) {
  return __builtin_bit_cast(float, row_ror<N>(__builtin_bit_cast(uint32_t, v)));
}
// op over the sixteen lanes of a row, in every lane.
template <class X, class Op>
__device__ __forceinline__ X row_all(X v, Op op) {
  v = op(v, row_ror<8>(v));
  v = op(v, row_ror<4>(v));
  v = op(v, row_ror<2>(v));
  return op(v, row_ror<1>(v));
}
__device__ __forceinline__ float row_max(float v) {
  return row_all(v, [](float x, float y) { return __builtin_fmaxf(x, y); });
}
__device__ __forceinline__ float row_sum(float v) {
  return row_all(v, [](float x, float y) { return x + y; });
}
// The value of the lane behind this one (lane 15: its own row's lane 0's).
__device__ __forceinline__ float next_lane(float v) { return row_ror<15>(v); }
// The row's sixteen bits of a ballot.
__device__ __forceinline__ uint32_t row_bits(bool c) {
  return (uint32_t)(__ballot(c) >> (lane_id() & 48)) & 0xffffu;
}

// The largest over the wave, in scalar registers.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = row_all(v, [](uint32_t x, uint32_t y) { return x > y ? x : y; });
  uint32_t m = 0u;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const uint32_t o = (uint32_t)__builtin_amdgcn_readlane((int)v, 16 * r);
    m = o > m ? o : m;
  }
  return m;
}

// The index of the largest value over the wave, of equal ones the lowest; -1 if all
// are -infinity.  (Three maxima of 32 bits, of the high and the low half of the
// bits in the order of the values and of the index, stay in registers; shuffles
// of the values took three times as long.)
__device__ __forceinline__ int best_of_wave(double v, int e) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v + 0.0);   // (-0 is 0)
  const uint64_t u = b ^ ((uint64_t)((int64_t)b >> 63) | 0x8000000000000000ull);
  const uint32_t hi = (uint32_t)(u >> 32), lo = (uint32_t)u;
  const uint32_t top = wave_max(hi);
  const uint32_t low = wave_max(hi == top ? lo : 0u);
  const uint32_t first = ~wave_max(hi == top && lo == low ? ~(uint32_t)e : 0u);
  return top < 0x00100000u ? -1 : (int)first;
}

// A chosen expert's score relative to that of the largest chosen logit `top`, so
// that shares stay where the scores themselves underflow.
__device__ __forceinline__ float share_score(bool on, float l, float top, int sigmoid) {
  if (!on || l == -kInf) return 0.0f;
  if (!sigmoid) return expf(l - top);
  const float c = __builtin_fminf(top, 0.0f);
  return 1.0f / (expf(c) + expf(c - l));
}

// The shares of the chosen experts, a lane each (`on`): s over the sum of s.
__device__ __forceinline__ float share_of(bool on, float l, int sigmoid) {
  const float top = wave_max(on ? l : -kInf);
  const float t = share_score(on, l, top, sigmoid);
  const float total = wave_sum(t);
  return total == 0.0f ? 0.0f : t / total;
}

__device__ __forceinline__ float sigmoid_of(float l) { return 1.0f / (1.0f + expf(-l)); }

// Token t by a whole wave, in 64 bits: lane l has experts l, l + 64, ...
template <int V>
struct WaveLds {
  double value[V * 64];
  uint8_t keep[V * 64];   // by group
};

template <class T, int V>
__device__ __forceinline__ void route_wave(const RouteArgs& a, int64_t t, WaveLds<V>& lds) {
  const int lane = lane_id();
  const T* row = (const T*)a.logits + t * a.ldl;
  const int E = a.experts;

  float l[V];
  float top = -kInf;
  bool nan = false;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = i * 64 + lane;
    l[i] = e < E ? (float)row[e] : -kInf;
    nan |= l[i] != l[i];
    top = __builtin_fmaxf(top, l[i]);
  }
  top = wave_max(top);
  // A NaN (or, for a softmax, +infinity) leaves no weights.
  const bool bad = __ballot(nan) != 0 || (!a.sigmoid && top == kInf);
  const double dtop = __builtin_fminf(top, kMax);

  double s[V], sum = 0.0;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const double x = l[i] < kMax ? l[i] : kMax;   // (NaN: any value, not chosen)
    s[i] = 0.0;
    if (l[i] > -kInf) s[i] = a.sigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x - dtop);
    sum += s[i];
  }
  if (!a.sigmoid) sum = wave_sum(sum);
  // Values: scores where they are added to something, else the logits.
  const bool sums = a.bias != nullptr || (a.top_groups < a.groups && a.group_best == 2);
  double v[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = i * 64 + lane;
    if (!a.sigmoid) s[i] /= sum;
    v[i] = -__builtin_inf();
    if (l[i] > -kInf) {
      const double b = sums ? s[i] + (a.bias != nullptr ? (double)a.bias[e] : 0.0) : (double)l[i];
      if (b > -__builtin_inf()) v[i] = b;   // (a bias of NaN or -infinity: never)
    }
  }

  if (a.top_groups < a.groups) {
    const int size = E / a.groups;
#pragma unroll
    for (int i = 0; i < V; ++i) lds.value[i * 64 + lane] = v[i];
    // A lane's groups: their value, or -infinity.
    wave_sync();
    double gv[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int g = i * 64 + lane;
      double one = -__builtin_inf(), two = -__builtin_inf();
      if (g < a.groups)
#pragma unroll 4
        for (int e = 0; e < size; ++e) {
          const double x = lds.value[g * size + e];
          if (x > one) {
            two = one;
            one = x;
          } else if (x > two) {
            two = x;
          }
        }
      gv[i] = a.group_best == 2 && two > -__builtin_inf() ? one + two : one;
      lds.keep[g] = 0;
    }
    for (int j = 0; j < a.top_groups; ++j) {
      double best = -__builtin_inf();
      int at = lane;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (gv[i] > best) {
          best = gv[i];
          at = i * 64 + lane;
        }
      at = best_of_wave(best, at);
      if (at < 0) break;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (at == i * 64 + lane) {
          gv[i] = -__builtin_inf();
          lds.keep[at] = 1;
        }
    }
    wave_sync();
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = i * 64 + lane;
      if (e < E && lds.keep[e / size] == 0) v[i] = -__builtin_inf();
      // (The groups' sums are done.)
      if (a.bias == nullptr && v[i] > -__builtin_inf()) v[i] = (double)l[i];
    }
  }

  int id = -1;          // choice `lane`
  float chosen = 0.0f;  // its logit
  for (int j = 0; j < a.k; ++j) {
    double best = -__builtin_inf();
    int at = lane;
    float x = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (v[i] > best) {
        best = v[i];
        at = i * 64 + lane;
        x = l[i];
      }
    at = best_of_wave(best, at);
    if (at < 0) break;
    x = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), at & 63));
    if (lane == j) {
      id = at;
      chosen = x;
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (at == i * 64 + lane) v[i] = -__builtin_inf();
  }

  float w;
  if (a.renormalize) {
    w = share_of(id >= 0, chosen, a.sigmoid);
  } else {
    // (sum: of exp(l - top) in 64 bits, rounded once)
    w = a.sigmoid ? sigmoid_of(chosen) : expf(chosen - top) / (float)sum;
    if (id < 0) w = 0.0f;
  }
  if (lane < a.k) {
    a.ids[t * a.k + lane] = id;
    a.weights[t * a.k + lane] = bad ? __builtin_nanf("") : a.factor * w;
  }
}

// ---- sixteen lanes a token ----------------------------------------------------------

constexpr int kRowExperts = 16;   // experts a lane
constexpr int kRowChoices = 15;   // choices a lane each, and one or more that only bound them

// A float's bits in the order of its values, and back.
__device__ __forceinline__ uint32_t ordered(float f) {
  const uint32_t b = __builtin_bit_cast(uint32_t, f);
  return b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t u) {
  return __builtin_bit_cast(float, u ^ ((u & 0x80000000u) ? 0x80000000u : 0xffffffffu));
}

// Two values, one >= two, of the best of this lane and another.
__device__ __forceinline__ void merge_two(float& one, float& two, float o1, float o2) {
  two = __builtin_fmaxf(__builtin_fminf(one, o1), __builtin_fmaxf(two, o2));
  one = __builtin_fmaxf(one, o1);
}

// Token t by the sixteen lanes of this row; true where its choice is certain (and
// stored).  Lane c holds up to V neighbouring experts; the lanes of a group follow
// each other.  A value's key is its ordered bits with the low eight replaced by
// its lane and slot, lower ones larger, so a pick is a maximum of keys and says
// whose it is.
//
// Values are scores in FP32 plus bias; where neither bias nor a sum of two
// enters, the logits themselves.  Where two picks in a row are no further apart
// than what the values may be off by, their order is open: which experts are
// chosen is certain if a gap follows the last choice or one of the picks behind
// it, and the order of those up to there is settled in 64 bits.
//
// The logits come in whole lines, lane after lane, and through LDS to their lanes,
// four words between those of neighbouring lanes that take V each.
template <int V>
struct alignas(16) RowLds {
  static constexpr int N = 20 * V > 16 * V + 64 ? 20 * V : 16 * V + 64;
  static_assert(N % 4 == 0, "every token's row begins at sixteen bytes");
  float l[4][N], bias[N];
  __device__ static int at(int e) { return e + e / V * 4; }
};

template <class T, int V>
__device__ __forceinline__ bool route_row(const RouteArgs& a, int64_t t0, RowLds<V>& lds) {
  static_assert(V == 4 || V == 8 || V == 16, "sorted fours, a slot in four bits");
  constexpr uint32_t LOW = 255u;
  using Lds = RowLds<V>;
  const int c = lane_id() & 15, r = lane_id() >> 4;
  const int64_t t = t0 + r;
  const bool live = t < a.tokens;
  const int E = a.experts;
  {
    // (Past the last token or expert: the last one again.)
    constexpr int N = V / 4;
    T x[4][N];
    float b[N];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const T* row = (const T*)a.logits + (t0 + q < a.tokens ? t0 + q : a.tokens - 1) * a.ldl;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int e = i * 64 + lane_id() < E ? i * 64 + lane_id() : E - 1;
        x[q][i] = row[e];
        if (q == 0) b[i] = a.bias != nullptr ? a.bias[e] : 0.0f;
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
#pragma unroll
      for (int q = 0; q < 4; ++q) lds.l[q][Lds::at(i * 64 + lane_id())] = (float)x[q][i];
      lds.bias[Lds::at(i * 64 + lane_id())] = b[i];
    }
    wave_sync();
  }
  // This lane's experts: e0 .. e0 + n - 1, in group g.
  const int size = a.group_size, lpg = a.lanes_per_group, per = a.per_lane;
  const int g = c / lpg, part = c - g * lpg;
  const int e0 = g * size + part * per;
  int n = size - part * per;
  n = g >= a.groups || n < 0 ? 0 : (n < per ? n : per);

  float l[V], bias[V];
  const int at = n > 0 ? e0 : 0;
  if (size == lpg * V) {   // V experts for each lane that has any
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const f32x4 x = *(const f32x4*)&lds.l[r][Lds::at(at) + i], y = *(const f32x4*)&lds.bias[Lds::at(at) + i];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        l[i + e] = n > 0 ? x[e] : -kInf;
        bias[i + e] = y[e];
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = Lds::at(at + (i < n ? i : 0));
      l[i] = i < n ? lds.l[r][e] : -kInf;
      bias[i] = lds.bias[e];
    }
  }
  bool nan = false;
#pragma unroll
  for (int i = 0; i < V; ++i) nan |= l[i] != l[i];
  float top = -kInf;   // (of a softmax)
  if (!a.sigmoid) {
#pragma unroll
    for (int i = 0; i < V; ++i) top = __builtin_fmaxf(top, l[i]);
    top = row_max(top);
  }
  const bool bad = row_bits(nan) != 0 || top == kInf;

  // Values: -infinity where an expert is none to choose (NaN never is).
  const bool limited = a.top_groups < a.groups;
  const bool plain = a.bias == nullptr && !(limited && a.group_best == 2);   // by the logits
  float v[V], sum = 0.0f;
  if (plain) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = l[i] > -kInf ? l[i] + 0.0f : -kInf;   // (-0 is 0)
  } else if (a.sigmoid) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      v[i] = __builtin_amdgcn_rcpf(1.0f + __expf(-l[i])) + bias[i];
      v[i] = l[i] > -kInf && v[i] > -kInf ? v[i] : -kInf;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) sum += l[i] > -kInf ? __expf(l[i] - top) : 0.0f;
    sum = row_sum(sum);
    const float inv = 1.0f / sum;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      v[i] = __expf(l[i] - top) * inv + bias[i];
      v[i] = l[i] > -kInf && v[i] > -kInf ? v[i] : -kInf;
    }
  }
  // What two values may be off by: scores 2^-21 on either side of a difference, a
  // softmax's with its sum 2^-19, without a bias relative to the value; cut keys
  // 2^-15 of a value, or of the smallest normal numbers.
  const float margin = a.bias == nullptr ? 0x1p-140f : (a.sigmoid ? 0x1p-20f : 0x1p-18f);
  constexpr float kRel = 0x1.8p-15f;
  auto far = [&](float x, float y) { return x - y > margin + kRel * __builtin_fabsf(x) || y == -kInf; };

  bool sure = plain || !bad;
  if (limited) {
    // The two best of the group: of this lane, then of the lanes up to lpg - 1 away on
    // either side.  (Medians of three: no NaN is left, which fmax would look for.)
    float one = -kInf, two = -kInf;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      two = __builtin_amdgcn_fmed3f(one, two, v[i]);
      one = __builtin_amdgcn_fmed3f(one, v[i], kInf);
    }
    float b1 = one, b2 = two;
    for (int d = 1; d < lpg; ++d) {
      const int up = (lane_id() & 48) + ((c + d) & 15), down = (lane_id() & 48) + ((c - d) & 15);
      const float u1 = __shfl(one, up), u2 = __shfl(two, up), d1 = __shfl(one, down), d2 = __shfl(two, down);
      if (part + d < lpg) merge_two(b1, b2, u1, u2);
      if (part - d >= 0) merge_two(b1, b2, d1, d2);
    }
    // (A sum below FP32's range is its lowest value: -infinity is a group with no expert.)
    const float mine = g >= a.groups ? -kInf : (a.group_best == 2 && b2 > -kInf ? __builtin_fmaxf(b1 + b2, -kMax) : b1);
    // Groups of larger value (of equal ones, lower), each seen by its first lane.
    // (The others show NaN, which is neither.)
    int larger = 0;
    const float shown = part == 0 && g < a.groups ? mine : __builtin_nanf("");
    // (d lanes away; multiples of lpg are enough where lanes of one part are that far apart all round.)
    const bool even = lpg * a.groups == 16;
    auto see = [&](float o, uint32_t og) { larger += o > mine || (o == mine && (int)og < g); };
#define DG_SEE(d) \
  if (!even) see(row_ror<d>(shown), row_ror<d>((uint32_t)g)); \
  else if (d % lpg == 0) see(row_ror<d>(mine), row_ror<d>((uint32_t)g))
    DG_SEE(1); DG_SEE(2); DG_SEE(3); DG_SEE(4); DG_SEE(5); DG_SEE(6); DG_SEE(7); DG_SEE(8);
    DG_SEE(9); DG_SEE(10); DG_SEE(11); DG_SEE(12); DG_SEE(13); DG_SEE(14); DG_SEE(15);
#undef DG_SEE
    bool stays = g < a.groups && larger < a.top_groups;
    const float kept = -row_max(stays ? -mine : -kInf), lost = row_max(stays ? -kInf : mine);
    // (Logits are exact.  Else two values of a group each, four roundings of the largest of
    // them; without a bias 2^-16.8 of a value whose exponential has an argument near -88,
    // and of smaller ones nothing is left.)
    const float most = __builtin_fmaxf(b1 > -kInf ? __builtin_fabsf(b1) : 0.0f, b2 > -kInf ? __builtin_fabsf(b2) : 0.0f);
    const float room = a.bias != nullptr ? 2 * margin + 0x1p-21f * row_max(most)
                                         : 0x1p-16f * (kept + lost) + 0x1p-120f;
    const bool near = !(plain || kept == -kInf || lost == -kInf || kept - lost > room);
    if (__ballot(near) != 0) {
      if (!a.sigmoid) {
        sure = sure && !near;
      } else {
        // Groups by sigmoids in 64 bits: each lane's values that may be among its
        // group's best, then the lanes of a group, then the groups.
        const float least = (a.group_best == 2 ? b2 : b1) - room;
        uint32_t open = 0u;
#pragma unroll
        for (int i = 0; i < V; ++i) open |= v[i] > -kInf && !(v[i] < least) ? 1u << i : 0u;
        double d1 = -__builtin_inf(), d2 = -__builtin_inf();
        while (__ballot(open != 0u) != 0) {
          if (open != 0u) {
            const int e = Lds::at(at + __builtin_ctz(open));
            open &= open - 1u;
            const double d = 1.0 / (1.0 + exp(-(double)lds.l[r][e])) + (double)lds.bias[e];
            d2 = fmax(d2, fmin(d1, d));
            d1 = fmax(d1, d);
          }
        }
        double g1 = d1, g2 = d2;
        for (int d = 1 - lpg; d < lpg; ++d) {
          const int from = (lane_id() & 48) + ((c + d) & 15);
          const double o1 = __shfl(d1, from), o2 = __shfl(d2, from);
          if (d != 0 && part + d >= 0 && part + d < lpg) {
            g2 = fmax(fmin(g1, o1), fmax(g2, o2));
            g1 = fmax(g1, o1);
          }
        }
        const double exact = g >= a.groups ? -__builtin_inf() : (a.group_best == 2 && g2 > -__builtin_inf() ? g1 + g2 : g1);
        int above = 0;
        for (int d = 1; d < 16; ++d) {
          const int from = (lane_id() & 48) + ((c + d) & 15);
          const double o = __shfl(exact, from);
          const int og = __shfl(part == 0 && g < a.groups ? g : kMaxExperts, from);
          above += og < kMaxExperts && (o > exact || (o == exact && og < g));
        }
        if (near) stays = g < a.groups && above < a.top_groups;
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = stays ? v[i] : -kInf;
  }

  // Keys, in falling fours; those of -infinity are below kNone.
  constexpr uint32_t kNone = 0x00800000u;
  auto max_key = [](uint32_t x, uint32_t y) { return x > y ? x : y; };
  uint32_t key[V];
#pragma unroll
  for (int i = 0; i < V; ++i) key[i] = (ordered(v[i]) & ~LOW) | (uint32_t)((15 - c) << 4 | (15 - i));
#pragma unroll
  for (int i = 0; i < V; i += 4) {
    auto order = [&](int x, int y) {
      const uint32_t hi = max_key(key[i + x], key[i + y]), lo = key[i + x] < key[i + y] ? key[i + x] : key[i + y];
      key[i + x] = hi;
      key[i + y] = lo;
    };
    order(0, 1); order(2, 3); order(0, 2); order(1, 3); order(1, 2);
  }
  // Picks: lane j keeps pick j.
  uint32_t pick = 0u;
  auto take = [&](int j) {
    uint32_t m = key[0];
#pragma unroll
    for (int i = 4; i < V; i += 4) m = max_key(m, key[i]);
    const uint32_t best = row_all(m, max_key);
    if (c == j) pick = best;
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const bool gone = key[i] == best;
      key[i] = gone ? key[i + 1] : key[i];
      key[i + 1] = gone ? key[i + 2] : key[i + 1];
      key[i + 2] = gone ? key[i + 3] : key[i + 2];
      key[i + 3] = gone ? 0u : key[i + 3];
    }
  };
  auto value = [&]() { return pick >= kNone ? unordered(pick & ~LOW) : -kInf; };
  // One more than the choices, and on while no gap follows the last choice.  (All
  // lanes take part in what reads the next one's value.)
  int taken = 0;
  while (taken < 16) {
    take(taken);
    if (taken++ < a.k) continue;
    const bool apart = far(value(), next_lane(value()));
    if (__ballot(live && (row_bits(apart) & (1u << (taken - 1)) - 1u) >> (a.k - 1) == 0) == 0) break;
  }
  const int from = 15 - (int)(pick >> 4 & 15u), slot = 15 - (int)(pick & 15u);
  const int first = __shfl(e0, (lane_id() & 48) + from);
  int id = pick >= kNone ? first + slot : -1;
  float x = id >= 0 ? lds.l[r][Lds::at(id)] : -kInf;
  // (Exponentials of arguments past -32 are off by more than the margin has room for.)
  const bool wide = !plain && id >= 0 && !((a.sigmoid ? x : x - top) > -32.0f);
  const bool gap = far(value(), next_lane(value())) && !wide;
  const uint32_t gaps = row_bits(gap);
  // The picks before the first gap from the last choice on are as many largest; their
  // order is settled in 64 bits where two are near: by the logits if nothing else
  // differs, else by sigmoids plus biases.  (The last pick's gap is to none.)
  const uint32_t ends = (gaps & (1u << (taken - 1)) - 1u) >> (a.k - 1);
  sure = sure && ends != 0;
  const int among = a.k + (ends != 0 ? __builtin_ctz(ends) : 0);
  const bool near = sure && (~gaps & ((1u << among) - 1u) >> 1) != 0;
  if (__ballot(near) != 0) {
    if (a.bias != nullptr && !a.sigmoid) {
      sure = sure && !near;
    } else {
      const bool in = c < among && id >= 0;
      double exact = -__builtin_inf();
      if (in) exact = a.bias == nullptr ? (double)x : 1.0 / (1.0 + exp(-(double)x)) + (double)lds.bias[Lds::at(id)];
      int tag = in ? id : kMaxExperts + c;   // (those behind stay there, in their order)
      // Neighbours change places until two rounds, of even and of odd ones, changed none.
      for (int round = 0, still = 0; still < 2; ++round) {
        const int o = round & 1 ? ((c + 1) ^ 1) - 1 : c ^ 1;
        const int other = o < 0 || o > 15 ? c : o;
        const int lane = (lane_id() & 48) + other;
        const double oe = __shfl(exact, lane);
        const float ox = __shfl(x, lane);
        const int ot = __shfl(tag, lane), oid = __shfl(id, lane);
        const bool ahead = oe > exact || (oe == exact && ot < tag);   // the other belongs ahead of this one
        const bool swap = near && other != c && (other > c ? ahead : !ahead);
        if (swap) {
          exact = oe;
          x = ox;
          tag = ot;
          id = oid;
        }
        still = __ballot(swap) != 0 ? 0 : still + 1;
      }
    }
  }
  const bool on = c < a.k && id >= 0;
  float w;
  if (a.renormalize) {
    const float peak = row_max(on ? x : -kInf);
    w = share_score(on, x, peak, a.sigmoid);
    const float total = row_sum(w);
    w = total == 0.0f ? 0.0f : w / total;
  } else {
    if (plain && !a.sigmoid) {
#pragma unroll
      for (int i = 0; i < V; ++i) sum += l[i] > -kInf ? expf(l[i] - top) : 0.0f;
      sum = row_sum(sum);
    }
    w = a.sigmoid ? sigmoid_of(x) : expf(x - top) / sum;
    if (!on) w = 0.0f;
  }
  if (live && sure && c < a.k) {
    a.ids[t * a.k + c] = id;
    a.weights[t * a.k + c] = bad ? __builtin_nanf("") : a.factor * w;
  }
  return sure || !live;
}

template <class T, int V>
__global__ void __launch_bounds__(256) route_kernel(const RouteArgs a) {
  constexpr int WV = (V + 3) / 4;
  union Lds {
    RowLds<V> row;
    WaveLds<WV> wave;
  };
  static_assert(alignof(Lds) >= 16, "route_row reads sixteen bytes at a time");
  __shared__ Lds lds[4];
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int64_t t0 = ((int64_t)blockIdx.x * 4 + wave) * 4;   // (a wave's LDS is its own: no barrier)
  const bool sure = t0 >= a.tokens || route_row<T, V>(a, t0, lds[wave].row);
  const uint64_t open = __ballot(!sure);
  wave_sync();
  for (int r = 0; r < 4; ++r)
    if (open >> (16 * r) & 1) route_wave<T, WV>(a, t0 + r, lds[wave].wave);
}

// Every token by a wave.
template <class T, int V>
__global__ void __launch_bounds__(256) route_wide_kernel(const RouteArgs a) {
  __shared__ WaveLds<V> lds[4];
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int64_t t = (int64_t)blockIdx.x * 4 + wave;
  if (t < a.tokens) route_wave<T, V>(a, t, lds[wave]);
}

// The gradient.  Of a share r_j = s_j / sum s (renormalised): with G_j = f dw_j,
// softmax dl_j = r_j (G_j - sum_m G_m r_m) at the chosen experts and 0 elsewhere;
// sigmoid the same times 1 - s_j.  Of the scores themselves: softmax dl_e =
// s_e (G_e - sum_m G_m s_m) for every expert, sigmoid G_j s_j (1 - s_j).
template <class T, int V>
__global__ void __launch_bounds__(256) route_grad_kernel(const RouteArgs a) {
  __shared__ float grad[4][V * 64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int64_t t = (int64_t)blockIdx.x * 4 + wave;
  if (t >= a.tokens) return;
  const T* row = (const T*)a.logits + t * a.ldl;
  const int E = a.experts;
  int id = -1;
  float l = 0.0f, g = 0.0f;
  if (lane < a.k) {
    id = a.ids_in[t * a.k + lane];
    if ((uint32_t)id < (uint32_t)E) {
      l = (float)row[id];
      g = a.factor * a.dw[t * a.k + lane];
    } else {
      id = -1;
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) grad[wave][i * 64 + lane] = 0.0f;
  wave_sync();
  float out[V];
  if (a.renormalize || a.sigmoid) {
    float d = g;
    if (a.renormalize) {
      const float r = share_of(id >= 0, l, a.sigmoid);
      d = r * (g - wave_sum(g * r));
      if (a.sigmoid) d *= sigmoid_of(-l);   // 1 - s
    } else {
      d = g * sigmoid_of(l) * sigmoid_of(-l);
    }
    if (id >= 0) atomicAdd(&grad[wave][id], d);
    wave_sync();
#pragma unroll
    for (int i = 0; i < V; ++i) out[i] = grad[wave][i * 64 + lane];
  } else {
    if (id >= 0) atomicAdd(&grad[wave][id], g);
    float x[V], top = -kInf, sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = i * 64 + lane;
      x[i] = e < E ? (float)row[e] : -kInf;
      top = __builtin_fmaxf(top, x[i]);
    }
    top = wave_max(top);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      x[i] = x[i] == -kInf ? 0.0f : expf(x[i] - top);
      sum += x[i];
    }
    sum = wave_sum(sum);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    wave_sync();
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      x[i] *= inv;
      out[i] = grad[wave][i * 64 + lane];
      dot += out[i] * x[i];
    }
    dot = wave_sum(dot);
#pragma unroll
    for (int i = 0; i < V; ++i) out[i] = x[i] * (out[i] - dot);
  }
  T* to = (T*)a.dl + t * a.lddl;
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (i * 64 + lane < E) to[i * 64 + lane] = (T)out[i];
}

// The same with sixteen lanes a token, for up to 16 V experts and sixteen choices: rows
// are put together in LDS and leave in whole lines.
template <class T, int V>
__global__ void __launch_bounds__(256) route_grad_rows_kernel(const RouteArgs a) {
  using Lds = RowLds<V>;
  static_assert(alignof(Lds) >= 16, "read and written sixteen bytes at a time");
  __shared__ Lds all[4];
  Lds& lds = all[threadIdx.x >> 6];
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int64_t t0 = ((int64_t)blockIdx.x * 4 + wave) * 4;
  if (t0 >= a.tokens) return;   // (a wave's LDS is its own: no barrier)
  const int c = lane_id() & 15, r = lane_id() >> 4;
  const int64_t t = t0 + r;
  const int E = a.experts;
  int id = -1;
  float l = 0.0f, g = 0.0f;
  if (t < a.tokens && c < a.k) {
    id = a.ids_in[t * a.k + c];
    if ((uint32_t)id < (uint32_t)E) {
      l = (float)((const T*)a.logits)[t * a.ldl + id];
      g = a.factor * a.dw[t * a.k + c];
    } else {
      id = -1;
    }
  }
#pragma unroll
  for (int i = 0; i < V; i += 4) *(f32x4*)&lds.l[r][Lds::at(c * V) + i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  wave_sync();
  if (a.renormalize || a.sigmoid) {
    float d = g;
    if (a.renormalize) {
      const float s = share_score(id >= 0, l, row_max(id >= 0 ? l : -kInf), a.sigmoid), total = row_sum(s);
      const float share = total == 0.0f ? 0.0f : s / total;
      d = share * (g - row_sum(g * share));
      if (a.sigmoid) d *= sigmoid_of(-l);   // 1 - s
    } else {
      d = g * sigmoid_of(l) * sigmoid_of(-l);
    }
    if (id >= 0) atomicAdd(&lds.l[r][Lds::at(id)], d);
    wave_sync();
  } else {
    if (id >= 0) atomicAdd(&lds.l[r][Lds::at(id)], g);
    // (This lane's experts: c V ..; past the last one none.)
    const T* row = (const T*)a.logits + (t < a.tokens ? t : a.tokens - 1) * a.ldl;
    float x[V], top = -kInf, sum = 0.0f, dot = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = c * V + i;
      x[i] = (float)row[e < E ? e : E - 1];
      x[i] = e < E ? x[i] : -kInf;
      top = __builtin_fmaxf(top, x[i]);
    }
    top = row_max(top);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      x[i] = x[i] == -kInf ? 0.0f : expf(x[i] - top);
      sum += x[i];
    }
    sum = row_sum(sum);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    wave_sync();
    float out[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      x[i] *= inv;
      out[i] = lds.l[r][Lds::at(c * V) + i];
      dot += out[i] * x[i];
    }
    dot = row_sum(dot);
#pragma unroll
    for (int i = 0; i < V; ++i) lds.l[r][Lds::at(c * V) + i] = x[i] * (out[i] - dot);
    wave_sync();
  }
  // Four experts a lane at a time.
#pragma unroll
  for (int i = 0; i < V / 4; ++i) {
    const int flat = (i * 64 + lane_id()) * 4, q = flat / (16 * V), e = flat % (16 * V);
    if (t0 + q >= a.tokens || e >= E) continue;
    const f32x4 d = *(const f32x4*)&lds.l[q][Lds::at(e)];
    T* to = (T*)a.dl + (t0 + q) * a.lddl + e;
    typedef T T4 __attribute__((ext_vector_type(4)));
    typedef T4 T4_any __attribute__((aligned(sizeof(T))));
    if (e + 4 <= E) {
      *(T4_any*)to = T4{(T)d[0], (T)d[1], (T)d[2], (T)d[3]};
    } else {
#pragma unroll
      for (int o = 0; o < 4; ++o)
        if (e + o < E) to[o] = (T)d[o];
    }
  }
}

template <class T>
const void* grad_rows_choice(int experts) {
  if (experts <= 64) return (const void*)&route_grad_rows_kernel<T, 4>;
  if (experts <= 128) return (const void*)&route_grad_rows_kernel<T, 8>;
  return (const void*)&route_grad_rows_kernel<T, 16>;
}

template <class T>
const void* grad_choice(int experts) {
  if (experts <= 64) return (const void*)&route_grad_kernel<T, 1>;
  if (experts <= 128) return (const void*)&route_grad_kernel<T, 2>;
  if (experts <= 256) return (const void*)&route_grad_kernel<T, 4>;
  if (experts <= 512) return (const void*)&route_grad_kernel<T, 8>;
  return (const void*)&route_grad_kernel<T, 16>;
}

template <class T>
const void* wide_choice(int experts) {
  if (experts <= 64) return (const void*)&route_wide_kernel<T, 1>;
  if (experts <= 128) return (const void*)&route_wide_kernel<T, 2>;
  if (experts <= 256) return (const void*)&route_wide_kernel<T, 4>;
  if (experts <= 512) return (const void*)&route_wide_kernel<T, 8>;
  return (const void*)&route_wide_kernel<T, 16>;
}

// The kernel of sixteen lanes a token, for groups and choices that fit them.
template <class T>
const void* row_choice(int per_lane) {
  if (per_lane <= 4) return (const void*)&route_kernel<T, 4>;
  if (per_lane <= 8) return (const void*)&route_kernel<T, 8>;
  return (const void*)&route_kernel<T, 16>;
}

// Launches of at most kMaxRowBlocks workgroups of `per` tokens.
int launch_rows(const void* fn, RouteArgs a, int per, int elem, void* stream) {
  const int64_t tokens = a.tokens, step = kMaxRowBlocks * per;
  for (int64_t at = 0; at < tokens; at += step) {
    RouteArgs part = a;
    part.tokens = tokens - at < step ? tokens - at : step;
    part.logits = (const char*)a.logits + at * a.ldl * elem;
    if (a.ids != nullptr) part.ids = a.ids + at * a.k;
    if (a.weights != nullptr) part.weights = a.weights + at * a.k;
    if (a.ids_in != nullptr) part.ids_in = a.ids_in + at * a.k;
    if (a.dw != nullptr) part.dw = a.dw + at * a.k;
    if (a.dl != nullptr) part.dl = (char*)a.dl + at * a.lddl * elem;
    if (const int st = launch_kernel(fn, (part.tokens + per - 1) / per, 256, &part, stream)) return st;
  }
  return DGEMM_OK;
}

}  // namespace
}  // namespace dg

extern "C" {

int expert_route(int64_t tokens, int64_t experts, int64_t k, int type, const void* logits, int64_t ldl,
                 const float* bias, int score, int64_t groups, int64_t top_groups, int group_best, int renormalize,
                 float factor, int32_t* ids, float* weights, void* stream) {
  using namespace dg;
  if (!valid_type(type)) return DGEMM_ERR_INVALID_TYPE;
  if (tokens < 0 || experts < 0 || k < 0 || k > experts) return DGEMM_ERR_INVALID_DIM;
  if (score != DGEMM_SOFTMAX && score != DGEMM_SIGMOID) return DGEMM_ERR_INVALID_DIM;
  if (groups < 1 || top_groups < 1 || top_groups > groups || experts % groups != 0 ||
      (group_best != 1 && group_best != 2))
    return DGEMM_ERR_INVALID_DIM;
  if (experts > 0 && k > top_groups * (experts / groups)) return DGEMM_ERR_INVALID_DIM;
  if (tokens == 0 || k == 0) return DGEMM_OK;
  if (logits == nullptr || ids == nullptr || weights == nullptr) return DGEMM_ERR_NULL_POINTER;
  if (ldl < experts) return DGEMM_ERR_INVALID_LD;
  if (!aligned_to(logits, type_bytes(type)) || !aligned_to(bias, 4) || !aligned_to(ids, 4) || !aligned_to(weights, 4))
    return DGEMM_ERR_MISALIGNED;
  if (experts > kMaxExperts || k > kMaxChoices || tokens > kMaxCount / k) return DGEMM_ERR_UNSUPPORTED;
  RouteArgs a{};
  a.logits = logits; a.ldl = ldl; a.bias = bias; a.ids = ids; a.weights = weights;
  a.tokens = tokens; a.experts = (int)experts; a.k = (int)k;
  a.sigmoid = score == DGEMM_SIGMOID;
  a.groups = (int)groups; a.top_groups = (int)top_groups; a.group_best = group_best;
  a.renormalize = renormalize != 0; a.factor = factor;
  a.group_size = (int)(experts / groups);
  a.lanes_per_group = groups <= 16 ? 16 / (int)groups : 0;
  if (a.lanes_per_group > 0) a.per_lane = (a.group_size + a.lanes_per_group - 1) / a.lanes_per_group;
  const bool rows = a.lanes_per_group > 0 && a.per_lane <= kRowExperts && k <= kRowChoices;
  const void* fn = with_type(type, [&](auto t) {
    using T = decltype(t);
    return rows ? row_choice<T>(a.per_lane) : wide_choice<T>((int)experts);
  });
  return launch_rows(fn, a, rows ? 16 : 4, type_bytes(type), stream);
}

int expert_route_grad(int64_t tokens, int64_t experts, int64_t k, int type, const void* logits, int64_t ldl,
                      const int32_t* ids, const float* dweights, int score, int renormalize, float factor,
                      void* dlogits, int64_t lddl, void* stream) {
  using namespace dg;
  if (!valid_type(type)) return DGEMM_ERR_INVALID_TYPE;
  if (tokens < 0 || experts < 0 || k < 0) return DGEMM_ERR_INVALID_DIM;
  if (score != DGEMM_SOFTMAX && score != DGEMM_SIGMOID) return DGEMM_ERR_INVALID_DIM;
  if (tokens == 0 || experts == 0) return DGEMM_OK;
  if (logits == nullptr || (k > 0 && (ids == nullptr || dweights == nullptr)) || dlogits == nullptr)
    return DGEMM_ERR_NULL_POINTER;
  if (ldl < experts || lddl < experts) return DGEMM_ERR_INVALID_LD;
  if (!aligned_to(logits, type_bytes(type)) || !aligned_to(dlogits, type_bytes(type)) || !aligned_to(ids, 4) ||
      !aligned_to(dweights, 4))
    return DGEMM_ERR_MISALIGNED;
  if (experts > kMaxExperts || k > kMaxChoices || tokens > kMaxCount / (k > 0 ? k : 1)) return DGEMM_ERR_UNSUPPORTED;
  RouteArgs a{};
  a.logits = logits; a.ldl = ldl; a.ids_in = ids; a.dw = dweights; a.dl = dlogits; a.lddl = lddl;
  a.tokens = tokens; a.experts = (int)experts; a.k = (int)k;
  a.sigmoid = score == DGEMM_SIGMOID;
  a.renormalize = renormalize != 0; a.factor = factor;
  const bool rows = experts <= 16 * kRowExperts && k <= 16;
  const void* fn = with_type(type, [&](auto t) {
    using T = decltype(t);
    return rows ? grad_rows_choice<T>((int)experts) : grad_choice<T>((int)experts);
  });
  return launch_rows(fn, a, rows ? 16 : 4, type_bytes(type), stream);
}

}  // extern "C"
