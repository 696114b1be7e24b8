// route_topk.cu — routing of any number of experts and choices per token
// (moe_topk_route), its backward pass and the dispatch of its choice.
//
// One warp takes one token. Lane L holds the logits of the experts L * VPL ..
// L * VPL + VPL - 1 (VPL = E / 32 rounded up to a power of two). With groups each group
// has a run of lanes of its own (32 lanes over the groups, rounded to powers of two), so
// that what is asked of a group is a reduction within its run. "The lower expert" is the
// lower lane, then the lower register.
//
// Bound by instructions, not by the logits' bytes (16384 tokens x 256 experts: 16.8 MB,
// 2.6 us at the copy rate), so the common path is built of few of them. A rank value
// becomes a 32-bit key that sorts like it (as an unsigned number), whose lowest
// log2(VPL) bits are replaced by the register index. Each lane sorts its keys once
// (VPL <= 8), and each of the k rounds is one redux of the lanes' first keys, one ballot
// for the lowest lane that holds it, and a shift in that lane.
//
// The choice is that of the 64-bit values. What a key may be off by is known (`err`: the
// bits given to the index, and with a bias the fp32 rounding of score + bias, derived
// at score_error); a round whose winner is less than 2 err ahead of the next value, or
// a group limit that close, is undecided, and those experts are compared again in 64
// bits. With normal logits that is about one token in a hundred. Logits of
// few mantissa bits (bf16 ones) lose nothing to the index and are decided exactly.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "moe_internal.cuh"
#include "sm100.cuh"

namespace moe {
namespace {

constexpr int kTopkBlock = 32;      // tokens of a routing CTA: one bit each of a 32-bit mask per expert
constexpr int kMaxExperts = 1024;
constexpr unsigned kFull = 0xffffffffu;

struct TopkParams {
  const void* logits;
  const float* bias;
  const int32_t* n_tokens;
  int64_t T;
  int32_t E, k, n_groups, topk_groups, group_size, score, rule, renorm;
  int32_t lane_run;     // lanes per group (a power of two); 0: one group, or too many for runs
  int32_t run_shift;    // its logarithm
  float scale;
  int32_t* idx;
  float* weights;
  float* scores;
  // dispatch (counts == nullptr: none); hist and totals with more than kClusterBlocks blocks
  int32_t* counts;
  int32_t* offsets;
  int32_t* perm_token;
  int32_t* perm_slot;
  int32_t* slot_pos;
  float* gate_perm;
  int32_t* hist;    // [nblk, E] slots per token block, then their exclusive prefix over blocks
  int32_t* totals;  // [E]
  int64_t nblk;
  uint32_t* status; // status word of the workspace, if one is given: nothing here can fail, so it is set to 0
};

__device__ __forceinline__ int64_t token_count(const TopkParams& p) {
  if (p.n_tokens == nullptr) return p.T;
  const int64_t n = __ldg(p.n_tokens);
  return n < 0 ? 0 : (n < p.T ? n : p.T);
}

// fp32 value of a logit as the routing sees it: NaN masks (the maximum of NaN and a
// number is the number), +inf is the largest.
__device__ __forceinline__ float clean(float l) { return fminf(fmaxf(l, -INFINITY), FLT_MAX); }

template <bool BF16>
__device__ __forceinline__ float load_logit(const void* logits, int64_t at) {
  if (BF16) return clean(__bfloat162float(static_cast<const __nv_bfloat16*>(logits)[at]));
  return clean(static_cast<const float*>(logits)[at]);
}

// Experts of a lane: `first`, and the end of those it may hold (those of its group, or all).
struct LaneExperts {
  int first, end;
};
template <int VPL>
__device__ __forceinline__ LaneExperts lane_experts(const TopkParams& p, int lane) {
  if (p.lane_run == 0) return {lane * VPL, p.E};
  const int g = lane >> p.run_shift;
  if (g >= p.n_groups) return {p.E, p.E};
  return {g * p.group_size + (lane & (p.lane_run - 1)) * VPL, (g + 1) * p.group_size};
}

// W values of a type next to one another in memory, as one access.
template <typename T, int W>
struct alignas(sizeof(T) * W) Pack {
  T v[W];
};

// Calls f with the widest access (16 bytes at most) that divides a lane's registers and
// `unit` experts: all rows and lanes then start on its boundary. (Rows of 372 bf16 logits
// one by one: gradient of 11275 tokens 36 us a call.)
template <int VPL, int MOST, typename F>
__device__ __forceinline__ void with_width(int unit, F f) {
  if constexpr (MOST > VPL) {
    with_width<VPL, MOST / 2>(unit, f);
  } else if constexpr (MOST == 1) {
    f(std::integral_constant<int, 1>{});
  } else {
    if (unit % MOST == 0) f(std::integral_constant<int, MOST>{});
    else with_width<VPL, MOST / 2>(unit, f);
  }
}

// Logits of this lane's experts; -inf past the last one.
template <bool BF16, int VPL>
__device__ __forceinline__ void load_row(const void* logits, int64_t t, int row_len, int unit, LaneExperts mine,
                                         float (&l)[VPL]) {
  using T = std::conditional_t<BF16, uint16_t, float>;
  const T* at = static_cast<const T*>(logits) + t * row_len + mine.first;
  with_width<VPL, 16 / sizeof(T)>(unit, [&](auto width) {
    constexpr int W = decltype(width)::value;
#pragma unroll
    for (int v = 0; v < VPL; v += W) {
      if (mine.first + v < mine.end) {
        const Pack<T, W> w = *reinterpret_cast<const Pack<T, W>*>(at + v);
#pragma unroll
        for (int j = 0; j < W; ++j) {
          if constexpr (BF16) l[v + j] = clean(__uint_as_float(static_cast<uint32_t>(w.v[j]) << 16));
          else l[v + j] = clean(w.v[j]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < W; ++j) l[v + j] = -INFINITY;
      }
    }
  });
}

// Biases of this lane's experts (left as they are past the last one).
template <int VPL>
__device__ __forceinline__ void load_bias(const float* bias, int unit, LaneExperts mine, float (&b)[VPL]) {
  with_width<VPL, 4>(unit, [&](auto width) {
    constexpr int W = decltype(width)::value;
#pragma unroll
    for (int v = 0; v < VPL; v += W) {
      if (mine.first + v >= mine.end) continue;
      const Pack<float, W> w = *reinterpret_cast<const Pack<float, W>*>(bias + mine.first + v);
#pragma unroll
      for (int j = 0; j < W; ++j) b[v + j] = w.v[j];
    }
  });
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
  return v;
}
template <typename V>
__device__ __forceinline__ V warp_add(V v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

// 2^x within 2 ulp and 1 / x within 1 ulp, results below the normal range as zero.
__device__ __forceinline__ float ex2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float sigmoid(float l) { return 1.0f / (1.0f + expf(-l)); }

// Order-preserving map of floats to unsigned and back. -0 and +0 are made one first,
// so that they tie.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
constexpr uint32_t kNoKey = 0;
// Keys of finite and infinite values start here; smaller ones (-inf, or cleared) stand
// for experts that cannot be chosen.
constexpr uint32_t kFirstKey = 0x00800000u;

// ---- 64-bit values -------------------------------------------------------------
// Near ties are decided on 64-bit keys that sort like doubles. One such token can be the
// last of its kernel, so its own time counts (it was 10 us of 35 for 16384 tokens of 256
// experts while every expert was scored again), and much of that is fetching instructions
// that no cache holds: only the experts in question are scored again, by one shared
// function, a lane each, and what must look at all experts keeps its loops rolled.

// 64-bit score of a logit (softmax: the logit less the row's largest; z: the row's sum).
__device__ __noinline__ double exact_score(int score, double x, double z) {
  const bool soft = score == MOE_SCORE_SOFTMAX;
  const double e = exp(soft ? x : -x);
  return (soft ? e : 1.0) / (soft ? z : 1.0 + e);
}

// What a token's 64-bit values take besides the logit.
struct ExactRow {
  double top = 0.0, z = 1.0;  // softmax: the largest logit and the sum
};

template <bool BF16, int VPL>
__device__ __noinline__ ExactRow exact_row(const TopkParams& p, int64_t t, int lane) {
  ExactRow r;
  if (p.score != MOE_SCORE_SOFTMAX) return r;
  float m = -INFINITY;
#pragma unroll 1
  for (int e = lane; e < p.E; e += 32) m = fmaxf(m, load_logit<BF16>(p.logits, t * p.E + e));
  m = warp_max(m);
  if (m > -INFINITY) r.top = static_cast<double>(m);
  r.z = 0.0;
#pragma unroll 1
  for (int e = lane; e < p.E; e += 32)
    r.z += exact_score(MOE_SCORE_SOFTMAX, static_cast<double>(load_logit<BF16>(p.logits, t * p.E + e)) - r.top, 1.0);
  r.z = warp_add(r.z);
  return r;
}

// 64-bit value of expert e of token t: score + bias, or the logit.
template <bool BF16>
__device__ __forceinline__ double exact_value(const TopkParams& p, int64_t t, int e, bool by_score, const ExactRow& r) {
  const double x = static_cast<double>(load_logit<BF16>(p.logits, t * p.E + e));
  if (!by_score) return x;
  const double s = exact_score(p.score, p.score == MOE_SCORE_SOFTMAX ? x - r.top : x, r.z);
  return p.bias != nullptr ? s + static_cast<double>(__ldg(p.bias + e)) : s;
}

__device__ __forceinline__ uint64_t order_key64(double v) {
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(v + 0.0));
  return b ^ (static_cast<uint64_t>(static_cast<int64_t>(b) >> 63) | 0x8000000000000000ull);
}
__device__ __forceinline__ double key_value64(uint64_t k) {
  return __longlong_as_double(
      static_cast<long long>(k & 0x8000000000000000ull ? k ^ 0x8000000000000000ull : ~k));
}
constexpr uint64_t kFirstKey64 = 0x0010000000000000ull;  // below: -inf, or no value

// The warp's largest key (0 = none) and the lowest lane that holds it.
__device__ __forceinline__ uint64_t warp_best64(uint64_t k, int& src) {
  const uint32_t hi = static_cast<uint32_t>(k >> 32);
  const uint32_t mh = __reduce_max_sync(kFull, hi);
  const uint32_t lo = hi == mh ? static_cast<uint32_t>(k) : 0;
  const uint32_t ml = __reduce_max_sync(kFull, lo);
  src = __ffs(__ballot_sync(kFull, hi == mh && static_cast<uint32_t>(k) == ml)) - 1;
  return static_cast<uint64_t>(mh) << 32 | ml;
}

// Two largest of a set, held as (a >= b).
__device__ __forceinline__ void push2(uint64_t& a, uint64_t& b, uint64_t v) {
  b = max(b, min(a, v));
  a = max(a, v);
}

// Bits of the leaders of the groups that stay (see kept_groups).
template <int VPL>
__device__ __forceinline__ unsigned kept_groups_exact(const TopkParams& p, int lane, const uint64_t* key) {
  const int G = p.n_groups;
  const bool runs = p.lane_run > 0;
  uint64_t a = 0, b = 0;
#pragma unroll 1
  for (int g = 0; g < (runs ? 1 : G); ++g) {
    uint64_t c = 0, d = 0;
#pragma unroll 1
    for (int j = 0; j < VPL; ++j)
      if (runs || (lane * VPL + j) / p.group_size == g) push2(c, d, key[j]);
#pragma unroll 1
    for (int o = 1; o < (runs ? p.lane_run : 32); o <<= 1) {
      const uint64_t c2 = __shfl_xor_sync(kFull, c, o), d2 = __shfl_xor_sync(kFull, d, o);
      push2(c, d, c2);
      push2(c, d, d2);
    }
    if (runs || lane == g) {
      a = c;
      b = d;
    }
  }
  const bool leader = runs ? (lane & (p.lane_run - 1)) == 0 && lane < G * p.lane_run : lane < G;
  double mine = -INFINITY;
  if (a >= kFirstKey64) {
    mine = key_value64(a);
    if (p.rule == MOE_GROUP_TOP2_SUM && b >= kFirstKey64) mine += key_value64(b);
  }
  uint64_t left = leader ? order_key64(mine) + 1 : 0;  // an empty group is above no group
  unsigned kept = 0;
#pragma unroll 1
  for (int i = 0; i < p.topk_groups; ++i) {
    int src;
    warp_best64(left, src);
    kept |= 1u << src;
    if (lane == src) left = 0;
  }
  return kept;
}

template <int VPL>
__device__ __forceinline__ int take_k_exact(uint64_t* key, int k, int lane, int e0) {
  int pick = -1;
#pragma unroll 1
  for (int i = 0; i < k; ++i) {
    uint64_t best = 0;
    int at = 0;
#pragma unroll 1
    for (int j = 0; j < VPL; ++j)
      if (key[j] > best) {
        best = key[j];
        at = j;
      }
    int src;
    if (warp_best64(best, src) < kFirstKey64) break;
    const int e = __shfl_sync(kFull, e0 + at, src);
    if (lane == i) pick = e;
    if (lane == src) key[at] = 0;
  }
  return pick;
}

// ---- common path: 32-bit keys ------------------------------------------------

// Largest first.
template <int VPL>
__device__ __forceinline__ void sort_keys(uint32_t (&k)[VPL]) {
  auto order = [&](int i, int j) {
    const uint32_t hi = max(k[i], k[j]), lo = min(k[i], k[j]);
    k[i] = hi;
    k[j] = lo;
  };
  if constexpr (VPL == 2) {
    order(0, 1);
  } else if constexpr (VPL == 4) {
    order(0, 1); order(2, 3); order(0, 2); order(1, 3); order(1, 2);
  } else if constexpr (VPL == 8) {  // odd-even merges of sorted halves
    order(0, 1); order(2, 3); order(4, 5); order(6, 7);
    order(0, 2); order(1, 3); order(4, 6); order(5, 7);
    order(1, 2); order(5, 6);
    order(0, 4); order(1, 5); order(2, 6); order(3, 7);
    order(2, 4); order(3, 5);
    order(1, 2); order(3, 4); order(5, 6);
  }
}

// Two largest of two such pairs (a >= b, c >= d).
__device__ __forceinline__ void merge2(uint32_t& a, uint32_t& b, uint32_t c, uint32_t d) {
  b = max(min(a, c), max(b, d));
  a = max(a, c);
}

// Value of a key without its index bits, and what that may differ from the value the key
// was made of, in units of its magnitude: VPL - 1 steps of at most 2^-23, half a step
// for the addition of a bias and half for the sum of two.
template <int VPL>
__device__ __forceinline__ float bare_value(uint32_t k) {
  return key_value(k & ~static_cast<uint32_t>(VPL - 1));
}
template <int VPL>
__device__ constexpr float key_slack() {
  return 1.2e-7f * VPL + 1.2e-7f;
}
// Below the normal range a step is 2^-149 whatever the value and the slack rounds to nothing:
// what a key is off by there, as a value's own error (comparisons take it twice or more).
template <int VPL>
__device__ constexpr float key_floor() {
  return VPL * 0x1p-149f;
}

// The same from 64-bit values, for groups that are runs of lanes: every lane scores those
// of its experts again that may be one of the group's two largest (a, b: the group's two
// largest keys), one after the other.
template <bool BF16, int VPL>
__device__ __noinline__ unsigned settle_groups(const TopkParams& p, int64_t t, int lane, const uint32_t (&key)[VPL],
                                               bool by_score, float err, uint32_t a, uint32_t b) {
  const bool sum = p.rule == MOE_GROUP_TOP2_SUM;
  const uint32_t least = sum ? b : a;
  float limit = -INFINITY;
  if (least >= kFirstKey) {
    const float v = bare_value<VPL>(least);
    limit = v < INFINITY ? v - 2.0f * err - 3.0f * key_slack<VPL>() * fabsf(v) : v;
  }
  const ExactRow row = by_score ? exact_row<BF16, VPL>(p, t, lane) : ExactRow{};
  const int e0 = lane_experts<VPL>(p, lane).first;
  uint64_t c = 0, d = 0;
  uint32_t below = 0xffffffffu;
  for (int j = 0; j < VPL; ++j) {
    // the lane's largest key below the last one (keys of a lane differ in their index bits)
    uint32_t k = kNoKey;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (key[i] < below) k = max(k, key[i]);
    below = k;
    const bool look = k >= kFirstKey && bare_value<VPL>(k) >= limit;
    if (!__any_sync(kFull, look)) break;
    if (look) {
      const double v = exact_value<BF16>(p, t, e0 + VPL - 1 - static_cast<int>(k & (VPL - 1)), by_score, row);
      push2(c, d, order_key64(v));
    }
    __syncwarp();
  }
  for (int o = 1; o < p.lane_run; o <<= 1) {
    const uint64_t c2 = __shfl_xor_sync(kFull, c, o), d2 = __shfl_xor_sync(kFull, d, o);
    push2(c, d, c2);
    push2(c, d, d2);
  }
  double mine = -INFINITY;
  if (c >= kFirstKey64) mine = key_value64(c) + (sum && d >= kFirstKey64 ? key_value64(d) : 0.0);
  const bool leader = (lane & (p.lane_run - 1)) == 0 && lane < p.n_groups * p.lane_run;
  uint64_t left = leader ? order_key64(mine) + 1 : 0;
  unsigned kept = 0;
  for (int i = 0; i < p.topk_groups; ++i) {
    int src;
    warp_best64(left, src);
    kept |= 1u << src;
    if (lane == src) left = 0;
  }
  return kept;
}

// Bits of the leaders of the groups that stay (lane g for group g, or the first lane of
// its run where groups are whole runs of lanes), from the keys the groups go by.
// Where two groups on either side of the limit are closer than their errors, the groups
// are valued again in 64 bits; `undecided` is set where groups are no runs of lanes, or
// values infinite.
template <bool BF16, int VPL>
__device__ __forceinline__ unsigned kept_groups(const TopkParams& p, int64_t t, int lane, const uint32_t (&key)[VPL],
                                                bool by_score, float err, bool& undecided) {
  constexpr bool kSorted = VPL <= 8;
  const int gs = p.group_size, G = p.n_groups;
  const bool sum = p.rule == MOE_GROUP_TOP2_SUM;
  uint32_t a = kNoKey, b = kNoKey;  // leaders: the two largest keys of the group
  bool leader = lane < G;
  if (p.lane_run > 0) {
    // a group is a run of whole lanes, a power of two of them: reduce within the run
    if (kSorted) {
      a = key[0];
      b = VPL > 1 ? key[VPL > 1 ? 1 : 0] : kNoKey;
    } else {
#pragma unroll
      for (int j = 0; j < VPL; ++j) merge2(a, b, key[j], kNoKey);
    }
    for (int o = 1; o < p.lane_run; o <<= 1) {
      const uint32_t c = __shfl_xor_sync(kFull, a, o), d = __shfl_xor_sync(kFull, b, o);
      merge2(a, b, c, d);
    }
    leader = (lane & (p.lane_run - 1)) == 0 && lane < G * p.lane_run;
  } else {
    for (int g = 0; g < G; ++g) {
      uint32_t c = kNoKey, d = kNoKey;
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        // the register a key came from: its own place, or its index bits once sorted
        const int e = lane * VPL + (kSorted ? VPL - 1 - static_cast<int>(key[j] & (VPL - 1)) : j);
        if (e / gs == g) merge2(c, d, key[j], kNoKey);
      }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t c2 = __shfl_xor_sync(kFull, c, o), d2 = __shfl_xor_sync(kFull, d, o);
        merge2(c, d, c2, d2);
      }
      if (lane == g) {
        a = c;
        b = d;
      }
    }
  }
  float mine = -INFINITY, size = 0.0f;  // the group's value, and the magnitude its error goes by
  if (a >= kFirstKey) {
    mine = bare_value<VPL>(a);
    size = fabsf(mine);
    if (sum && b >= kFirstKey) {
      const float second = bare_value<VPL>(b);
      // a sum that leaves the fp32 range to -inf would tie with an empty group; its size is
      // infinite, so that the limit next to it is decided in 64 bits
      mine = fmaxf(mine + second, -FLT_MAX);
      size += fabsf(second);
    }
  }
  // largest first, the lower group among equal ones; + 1: an empty group is above no group
  uint32_t left = leader ? order_key(mine) + 1 : 0;
  unsigned kept = 0;
  int src = 0;
  for (int i = 0; i < p.topk_groups; ++i) {
    src = __ffs(__ballot_sync(kFull, left == __reduce_max_sync(kFull, left))) - 1;
    kept |= 1u << src;
    if (lane == src) left = 0;
  }
  if (p.topk_groups < G && err >= 0.0f) {
    // the worst of those that stay against the best of those that go
    const int next = __ffs(__ballot_sync(kFull, left == __reduce_max_sync(kFull, left))) - 1;
    const float low = __shfl_sync(kFull, mine, src), high = __shfl_sync(kFull, mine, next);
    const float sizes = __shfl_sync(kFull, size, src) + __shfl_sync(kFull, size, next);
    // an empty group is exact
    if (high != -INFINITY && !(low - high > 4.0f * err + key_slack<VPL>() * sizes)) {
      if (p.lane_run == 0 || !(sizes < INFINITY)) undecided = true;
      else kept = settle_groups<BF16, VPL>(p, t, lane, key, by_score, err, a, b);
    }
  }
  return kept;
}

// The m choices that lanes 0 .. m-1 hold (in `pick`), put in the order of their 64-bit
// values: lane i ends with the i-th.
template <bool BF16, int VPL>
__device__ __noinline__ int settle_order(const TopkParams& p, int64_t t, int lane, int pick, int m, bool by_score) {
  const ExactRow row = by_score ? exact_row<BF16, VPL>(p, t, lane) : ExactRow{};
  double v = 0.0;
  if (lane < m) v = exact_value<BF16>(p, t, pick, by_score, row);
  __syncwarp();
  int place = 0, sorted = -1;
  for (int i = 0; i < m; ++i) {
    const double o = __shfl_sync(kFull, v, i);
    const int e = __shfl_sync(kFull, pick, i);
    place += (o > v || (o == v && e < pick)) ? 1 : 0;
  }
  for (int i = 0; i < m; ++i) {
    const int at = __shfl_sync(kFull, place, i), e = __shfl_sync(kFull, pick, i);
    if (lane == at) sorted = e;
  }
  return sorted;
}

// k rounds of the warp's largest key. Lane i ends with the i-th choice in `pick` (-1:
// none left). `err` < 0: the keys lost nothing, every comparison is exact. Else one or two
// more rounds look at the values behind the last; where neighbours are closer than both may
// be off, and the k-th or the one behind it is clear of the next, those before that gap
// are put in the order of their 64-bit values. `undecided`: there is no such gap.
template <bool BF16, int VPL>
__device__ __forceinline__ void take_k(const TopkParams& p, int64_t t, uint32_t (&key)[VPL], int lane, bool by_score,
                                       float err, bool& undecided, int& pick) {
  constexpr bool kSorted = VPL <= 8;
  constexpr uint32_t kIndex = VPL - 1;
  const int k = p.k;
  uint32_t best = key[0], mine = kNoKey;
  if (!kSorted) {
#pragma unroll
    for (int j = 1; j < VPL; ++j) best = max(best, key[j]);
  }
  int from = 0;
  // Two neighbours closer than both may be off (infinite values are close to everything).
  auto near = [&](uint32_t hi, uint32_t lo) {
    const float a = key_value(hi), b = key_value(lo);
    return lo >= kFirstKey && !(a - b > 2.0f * err + key_slack<VPL>() * (fabsf(a) + fabsf(b)));
  };
  auto round = [&](int i) {
    // the values alone decide; among equal ones the lowest lane, in it the lowest register
    const uint32_t head = best | kIndex;
    const uint32_t m = __reduce_max_sync(kFull, head);
    if (m < kFirstKey) return false;
    const int src = __ffs(__ballot_sync(kFull, head == m)) - 1;
    const uint32_t full = __shfl_sync(kFull, best, src);
    mine = lane == i ? full : mine;
    from = lane == i ? src : from;
    const bool own = lane == src;
    if (kSorted) {
#pragma unroll
      for (int j = 0; j + 1 < VPL; ++j) key[j] = own ? key[j + 1] : key[j];
      key[VPL - 1] = own ? kNoKey : key[VPL - 1];
      best = key[0];
    } else if (own) {
      best = kNoKey;
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        if (key[j] == full) key[j] = kNoKey;
        best = max(best, key[j]);
      }
    }
    return true;
  };
  const int rounds = err >= 0.0f ? min(k + 1, 32) : k;
  for (int i = 0; i < rounds; ++i)
    if (!round(i)) break;
  bool has = mine >= kFirstKey;
  if (err >= 0.0f) {
    // lanes whose value is near the next lane's (lane 31 knows no next)
    auto close = [&] {
      const uint32_t next = __shfl_down_sync(kFull, mine, 1);
      return __ballot_sync(kFull, has && (lane == 31 || near(mine, next)));
    };
    unsigned near_next = close();
    if (near_next & (k == 32 ? kFull : (1u << k) - 1u)) {  // among the choices, or behind the last
      int m = k;
      if ((near_next >> (k - 1)) & 1u) {  // is the one behind the last clear of the next?
        if (k < 31) round(k + 1);
        has = mine >= kFirstKey;
        near_next = close();
        m = k < 31 && !((near_next >> k) & 1u) ? k + 1 : 0;
      }
      pick = has ? lane_experts<VPL>(p, from).first + (VPL - 1 - static_cast<int>(mine & kIndex)) : -1;
      if (m == 0 || __any_sync(kFull, has && !(fabsf(key_value(mine)) < INFINITY))) undecided = true;
      else pick = settle_order<BF16, VPL>(p, t, lane, pick, min(m, __popc(__ballot_sync(kFull, has))), by_score);
      if (lane >= k) pick = -1;
      return;
    }
  }
  pick = has && lane < k ? lane_experts<VPL>(p, from).first + (VPL - 1 - static_cast<int>(mine & kIndex)) : -1;
}

// Scores of this lane's experts, the row's largest logit and, for softmax, the sum.
template <int VPL>
__device__ __forceinline__ void row_scores(int score, const float (&l)[VPL], float (&s)[VPL], float& top, float& z) {
  top = -INFINITY;
  z = 1.0f;
  if (score == MOE_SCORE_SIGMOID) {
#pragma unroll
    for (int j = 0; j < VPL; ++j) s[j] = l[j] == -INFINITY ? 0.0f : sigmoid(l[j]);
    return;
  }
#pragma unroll
  for (int j = 0; j < VPL; ++j) top = fmaxf(top, l[j]);
  top = warp_max(top);
  float sum = 0.0f;
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    s[j] = l[j] == -INFINITY ? 0.0f : expf(l[j] - top);
    sum += s[j];
  }
  z = warp_add(sum);
  if (!(z > 0.0f)) z = 1.0f;
#pragma unroll
  for (int j = 0; j < VPL; ++j) s[j] /= z;
}

// Scores for the ranking alone: approximate exponential and quotient, and for softmax the
// largest logit and the sum. Written scores are row_scores'. Softmax weights that are not
// renormalised divide an accurate exponential by the sum at hand: this one, within 2.8e-6 of
// the exact sum (score_error), unless the scores are written, too, so their last bits
// may differ between calls with and without them.
template <int VPL>
__device__ __forceinline__ void rank_scores(int score, const float (&l)[VPL], float (&s)[VPL], float& s_top,
                                            float& top, float& z) {
  if (score == MOE_SCORE_SIGMOID) {
#pragma unroll
    for (int j = 0; j < VPL; ++j) s[j] = rcp_fast(1.0f + ex2_fast(-kLog2e * l[j]));
    s_top = 1.0f;
    return;
  }
  top = -INFINITY;
#pragma unroll
  for (int j = 0; j < VPL; ++j) top = fmaxf(top, l[j]);
  top = key_value(__reduce_max_sync(kFull, order_key(top)));
  float sum = 0.0f;
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    s[j] = l[j] == -INFINITY ? 0.0f : ex2_fast(kLog2e * (l[j] - top));
    sum += s[j];
  }
  z = warp_add(sum);
  if (!(z > 0.0f)) z = 1.0f;
  s_top = rcp_fast(z);
#pragma unroll
  for (int j = 0; j < VPL; ++j) s[j] *= s_top;
}

// What rank_scores may be off by, with u = 2^-24. 2^(x log2 e): the product's rounding
// and log2 e's own count 2 |x| u in the exponent, ex2 2 ulp (4 u). Sigmoid, x = -l: s =
// 1 / (1 + e^x), so a relative error d of the exponential is s (1 - s) d absolute; with
// s (1 - s) <= 0.25 and |x| s (1 - s) <= 0.23 at most (0.46 + 1) u, plus sum u and
// reciprocal 2 u: below 5 u; scores that e^x > 2^126 flushes to zero are below 2^-126.
// Softmax, x = l - max <= 0, itself rounded by |x| u: |x| e^x <= 0.37, so a term is off by
// at most 3 * 0.37 + 4 < 6 u of the largest term, the sum of 1024 terms by that and
// 37 u, reciprocal 2 u, product u: 46 u of the largest score. The addition of the bias:
// u |c|, part of key_slack.
__device__ __forceinline__ float score_error(int score, float s_top) {
  return score == MOE_SCORE_SIGMOID ? 3.0e-7f : 3.0e-6f * s_top;
}

// The choice from 64-bit values. A call of its own: its registers are not those
// of the common path.
template <bool BF16, int VPL>
__device__ __noinline__ int choose_exact(const TopkParams& p, int64_t t, int lane) {
  const bool biased = p.bias != nullptr, sums = p.n_groups > 1 && p.rule == MOE_GROUP_TOP2_SUM;
  const ExactRow row = biased || sums ? exact_row<BF16, VPL>(p, t, lane) : ExactRow{};
  const LaneExperts own = lane_experts<VPL>(p, lane);
  uint64_t key[VPL];
  unsigned kept = kFull;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {  // sums without a bias: groups by scores, then experts by logits
    const bool by_score = biased || (pass == 0 && sums);
#pragma unroll 1
    for (int j = 0; j < VPL; ++j) {
      const int e = own.first + j;
      uint64_t k = 0;
      if (e < own.end && load_logit<BF16>(p.logits, t * p.E + e) > -INFINITY) {
        const double v = exact_value<BF16>(p, t, e, by_score, row);
        if (!(v != v)) k = order_key64(v);
      }
      key[j] = k;
      __syncwarp();
    }
    if (pass == 0 && p.n_groups > 1) kept = kept_groups_exact<VPL>(p, lane, key);
    if (biased || !sums) break;
  }
  if (p.n_groups > 1) {
#pragma unroll 1
    for (int j = 0; j < VPL; ++j) {
      const int g = p.lane_run > 0 ? lane & ~(p.lane_run - 1) : (lane * VPL + j) / p.group_size;
      if (g >= 32 || !((kept >> g) & 1u)) key[j] = 0;
    }
  }
  return take_k_exact<VPL>(key, p.k, lane, own.first);
}

// Share of each choice in the renormalised weights (P lanes of a warp, a power of two,
// hold the choices of one token; logit lv, -inf = none): s / sum s, computed from
// differences of logits, so that scores below the fp32 range still share. Sigmoid
// scores e^l / (1 + e^l) over e^top, unless the largest logit is positive: then the largest
// score is above a half, and scores below the fp32 range have no share in it.
__device__ __forceinline__ float share_of(int score, float lv, int P) {
  float top = lv;
  for (int o = 1; o < P; o <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
  float x = 0.0f;
  if (lv > -INFINITY) {
    if (score == MOE_SCORE_SIGMOID && top > 0.0f) x = sigmoid(lv);
    else x = expf(lv - top) / (score == MOE_SCORE_SIGMOID ? 1.0f + expf(lv) : 1.0f);
  }
  float sum = x;
  for (int o = 1; o < P; o <<= 1) sum += __shfl_xor_sync(kFull, sum, o);
  return sum > 0.0f ? x / sum : 0.0f;
}

// The choice of one token: lane i < k ends with choice i. For softmax weights and
// scores also the row's largest logit and its sum.
template <bool BF16, int VPL>
__device__ __forceinline__ int choose(const TopkParams& p, int64_t t, int lane, float& top, float& z) {
  float l[VPL];
  const LaneExperts own = lane_experts<VPL>(p, lane);
  load_row<BF16, VPL>(p.logits, t, p.E, p.group_size, own, l);
  const bool groups = p.n_groups > 1, sums = groups && p.rule == MOE_GROUP_TOP2_SUM;
  const bool biased = p.bias != nullptr;
  float s[VPL], s_top = 1.0f;
  if (p.scores != nullptr) {
    row_scores<VPL>(p.score, l, s, top, z);
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (own.first + j < own.end) p.scores[t * p.E + own.first + j] = s[j];
    if (p.score == MOE_SCORE_SOFTMAX) s_top = 1.0f / z;
  } else if (biased || sums || (p.score == MOE_SCORE_SOFTMAX && p.renorm == 0)) {
    rank_scores<VPL>(p.score, l, s, s_top, top, z);
  }
  // Keys by score + bias, or by the logit; groups that sum scores without a bias go
  // by keys of their own.
  uint32_t key[VPL];
  auto by_score = [&] {
    float bias[VPL];
#pragma unroll
    for (int j = 0; j < VPL; ++j) bias[j] = 0.0f;
    if (biased) load_bias<VPL>(p.bias, p.group_size, own, bias);
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      // 0 * l: NaN for a masked expert; the maximum turns NaN into -inf
      const float v = fmaxf(fmaf(l[j], 0.0f, s[j] + bias[j]), -INFINITY);
      key[j] = (order_key(v) & ~static_cast<uint32_t>(VPL - 1)) | static_cast<uint32_t>(VPL - 1 - j);
    }
    if (VPL <= 8) sort_keys<VPL>(key);
  };
  bool undecided = false;
  unsigned kept = kFull;
  float err = score_error(p.score, s_top);
  if (sums && !biased) {
    by_score();
    kept = kept_groups<BF16, VPL>(p, t, lane, key, true, err, undecided);
  }
  if (biased) {
    by_score();
  } else {
    uint32_t lost = 0;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      lost |= __float_as_uint(l[j]);
      key[j] = (order_key(l[j]) & ~static_cast<uint32_t>(VPL - 1)) | static_cast<uint32_t>(VPL - 1 - j);
    }
    if (VPL <= 8) sort_keys<VPL>(key);
    // exact where no logit has a bit that the index took
    err = VPL > 1 && __any_sync(kFull, (lost & (VPL - 1)) != 0) ? key_floor<VPL>() : -1.0f;
  }
  if (groups && !(sums && !biased)) kept = kept_groups<BF16, VPL>(p, t, lane, key, biased, err, undecided);
  if (groups && p.lane_run > 0) {
    if (!((kept >> (lane & ~(p.lane_run - 1))) & 1u)) {
#pragma unroll
      for (int j = 0; j < VPL; ++j) key[j] = kNoKey;
    }
  } else if (groups) {
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const int at = VPL <= 8 ? VPL - 1 - static_cast<int>(key[j] & (VPL - 1)) : j;
      const int g = (lane * VPL + at) / p.group_size;
      if (g >= 32 || !((kept >> g) & 1u)) key[j] = kNoKey;
    }
    if (VPL > 1 && VPL <= 8) sort_keys<VPL>(key);  // holes inside a lane
  }
  int pick;
  take_k<BF16, VPL>(p, t, key, lane, biased, err, undecided, pick);
  if (undecided) pick = choose_exact<BF16, VPL>(p, t, lane);  // the same on every lane
  return pick;
}

// Exclusive prefix of counts[0..E) over a CTA of NW warps, into
// pre[0..E] (shared). counts(e) is called once per expert.
template <int NW, typename F>
__device__ __forceinline__ void block_prefix(int E, int* pre, int* part, F counts) {
  constexpr int NT = NW * 32;
  constexpr int PER = kMaxExperts / NT;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  int c[PER], sum = 0;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int e = tid * PER + j;
    c[j] = e < E ? counts(e) : 0;
    sum += c[j];
  }
  int inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(kFull, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) part[warp] = inc;
  __syncthreads();
  int base = 0;
  for (int w = 0; w < warp; ++w) base += part[w];
  int at = base + inc - sum;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int e = tid * PER + j;
    if (e < E) pre[e] = at;
    at += c[j];
    if (e == E - 1) pre[E] = at;
  }
  __syncthreads();
}

// Places of one block's slots: start(e) = first permuted row of this block's slots
// of expert e; mask[e] = the block's tokens that chose e, so a slot's rank is the
// number of lower bits set.
template <int NW, typename F>
__device__ __forceinline__ void place_slots(const TopkParams& p, int64_t blk, const uint32_t* mask, int total,
                                            F start) {
  const int64_t t0 = blk * kTopkBlock;
  const int tokens = static_cast<int>(p.T - t0 < kTopkBlock ? p.T - t0 : kTopkBlock);
  for (int i = threadIdx.x; i < tokens * p.k; i += NW * 32) {
    const int tok = i / p.k;
    const int64_t at = t0 * p.k + i;
    const int e = p.idx[at];
    int pos = -1;
    if (e >= 0) {
      pos = start(e) + __popc(mask[e] & ((1u << tok) - 1u));
      p.perm_token[pos] = static_cast<int32_t>(t0 + tok);
      p.perm_slot[pos] = i - tok * p.k;
      p.gate_perm[pos] = p.weights[at];
    }
    p.slot_pos[at] = pos;
    if (at >= total) {  // behind the last permuted row
      p.perm_token[at] = -1;
      p.perm_slot[at] = -1;
      p.gate_perm[at] = 0.0f;
    }
  }
}

// Routing of one block of kTopkBlock tokens by NW warps: first the choices, a token per
// warp at a time, then the weights of all tokens side by side (as many tokens per warp as
// their choices leave room for). With the dispatch arrays also the block's slots per
// expert; a batch of up to kClusterBlocks blocks runs as one cluster that reads those of
// the other blocks from their shared memory and finishes the dispatch itself. Up to
// a block per SM the tokens of a block run side by side (NW = 32, or 16 where a lane's
// registers allow no more); with more blocks NW = 8, so that more blocks share an SM.
constexpr int kClusterBlocks = 8;

// CTAs per SM that the registers are cut for: NW = 8, us a call, 16384 tokens of 256 experts
// (VPL 8) 39.9 for four and 43.9 for three; 8427 of 308 (VPL 16) 27.5 for three, 34.9 uncut.
__host__ __device__ constexpr int route_ctas(int vpl, int nw) {
  return vpl <= 8 ? 32 / nw : (nw == 8 ? (vpl == 16 ? 3 : 2) : 1);
}

template <bool BF16, int VPL, int NW>
__global__ void __launch_bounds__(NW * 32, route_ctas(VPL, NW))
    moe_topk_route_kernel(const __grid_constant__ TopkParams p) {
  __shared__ uint32_t mask[kMaxExperts];
  __shared__ int pre[kMaxExperts + 1];
  __shared__ int below[kMaxExperts];
  __shared__ int part[NW];
  __shared__ int picks[kTopkBlock][32];
  __shared__ float tops[kTopkBlock], sums[kTopkBlock];
  sm100::launch_dependents();  // the scan may be set up meanwhile
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kTopkBlock;
  const int64_t n = token_count(p);
  const bool dispatch = p.counts != nullptr;
  if (dispatch) {
    for (int e = threadIdx.x; e < p.E; e += NW * 32) mask[e] = 0;
    __syncthreads();
  }
#pragma unroll 1
  for (int i = warp; i < kTopkBlock; i += NW) {
    const int64_t t = t0 + i;
    if (t >= p.T) break;
    int pick = -1;
    if (t < n) {
      float top = 0.0f, z = 1.0f;
      pick = choose<BF16, VPL>(p, t, lane, top, z);
      if (lane == 0) {
        tops[i] = top;
        sums[i] = z;
      }
    } else if (p.scores != nullptr) {
      for (int e = lane; e < p.E; e += 32) p.scores[t * p.E + e] = 0.0f;
    }
    picks[i][lane] = pick;
    if (dispatch && pick >= 0) atomicOr(&mask[pick], 1u << i);
  }
  __syncthreads();
  const int P = p.k <= 1 ? 1 : 1 << (32 - __clz(p.k - 1));  // lanes of a token
  for (int i0 = 0; i0 < kTopkBlock * P; i0 += NW * 32) {
    const int i = i0 + threadIdx.x, tok = i / P, slot = i % P;
    const int64_t t = t0 + tok;
    const bool in = tok < kTopkBlock && t < p.T && slot < p.k;
    const int pick = in ? picks[tok][slot] : -1;
    const float lv = pick >= 0 ? load_logit<BF16>(p.logits, t * p.E + pick) : -INFINITY;
    float w = 0.0f;
    if (p.renorm) w = share_of(p.score, lv, P);
    else if (pick >= 0) w = p.score == MOE_SCORE_SIGMOID ? sigmoid(lv) : expf(lv - tops[tok]) / sums[tok];
    if (in) {
      p.idx[t * p.k + slot] = pick;
      p.weights[t * p.k + slot] = w * p.scale;
    }
  }
  if (blockIdx.x == 0 && threadIdx.x == 0 && p.status != nullptr) *p.status = 0;
  if (!dispatch) return;
  if (p.nblk > kClusterBlocks) {
    for (int e = threadIdx.x; e < p.E; e += NW * 32)
      p.hist[static_cast<int64_t>(blockIdx.x) * p.E + e] = __popc(mask[e]);
    return;
  }
  const int blocks = static_cast<int>(p.nblk), me = blockIdx.x;
  if (blocks > 1) sm100::cluster_sync();  // every block's masks are complete
  else __syncthreads();                   // idx and weights are written
  block_prefix<NW>(p.E, pre, part, [&](int e) {
    int all = 0, lower = 0;
    for (int b = 0; b < blocks; ++b) {
      const int c = __popc(b == me ? mask[e] : static_cast<uint32_t>(sm100::ld_shared_cluster_s32(
                                                   sm100::mapa_shared(&mask[e], b))));
      all += c;
      lower += b < me ? c : 0;
    }
    below[e] = lower;
    if (me == 0) p.counts[e] = all;
    return all;
  });
  if (me == 0)
    for (int e = threadIdx.x; e <= p.E; e += NW * 32) p.offsets[e] = pre[e];
  place_slots<NW>(p, me, mask, pre[p.E], [&](int e) { return pre[e] + below[e]; });
  if (blocks > 1) sm100::cluster_sync();  // no block leaves while another may read its masks
}

// Exclusive prefix over the token blocks of every expert's slots (in place), and the
// totals. A CTA takes 32 experts; thread (y, x) sums one of 32 runs of blocks of
// expert x, the runs are joined through shared memory.
__global__ void __launch_bounds__(1024) moe_topk_scan_kernel(const TopkParams p) {
  __shared__ int run[32][33];
  sm100::launch_dependents();
  sm100::wait_prerequisites();  // the blocks' histograms
  const int x = threadIdx.x % 32, y = threadIdx.x / 32;
  const int e = blockIdx.x * 32 + x;
  const int64_t per = (p.nblk + 31) / 32, b0 = y * per, b1 = b0 + per < p.nblk ? b0 + per : p.nblk;
  int sum = 0;
  if (e < p.E) {
#pragma unroll 8
    for (int64_t b = b0; b < b1; ++b) sum += p.hist[b * p.E + e];
  }
  run[y][x] = sum;
  __syncthreads();
  int at = 0;
  for (int i = 0; i < y; ++i) at += run[i][x];
  if (e < p.E) {
    int64_t b = b0;
    for (; b + 8 <= b1; b += 8) {
      int c[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) c[j] = p.hist[(b + j) * p.E + e];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        p.hist[(b + j) * p.E + e] = at;
        at += c[j];
      }
    }
    for (; b < b1; ++b) {
      const int c = p.hist[b * p.E + e];
      p.hist[b * p.E + e] = at;
      at += c;
    }
    if (y == 31) p.totals[e] = at;
  }
}

constexpr int kDispatchWarps = 8;

// Dispatch of one token block after the scan.
__global__ void __launch_bounds__(kDispatchWarps * 32) moe_topk_dispatch_kernel(const TopkParams p) {
  __shared__ uint32_t mask[kMaxExperts];
  __shared__ int pre[kMaxExperts + 1];
  __shared__ int part[kDispatchWarps];
  const int64_t blk = blockIdx.x;
  for (int e = threadIdx.x; e < p.E; e += kDispatchWarps * 32) mask[e] = 0;
  sm100::wait_prerequisites();  // the scan, which has waited for the routing
  block_prefix<kDispatchWarps>(p.E, pre, part, [&](int e) { return p.totals[e]; });
  const int64_t t0 = blk * kTopkBlock;
  const int tokens = static_cast<int>(p.T - t0 < kTopkBlock ? p.T - t0 : kTopkBlock);
  for (int i = threadIdx.x; i < tokens * p.k; i += kDispatchWarps * 32) {
    const int e = p.idx[t0 * p.k + i];
    if (e >= 0) atomicOr(&mask[e], 1u << (i / p.k));
  }
  __syncthreads();
  if (blk == 0) {
    for (int e = threadIdx.x; e < p.E; e += kDispatchWarps * 32) {
      p.counts[e] = p.totals[e];
      p.offsets[e] = pre[e];
    }
    if (threadIdx.x == 0) p.offsets[p.E] = pre[p.E];
  }
  place_slots<kDispatchWarps>(p, blk, mask, pre[p.E], [&](int e) { return pre[e] + p.hist[blk * p.E + e]; });
}

// ------------------------------------------------------------- backward --
// With p_j = w_j / scale and G the gradient of the scores (0 if none):
//   renormalised:  the weights depend on the chosen logits alone; with
//     d_j = scale * p_j * (g_j - sum_i g_i p_i)   softmax adds d_j to dl[idx_j],
//     sigmoid adds (1 - s) d_j; no division by the scores' sum is needed;
//   else ds[idx_j] += scale * g_j;
//   ds += G;  softmax dl = s (ds - sum ds s), sigmoid dl = s (1 - s) ds.
struct TopkGradParams {
  const void* logits;
  const int32_t* n_tokens;
  const int32_t* idx;
  const float* grad_weights;
  const float* grad_scores;
  void* grad_logits;
  int64_t T;
  int32_t E, k, score, renorm;
  float scale;
  int32_t tokens;  // per warp
};

constexpr int kGradWarps = 8;

// Tokens of a warp at a time, at most: their chosen experts' terms are computed side by side (k
// lanes each) and reach the experts' lanes through rows of shared memory; then each
// token's row in turn. Where a choice names an expert twice, its terms are added one
// after the other in slot order.
__host__ __device__ constexpr int grad_tokens(int vpl) { return vpl <= 8 ? 4 : (vpl == 16 ? 2 : 1); }

// Values of this lane's experts to memory.
template <bool BF16, int VPL>
__device__ __forceinline__ void store_row(void* out, int64_t t, int E, int lane, const float (&d)[VPL]) {
  using T = std::conditional_t<BF16, uint16_t, float>;
  const int e0 = lane * VPL;
  T* at = static_cast<T*>(out) + t * E + e0;
  with_width<VPL, 16 / sizeof(T)>(E, [&](auto width) {
    constexpr int W = decltype(width)::value;
#pragma unroll
    for (int v = 0; v < VPL; v += W) {
      if (e0 + v >= E) continue;
      Pack<T, W> w;
#pragma unroll
      for (int j = 0; j < W; ++j) {
        if constexpr (BF16) w.v[j] = __bfloat16_as_ushort(__float2bfloat16_rn(d[v + j]));
        else w.v[j] = d[v + j];
      }
      *reinterpret_cast<Pack<T, W>*>(at + v) = w;
    }
  });
}

template <bool BF16, int VPL>
__global__ void __launch_bounds__(kGradWarps * 32) moe_topk_grad_kernel(const __grid_constant__ TopkGradParams p) {
  constexpr int TOK = grad_tokens(VPL);
  __shared__ __align__(16) float rows[kGradWarps][TOK][32 * VPL];
  const int lane = threadIdx.x % 32;
  float (&mine)[TOK][32 * VPL] = rows[threadIdx.x / 32];
  const int64_t first = (static_cast<int64_t>(blockIdx.x) * kGradWarps + threadIdx.x / 32) * p.tokens;
  int64_t n = p.T;
  if (p.n_tokens != nullptr) n = min(static_cast<int64_t>(__ldg(p.n_tokens)), p.T);
  for (int i = lane * 4; i < TOK * 32 * VPL; i += 128) *reinterpret_cast<float4*>(&mine[0][0] + i) = make_float4(0, 0, 0, 0);
  __syncwarp();
  // ---- the chosen experts' terms, P lanes to a token
  const int P = p.k <= 1 ? 1 : 1 << (32 - __clz(p.k - 1));
  const int per = 32 / P;  // tokens side by side
  const int slot = lane % P;
#pragma unroll 1
  for (int t0 = 0; t0 < p.tokens; t0 += per) {
    const int tok = t0 + lane / P;
    const int64_t t = first + tok;
    int pick = -1;
    float g = 0.0f, lv = -INFINITY;
    if (tok < p.tokens && t < n && slot < p.k) {
      pick = p.idx[t * p.k + slot];
      if (pick < 0 || pick >= p.E) pick = -1;
    }
    if (pick >= 0) {
      g = p.scale * p.grad_weights[t * p.k + slot];
      lv = load_logit<BF16>(p.logits, t * p.E + pick);
    }
    if (p.renorm) {
      const float share = share_of(p.score, lv, P);
      float mean = pick >= 0 ? g * share : 0.0f;
      for (int o = 1; o < P; o <<= 1) mean += __shfl_xor_sync(kFull, mean, o);
      g = share * (g - mean);  // to the logit itself
      // 1 - s without the cancellation
      if (p.score == MOE_SCORE_SIGMOID) g = pick >= 0 ? g / (1.0f + expf(lv)) : 0.0f;
    }
    const unsigned same = __match_any_sync(kFull, pick >= 0 ? tok * kMaxExperts + pick : -1 - lane);
    if (__all_sync(kFull, (same & (same - 1)) == 0)) {
      if (pick >= 0) mine[tok][pick] = g;
    } else {
      for (int i = 0; i < P; ++i) {
        if (slot == i && pick >= 0) mine[tok][pick] += g;
        __syncwarp();
      }
    }
  }
  __syncwarp();
  // ---- every expert of each token
#pragma unroll 2
  for (int i = 0; i < p.tokens; ++i) {
    const int64_t t = first + i;
    if (t >= p.T) break;
    float d[VPL];
#pragma unroll
    for (int j = 0; j < VPL; ++j) d[j] = 0.0f;
    if (t < n) {
      float l[VPL], c[VPL];
      const LaneExperts own{lane * VPL, p.E};
      load_row<BF16, VPL>(p.logits, t, p.E, p.E, own, l);
      if (p.grad_scores != nullptr) load_bias<VPL>(p.grad_scores + t * p.E, p.E, own, d);
#pragma unroll
      for (int j = 0; j < VPL; ++j) c[j] = mine[i][lane * VPL + j];
      // renormalised weights reach the logits directly, the others through the scores
      if (p.score == MOE_SCORE_SIGMOID) {
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
          // s (1 - s) = e / (1 + e)^2 with e = exp(-|l|)
          const float e = ex2_fast(-kLog2e * fabsf(l[j])), r = rcp_fast(1.0f + e);
          d[j] = p.renorm ? fmaf(d[j], e * r * r, c[j]) : (d[j] + c[j]) * (e * r * r);
        }
      } else {
        float s[VPL], z, top, dot = 0.0f;
        row_scores<VPL>(p.score, l, s, top, z);
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
          if (!p.renorm) d[j] += c[j];
          dot += s[j] > 0.0f ? d[j] * s[j] : 0.0f;
        }
        dot = warp_add(dot);
#pragma unroll
        for (int j = 0; j < VPL; ++j) d[j] = fmaf(s[j], d[j] - dot, p.renorm ? c[j] : 0.0f);
      }
#pragma unroll
      for (int j = 0; j < VPL; ++j)
        if (l[j] == -INFINITY) d[j] = 0.0f;
    }
    store_row<BF16, VPL>(p.grad_logits, t, p.E, lane, d);
  }
}

// Calls f with the registers per lane as a constant: those that `per_lane` experts take.
template <typename F>
cudaError_t with_vpl(int per_lane, F f) {
  if (per_lane <= 1) return f(std::integral_constant<int, 1>{});
  if (per_lane <= 2) return f(std::integral_constant<int, 2>{});
  if (per_lane <= 4) return f(std::integral_constant<int, 4>{});
  if (per_lane <= 8) return f(std::integral_constant<int, 8>{});
  if (per_lane <= 16) return f(std::integral_constant<int, 16>{});
  return f(std::integral_constant<int, 32>{});
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct TopkLayout {
  size_t status, hist, totals, total;
  int64_t nblk;
};

TopkLayout plan_topk(int64_t T, int32_t E) {
  TopkLayout L{};
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  L.nblk = (T + kTopkBlock - 1) / kTopkBlock;
  L.status = 0;
  L.hist = 256;
  L.totals = L.hist + up(sizeof(int32_t) * L.nblk * E);
  L.total = L.nblk > kClusterBlocks ? L.totals + up(sizeof(int32_t) * E) : 0;
  return L;
}

moe_status_t check_topk(const moe_topk_args_t* a, bool routing) {
  if (!a) return MOE_ERR_INVALID_ARG;
  if (a->T < 0 || a->E <= 0 || a->k <= 0 || a->k > a->E) return MOE_ERR_INVALID_ARG;
  if (a->dtype != MOE_F32 && a->dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
  if (a->score != MOE_SCORE_SOFTMAX && a->score != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID_ARG;
  if (a->renormalize != 0 && a->renormalize != 1) return MOE_ERR_INVALID_ARG;
  if (!std::isfinite(a->scale)) return MOE_ERR_INVALID_ARG;
  if (routing) {
    if (a->n_groups < 1 || a->topk_groups < 1 || a->topk_groups > a->n_groups || a->E % a->n_groups != 0)
      return MOE_ERR_INVALID_ARG;
    if (a->group_rule != MOE_GROUP_MAX && a->group_rule != MOE_GROUP_TOP2_SUM) return MOE_ERR_INVALID_ARG;
    if (a->n_groups > 32) return MOE_ERR_UNSUPPORTED;
  }
  if (a->E > kMaxExperts || a->k > 32 || a->T > (int64_t(1) << 24)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_topk_workspace_size(int64_t T, int32_t E, int32_t k) {
  if (T <= 0 || E <= 0 || k <= 0 || k > E || E > kMaxExperts || k > 32 || T > (int64_t(1) << 24)) return 0;
  return plan_topk(T, E).total;
}

moe_status_t moe_topk_route(const moe_topk_args_t* a, const moe_topk_routed_t* r, void* workspace, size_t ws_bytes,
                            moe_stream_t stream) {
  const moe_status_t st = check_topk(a, true);
  if (st != MOE_OK) return st;
  if (!r) return MOE_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a->T == 0) {  // nothing routed: no launch, but the counts are those of an empty batch
    if (r->counts && cudaMemsetAsync(r->counts, 0, sizeof(int32_t) * a->E, s) != cudaSuccess) return MOE_ERR_CUDA;
    if (r->offsets && cudaMemsetAsync(r->offsets, 0, sizeof(int32_t) * (a->E + 1), s) != cudaSuccess)
      return MOE_ERR_CUDA;
    return MOE_OK;
  }
  void* const disp[6] = {r->counts, r->offsets, r->perm_token, r->perm_slot, r->slot_pos, r->gate_perm};
  int given = 0;
  for (void* q : disp) given += q != nullptr;
  if (given != 0 && given != 6) return MOE_ERR_INVALID_ARG;
  const bool dispatch = given == 6;
  for (void* q : disp)
    if (!aligned16(q)) return MOE_ERR_MISALIGNED;
  if (!a->logits || !r->idx || !r->weights) return MOE_ERR_INVALID_ARG;
  if (!aligned16(a->logits) || !aligned16(a->bias) || !aligned16(r->idx) || !aligned16(r->weights) ||
      !aligned16(r->scores) || (reinterpret_cast<uintptr_t>(a->n_tokens) & 3u) != 0)
    return MOE_ERR_MISALIGNED;
  const TopkLayout L = plan_topk(a->T, a->E);
  const bool ws = dispatch && L.nblk > kClusterBlocks;
  if (ws && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 || ws_bytes < L.total))
    return MOE_ERR_WORKSPACE;
  TopkParams p{};
  p.logits = a->logits;
  p.bias = a->bias;
  p.n_tokens = a->n_tokens;
  p.T = a->T;
  p.E = a->E;
  p.k = a->k;
  p.n_groups = a->n_groups;
  p.topk_groups = a->topk_groups;
  p.group_size = a->E / a->n_groups;
  p.score = a->score;
  p.rule = a->group_rule;
  p.renorm = a->renormalize;
  p.scale = a->scale;
  p.idx = r->idx;
  p.weights = r->weights;
  p.scores = r->scores;
  p.counts = r->counts;
  p.offsets = r->offsets;
  p.perm_token = r->perm_token;
  p.perm_slot = r->perm_slot;
  p.slot_pos = r->slot_pos;
  p.gate_perm = r->gate_perm;
  p.nblk = L.nblk;
  if (ws) {
    p.hist = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + L.hist);
    p.totals = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + L.totals);
  }
  if (workspace && (reinterpret_cast<uintptr_t>(workspace) & 255u) == 0 && ws_bytes >= sizeof(uint32_t))
    p.status = static_cast<uint32_t*>(workspace);
  const unsigned grid = static_cast<unsigned>(L.nblk);
  const bool few = L.nblk <= device_sm_count();
  const bool cluster = dispatch && L.nblk > 1 && L.nblk <= kClusterBlocks;
  // Lanes of a group: 32 over the number of groups, rounded to a power of two. A group count
  // that is none can need more registers than the largest kernel has; then groups lie
  // across lanes.
  int per_lane = (a->E + 31) / 32;
  if (a->n_groups > 1) {
    int run = 32, shift = 5;
    while (run > 1 && run * a->n_groups > 32) {
      run /= 2;
      --shift;
    }
    if ((p.group_size + run - 1) / run <= 32) {
      per_lane = (p.group_size + run - 1) / run;
      p.lane_run = run;
      p.run_shift = shift;
    }
  }
  const cudaError_t e = with_vpl(per_lane, [&](auto v) {
    constexpr int VPL = decltype(v)::value;
    constexpr int WIDE = VPL <= 8 ? 32 : 16;
    const unsigned threads = few ? WIDE * 32 : 8 * 32, blocks = cluster ? grid : 1;
    if (a->dtype == MOE_BF16)
      return few ? launch_kernel(moe_topk_route_kernel<true, VPL, WIDE>, grid, threads, 0, s, blocks, false, p)
                 : launch_kernel(moe_topk_route_kernel<true, VPL, 8>, grid, threads, 0, s, blocks, false, p);
    return few ? launch_kernel(moe_topk_route_kernel<false, VPL, WIDE>, grid, threads, 0, s, blocks, false, p)
               : launch_kernel(moe_topk_route_kernel<false, VPL, 8>, grid, threads, 0, s, blocks, false, p);
  });
  if (e != cudaSuccess) return MOE_ERR_CUDA;
  if (ws) {
    if (launch_kernel(moe_topk_scan_kernel, (a->E + 31) / 32, 1024, 0, s, 1, true, p) != cudaSuccess ||
        launch_kernel(moe_topk_dispatch_kernel, grid, kDispatchWarps * 32, 0, s, 1, true, p) != cudaSuccess)
      return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

moe_status_t moe_topk_route_backward(const moe_topk_args_t* a, const int32_t* idx, const float* grad_weights,
                                     const float* grad_scores, void* grad_logits, moe_stream_t stream) {
  const moe_status_t st = check_topk(a, false);
  if (st != MOE_OK || a->T == 0) return st;
  if (!a->logits || !idx || !grad_weights || !grad_logits) return MOE_ERR_INVALID_ARG;
  if (!aligned16(a->logits) || !aligned16(idx) || !aligned16(grad_weights) || !aligned16(grad_scores) ||
      !aligned16(grad_logits) || (reinterpret_cast<uintptr_t>(a->n_tokens) & 3u) != 0)
    return MOE_ERR_MISALIGNED;
  TopkGradParams p{a->logits, a->n_tokens, idx, grad_weights, grad_scores, grad_logits, a->T, a->E,
                   a->k,      a->score,    a->renormalize, a->scale,     1};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = with_vpl((a->E + 31) / 32, [&](auto v) {
    constexpr int VPL = decltype(v)::value;
    // one token per warp while that leaves SMs with less than two CTAs (4096 tokens of 8
    // experts: 4.6 us with one, 6.3 with four; 16384 of 256: 14.1 and 13.3)
    p.tokens = a->T >= 2 * kGradWarps * grad_tokens(VPL) * static_cast<int64_t>(device_sm_count()) ? grad_tokens(VPL) : 1;
    const int64_t per = kGradWarps * p.tokens;
    const unsigned grid = static_cast<unsigned>((a->T + per - 1) / per);
    if (a->dtype == MOE_BF16) moe_topk_grad_kernel<true, VPL><<<grid, kGradWarps * 32, 0, s>>>(p);
    else moe_topk_grad_kernel<false, VPL><<<grid, kGradWarps * 32, 0, s>>>(p);
    return cudaGetLastError();
  });
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
