// route_topk.cu — routing of any number of experts and choices per token
// (moe_topk_route), its backward pass and the dispatch of its choice.
//
// One warp takes one token. Lane L holds the logits of the experts L * VPL ..
// L * VPL + VPL - 1 (VPL = E / 32 rounded up to a power of two), so that a group of
// experts is a run of lanes and "the lower expert" is the lower lane, then the
// lower register. The k choices are k rounds of a warp maximum.
//
// The choice is that of the 64-bit values. Without a bias the rank value is the
// logit itself and every comparison is exact. With one it is score + bias, whose
// fp32 value is off by at most `err` (derived at rank_error); a round whose winner
// is less than 2 err ahead of the next value, or a group limit that close, is
// undecided, and that token is chosen again from 64-bit values. With normal logits
// that is about one token in five hundred, so the 64-bit pass costs nothing next
// to evaluating every score in it.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdint>

#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int kTopkWarps = 16;      // warps of a routing CTA
constexpr int kTopkBlock = 32;      // tokens of a routing CTA: one bit each of a 32-bit mask per expert
constexpr int kMaxExperts = 1024;
constexpr unsigned kFull = 0xffffffffu;

struct TopkParams {
  const void* logits;
  const float* bias;
  const int32_t* n_tokens;
  int64_t T;
  int32_t E, k, n_groups, topk_groups, group_size, score, rule, renorm;
  float scale;
  int32_t* idx;
  float* weights;
  float* scores;
  // dispatch (counts == nullptr: none)
  int32_t* counts;
  int32_t* offsets;
  int32_t* perm_token;
  int32_t* perm_slot;
  int32_t* slot_pos;
  float* gate_perm;
  int32_t* hist;    // [nblk, E] slots per token block, then their exclusive prefix over blocks
  int32_t* totals;  // [E]
  int64_t nblk;
  uint32_t* status; // workspace status word: nothing here can fail, so it is set to 0
};

__device__ __forceinline__ int64_t token_count(const TopkParams& p) {
  if (p.n_tokens == nullptr) return p.T;
  const int64_t n = __ldg(p.n_tokens);
  return n < 0 ? 0 : (n < p.T ? n : p.T);
}

// fp32 value of a logit as the routing sees it: NaN masks, +inf is the largest.
__device__ __forceinline__ float clean(float l) { return l != l ? -INFINITY : fminf(l, FLT_MAX); }

template <bool BF16>
__device__ __forceinline__ float load_logit(const void* logits, int64_t at) {
  if (BF16) return clean(__bfloat162float(static_cast<const __nv_bfloat16*>(logits)[at]));
  return clean(static_cast<const float*>(logits)[at]);
}

// Logits of this lane's experts; -inf past the last one. Rows whose start and
// length are whole vectors load 16 bytes at a time.
template <bool BF16, int VPL>
__device__ __forceinline__ void load_row(const void* logits, int64_t t, int E, int lane, float (&l)[VPL]) {
  const int64_t row = t * E;
  const int e0 = lane * VPL;
  constexpr int PER = BF16 ? 8 : 4;
  if (VPL >= PER && E % PER == 0) {
#pragma unroll
    for (int v = 0; v < (VPL >= PER ? VPL / PER : 0); ++v) {
      const int e = e0 + v * PER;
      if (e < E) {
        if (BF16) {
          const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(logits) + row + e);
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            l[(v * PER + 2 * j) % VPL] = clean(__uint_as_float(w[j] << 16));
            l[(v * PER + 2 * j + 1) % VPL] = clean(__uint_as_float(w[j] & 0xFFFF0000u));
          }
        } else {
          const float4 f = *reinterpret_cast<const float4*>(static_cast<const float*>(logits) + row + e);
          const float w[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) l[(v * PER + j) % VPL] = clean(w[j]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < PER; ++j) l[(v * PER + j) % VPL] = -INFINITY;
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < VPL; ++j) l[j] = e0 + j < E ? load_logit<BF16>(logits, row + e0 + j) : -INFINITY;
  }
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
  return v;
}
__device__ __forceinline__ double warp_max(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmax(v, __shfl_xor_sync(kFull, v, o));
  return v;
}
template <typename V>
__device__ __forceinline__ V warp_min(V v) {
  return -warp_max(-v);
}
template <typename V>
__device__ __forceinline__ V warp_add(V v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

__device__ __forceinline__ float exp_of(float x) { return expf(x); }
__device__ __forceinline__ double exp_of(double x) { return exp(x); }

template <typename V>
__device__ __forceinline__ V sigmoid(V l) {
  return V(1) / (V(1) + exp_of(-l));
}

template <typename V>
__device__ __forceinline__ V lowest() {
  return static_cast<V>(-INFINITY);
}

// Order-preserving map of floats to unsigned: one redux instruction finds a warp's
// maximum. -0 and +0 are made one first, so that they tie.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// The warp's largest value and the lowest lane that holds it.
__device__ __forceinline__ float warp_best(float v, int& src) {
  const uint32_t key = order_key(v), m = __reduce_max_sync(kFull, key);
  src = __ffs(__ballot_sync(kFull, key == m)) - 1;
  return key_value(m);
}
__device__ __forceinline__ double warp_best(double v, int& src) {
  const double m = warp_max(v);
  src = __ffs(__ballot_sync(kFull, v == m)) - 1;
  return m;
}

// Two largest values of a set, held as (a >= b).
template <typename V>
__device__ __forceinline__ void push2(V& a, V& b, V v) {
  if (v > a) {
    b = a;
    a = v;
  } else if (v > b) {
    b = v;
  }
}

// Mask of the groups that stay. `err`: what a value may be off by (0 = exact);
// undecided is set when two groups on either side of the limit are closer than
// their errors allow to tell apart. rank: the values the choice goes by;
// value: score + bias (the sum rule's terms).
template <typename V, int VPL>
__device__ __forceinline__ unsigned kept_groups(const TopkParams& p, int lane, const V (&rank)[VPL],
                                                const V (&value)[VPL], V err, bool& undecided) {
  const int gs = p.group_size, G = p.n_groups;
  const bool sum = p.rule == MOE_GROUP_TOP2_SUM;
  V mine = lowest<V>();  // lane g: value of group g
  const int run = gs / VPL;
  if (gs % VPL == 0 && (run & (run - 1)) == 0) {
    // a group is `run` whole lanes, a power of two: reduce within the run
    V a = lowest<V>(), b = lowest<V>();
#pragma unroll
    for (int j = 0; j < VPL; ++j) push2(a, b, rank[j] == lowest<V>() ? lowest<V>() : (sum ? value[j] : rank[j]));
    for (int o = 1; o < run; o <<= 1) {
      const V a2 = __shfl_xor_sync(kFull, a, o), b2 = __shfl_xor_sync(kFull, b, o);
      push2(a, b, a2);
      push2(a, b, b2);
    }
    const V gv = sum && b != lowest<V>() ? a + b : a;
    const V got = __shfl_sync(kFull, gv, (lane * run) & 31);
    if (lane < G) mine = got;
  } else {
    for (int g = 0; g < G; ++g) {
      V a = lowest<V>(), b = lowest<V>();
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        const int e = lane * VPL + j;
        if (e / gs == g && rank[j] != lowest<V>()) push2(a, b, sum ? value[j] : rank[j]);
      }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const V a2 = __shfl_xor_sync(kFull, a, o), b2 = __shfl_xor_sync(kFull, b, o);
        push2(a, b, a2);
        push2(a, b, b2);
      }
      if (lane == g) mine = sum && b != lowest<V>() ? a + b : a;
    }
  }
  int before = 0;  // groups ahead of this one
  for (int g = 0; g < G; ++g) {
    const V o = __shfl_sync(kFull, mine, g);
    before += (o > mine || (o == mine && g < lane)) ? 1 : 0;
  }
  const bool keep = lane < G && before < p.topk_groups;
  const unsigned mask = __ballot_sync(kFull, keep);
  if (err > V(0) && p.topk_groups < G) {
    const V low = warp_min(keep ? mine : static_cast<V>(INFINITY));
    const V high = warp_max(lane < G && !keep ? mine : lowest<V>());
    // two values of `err` each in a sum, on both sides; empty groups are exact
    if (high > lowest<V>() && !(low - high > V(4) * err)) undecided = true;
  }
  return mask;
}

// k rounds of the warp's largest rank value, dropped as they are taken. Lane i
// ends with the i-th choice in `pick` (-1: none left). With err > 0 one more
// round looks at the value behind the last, and `undecided` is set when two
// neighbours are closer than 2 err.
template <typename V, int VPL>
__device__ __forceinline__ void take_k(V (&rank)[VPL], int k, int lane, V err, bool& undecided, int& pick) {
  pick = -1;
  V best = lowest<V>();
  int at = 0;
#pragma unroll
  for (int j = 0; j < VPL; ++j)
    if (rank[j] > best) {
      best = rank[j];
      at = j;
    }
  V last = static_cast<V>(INFINITY);
  const int rounds = err > V(0) ? k + 1 : k;
  for (int i = 0; i < rounds; ++i) {
    int src;
    const V m = warp_best(best, src);
    if (m == lowest<V>()) break;
    if (err > V(0) && i > 0 && !(last - m > V(2) * err)) undecided = true;
    last = m;
    if (i == k) break;
    const int e = __shfl_sync(kFull, lane * VPL + at, src);
    if (lane == i) pick = e;
    if (lane == src) {
      best = lowest<V>();
      int next = 0;
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        if (j == at) rank[j] = lowest<V>();
        if (rank[j] > best) {
          best = rank[j];
          next = j;
        }
      }
      at = next;
    }
  }
}

// Scores of this lane's experts, the row's largest logit and, for softmax, the sum.
template <typename V, int VPL>
__device__ __forceinline__ void row_scores(int score, const float (&l)[VPL], V (&s)[VPL], float& top, V& z) {
  top = -INFINITY;
  z = V(1);
  if (score == MOE_SCORE_SIGMOID) {
#pragma unroll
    for (int j = 0; j < VPL; ++j) s[j] = l[j] == -INFINITY ? V(0) : sigmoid(static_cast<V>(l[j]));
    return;
  }
#pragma unroll
  for (int j = 0; j < VPL; ++j) top = fmaxf(top, l[j]);
  top = warp_max(top);
  V sum = V(0);
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    s[j] = l[j] == -INFINITY ? V(0) : exp_of(static_cast<V>(l[j]) - static_cast<V>(top));
    sum += s[j];
  }
  z = warp_add(sum);
  if (!(z > V(0))) z = V(1);
#pragma unroll
  for (int j = 0; j < VPL; ++j) s[j] /= z;
}

// What an fp32 score + bias may be off by from its 64-bit value, with u = 2^-24.
// Sigmoid: expf is within 2 u of relative error, the sum and the division add u each,
// and d s / d(e^-l) shrinks the first: at most 5 u s <= 3e-7. Softmax: the difference
// l - max is rounded (|l - max| u in the exponent, at most 0.37 u next to the largest
// term once multiplied by e^(l - max)), expf 2 u, and the sum of E <= 1024 terms in 32
// rounds and 5 levels 37 u more, the division u: at most 45 u s <= 2.7e-6 s. The
// addition of the bias: u |s + b|.
__device__ __forceinline__ float rank_error(int score, float s_top, float c_top) {
  return (score == MOE_SCORE_SIGMOID ? 3.6e-7f : 3.0e-6f) * s_top + 1.2e-7f * c_top;
}

template <bool BF16, int VPL, typename V>
__device__ __forceinline__ void rank_values(const TopkParams& p, int lane, const float (&l)[VPL], const V (&s)[VPL],
                                            V (&rank)[VPL], V (&value)[VPL]) {
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const int e = lane * VPL + j;
    value[j] = s[j];
    rank[j] = static_cast<V>(l[j]);
    if (p.bias != nullptr && e < p.E) {
      value[j] = s[j] + static_cast<V>(__ldg(p.bias + e));
      rank[j] = l[j] == -INFINITY || value[j] != value[j] ? lowest<V>() : value[j];
    }
  }
}

template <typename V, int VPL>
__device__ __forceinline__ void choose(const TopkParams& p, int lane, V (&rank)[VPL], const V (&value)[VPL],
                                       V group_err, V err, bool& undecided, int& pick) {
  if (p.n_groups > 1) {
    const unsigned kept = kept_groups<V, VPL>(p, lane, rank, value, group_err, undecided);
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const int g = (lane * VPL + j) / p.group_size;
      if (g >= 32 || !((kept >> g) & 1u)) rank[j] = lowest<V>();
    }
  }
  take_k<V, VPL>(rank, p.k, lane, err, undecided, pick);
}

// The choice from 64-bit values. A call of its own: its registers are not those
// of the common path.
template <bool BF16, int VPL>
__device__ __noinline__ int choose_exact(const TopkParams& p, int64_t t, int lane) {
  float l[VPL];
  load_row<BF16, VPL>(p.logits, t, p.E, lane, l);
  double s[VPL], rank[VPL], value[VPL], z;
  float top;
  row_scores<double, VPL>(p.score, l, s, top, z);
  rank_values<BF16, VPL, double>(p, lane, l, s, rank, value);
  bool undecided = false;
  int pick;
  choose<double, VPL>(p, lane, rank, value, 0.0, 0.0, undecided, pick);
  return pick;
}

// Share of each choice in the renormalised weights (lanes 0 .. k-1 hold one choice
// with logit lv, -inf = none): s / sum s, computed from differences of logits, so
// that scores below the fp32 range still share. Sigmoid scores of logits below -60
// are exp(l) to 26 digits.
__device__ __forceinline__ float share_of(int score, float lv, bool has) {
  const float top = warp_max(has ? lv : -INFINITY);
  float x = 0.0f;
  if (has && lv > -INFINITY) x = score == MOE_SCORE_SIGMOID && top > -60.0f ? sigmoid(lv) : expf(lv - top);
  const float sum = warp_add(x);
  return sum > 0.0f ? x / sum : 0.0f;
}

// One token by one warp: idx, weights, scores. Lane i < k ends with choice i and
// its weight.
template <bool BF16, int VPL>
__device__ __forceinline__ void route_token(const TopkParams& p, int64_t t, int lane, bool real, int& pick,
                                            float& weight) {
  pick = -1;
  weight = 0.0f;
  if (!real) {
    if (p.scores != nullptr)
      for (int e = lane; e < p.E; e += 32) p.scores[t * p.E + e] = 0.0f;
  } else {
    float l[VPL], s[VPL], z = 1.0f, top = 0.0f;
    load_row<BF16, VPL>(p.logits, t, p.E, lane, l);
    const bool sums = p.n_groups > 1 && p.rule == MOE_GROUP_TOP2_SUM;
    const bool need_all = p.bias != nullptr || p.scores != nullptr || sums ||
                          (p.score == MOE_SCORE_SOFTMAX && p.renorm == 0);
    if (need_all) {
      row_scores<float, VPL>(p.score, l, s, top, z);
    } else {
#pragma unroll
      for (int j = 0; j < VPL; ++j) s[j] = 0.0f;
    }
    if (p.scores != nullptr) {
#pragma unroll
      for (int j = 0; j < VPL; ++j)
        if (lane * VPL + j < p.E) p.scores[t * p.E + lane * VPL + j] = s[j];
    }
    float rank[VPL], value[VPL];
    rank_values<BF16, VPL, float>(p, lane, l, s, rank, value);
    float err = 0.0f;
    if (p.bias != nullptr || sums) {
      float st = 0.0f, ct = 0.0f;
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        st = fmaxf(st, s[j]);
        ct = fmaxf(ct, rank[j] == -INFINITY ? 0.0f : fabsf(value[j]));
      }
      err = fmaxf(rank_error(p.score, warp_max(st), warp_max(ct)), FLT_MIN);
    }
    bool undecided = false;
    choose<float, VPL>(p, lane, rank, value, err, p.bias != nullptr ? err : 0.0f, undecided, pick);
    if (undecided) pick = choose_exact<BF16, VPL>(p, t, lane);  // the same on every lane
    const bool has = pick >= 0;
    const float lv = has ? load_logit<BF16>(p.logits, t * p.E + pick) : -INFINITY;
    if (p.renorm) {
      weight = share_of(p.score, lv, has);
    } else if (has) {
      weight = p.score == MOE_SCORE_SIGMOID ? sigmoid(lv) : expf(lv - top) / z;
    }
    weight *= p.scale;
  }
  if (lane < p.k) {
    p.idx[t * p.k + lane] = pick;
    p.weights[t * p.k + lane] = weight;
  }
}

// Exclusive prefix of counts[0..E) over a CTA of kTopkWarps * 32 threads, into
// pre[0..E] (shared). counts(e) is called once per expert.
template <typename F>
__device__ __forceinline__ void block_prefix(int E, int* pre, int* part, F counts) {
  constexpr int NT = kTopkWarps * 32;
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
template <typename F>
__device__ __forceinline__ void place_slots(const TopkParams& p, int64_t blk, const uint32_t* mask, int total,
                                            F start) {
  const int64_t t0 = blk * kTopkBlock;
  const int tokens = static_cast<int>(p.T - t0 < kTopkBlock ? p.T - t0 : kTopkBlock);
  for (int i = threadIdx.x; i < tokens * p.k; i += kTopkWarps * 32) {
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

// Routing of one block of kTopkBlock tokens, two per warp; with the dispatch arrays
// also the block's slots per expert. A batch of one block is dispatched here too.
template <bool BF16, int VPL>
__global__ void __launch_bounds__(kTopkWarps * 32) moe_topk_route_kernel(const __grid_constant__ TopkParams p) {
  __shared__ uint32_t mask[kMaxExperts];
  __shared__ int pre[kMaxExperts + 1];
  __shared__ int part[kTopkWarps];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kTopkBlock;
  const int64_t n = token_count(p);
  const bool dispatch = p.counts != nullptr;
  if (dispatch) {
    for (int e = threadIdx.x; e < p.E; e += kTopkWarps * 32) mask[e] = 0;
    __syncthreads();
  }
#pragma unroll 1
  for (int i = warp; i < kTopkBlock; i += kTopkWarps) {
    const int64_t t = t0 + i;
    if (t >= p.T) break;
    int pick;
    float weight;
    route_token<BF16, VPL>(p, t, lane, t < n, pick, weight);
    if (dispatch && pick >= 0) atomicOr(&mask[pick], 1u << i);
  }
  if (!dispatch) return;
  __syncthreads();
  if (p.nblk > 1) {
    for (int e = threadIdx.x; e < p.E; e += kTopkWarps * 32)
      p.hist[static_cast<int64_t>(blockIdx.x) * p.E + e] = __popc(mask[e]);
    return;
  }
  block_prefix(p.E, pre, part, [&](int e) { return __popc(mask[e]); });
  for (int e = threadIdx.x; e < p.E; e += kTopkWarps * 32) {
    p.counts[e] = __popc(mask[e]);
    p.offsets[e] = pre[e];
  }
  if (threadIdx.x == 0) p.offsets[p.E] = pre[p.E];
  place_slots(p, 0, mask, pre[p.E], [&](int e) { return pre[e]; });
}

// Exclusive prefix over the token blocks of every expert's slots (in place), and the
// totals. A CTA takes 32 experts; thread (y, x) sums one of 32 runs of blocks of
// expert x, the runs are joined through shared memory.
__global__ void __launch_bounds__(1024) moe_topk_scan_kernel(const TopkParams p) {
  __shared__ int run[32][33];
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0;
  const int x = threadIdx.x % 32, y = threadIdx.x / 32;
  const int e = blockIdx.x * 32 + x;
  const int64_t per = (p.nblk + 31) / 32, b0 = y * per, b1 = b0 + per < p.nblk ? b0 + per : p.nblk;
  int sum = 0;
  if (e < p.E)
    for (int64_t b = b0; b < b1; ++b) sum += p.hist[b * p.E + e];
  run[y][x] = sum;
  __syncthreads();
  int at = 0;
  for (int i = 0; i < y; ++i) at += run[i][x];
  if (e < p.E) {
    for (int64_t b = b0; b < b1; ++b) {
      const int c = p.hist[b * p.E + e];
      p.hist[b * p.E + e] = at;
      at += c;
    }
    if (y == 31) p.totals[e] = at;
  }
}

// Dispatch of one token block after the scan.
__global__ void __launch_bounds__(kTopkWarps * 32) moe_topk_dispatch_kernel(const TopkParams p) {
  __shared__ uint32_t mask[kMaxExperts];
  __shared__ int pre[kMaxExperts + 1];
  __shared__ int part[kTopkWarps];
  const int64_t blk = blockIdx.x;
  for (int e = threadIdx.x; e < p.E; e += kTopkWarps * 32) mask[e] = 0;
  block_prefix(p.E, pre, part, [&](int e) { return p.totals[e]; });
  const int64_t t0 = blk * kTopkBlock;
  const int tokens = static_cast<int>(p.T - t0 < kTopkBlock ? p.T - t0 : kTopkBlock);
  for (int i = threadIdx.x; i < tokens * p.k; i += kTopkWarps * 32) {
    const int e = p.idx[t0 * p.k + i];
    if (e >= 0) atomicOr(&mask[e], 1u << (i / p.k));
  }
  __syncthreads();
  if (blk == 0) {
    for (int e = threadIdx.x; e < p.E; e += kTopkWarps * 32) {
      p.counts[e] = p.totals[e];
      p.offsets[e] = pre[e];
    }
    if (threadIdx.x == 0) p.offsets[p.E] = pre[p.E];
  }
  place_slots(p, blk, mask, pre[p.E], [&](int e) { return pre[e] + p.hist[blk * p.E + e]; });
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
};

template <bool BF16, int VPL>
__global__ void __launch_bounds__(256) moe_topk_grad_kernel(const __grid_constant__ TopkGradParams p) {
  const int lane = threadIdx.x % 32;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 8 + threadIdx.x / 32;
  if (t >= p.T) return;
  int64_t n = p.T;
  if (p.n_tokens != nullptr) n = __ldg(p.n_tokens);
  float d[VPL];
#pragma unroll
  for (int j = 0; j < VPL; ++j) d[j] = 0.0f;
  if (t < n) {
    float l[VPL], s[VPL], z, top;
    load_row<BF16, VPL>(p.logits, t, p.E, lane, l);
    row_scores<float, VPL>(p.score, l, s, top, z);
    int pick = -1;
    float g = 0.0f, lv = -INFINITY;
    if (lane < p.k) {
      pick = p.idx[t * p.k + lane];
      if (pick < 0 || pick >= p.E) pick = -1;
    }
    if (pick >= 0) {
      g = p.scale * p.grad_weights[t * p.k + lane];
      lv = load_logit<BF16>(p.logits, t * p.E + pick);
    }
    if (p.renorm) {
      const float share = share_of(p.score, lv, pick >= 0);
      const float mean = warp_add(pick >= 0 ? g * share : 0.0f);
      g = share * (g - mean);  // to the logit itself
      // 1 - s without the cancellation
      if (p.score == MOE_SCORE_SIGMOID) g = pick >= 0 ? g / (1.0f + expf(lv)) : 0.0f;
    }
    float direct[VPL];
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const int e = lane * VPL + j;
      direct[j] = 0.0f;
      d[j] = p.grad_scores != nullptr && e < p.E ? p.grad_scores[t * p.E + e] : 0.0f;
    }
    for (int i = 0; i < p.k; ++i) {
      const int e = __shfl_sync(kFull, pick, i);
      const float v = __shfl_sync(kFull, g, i);
      const int j0 = e - lane * VPL;  // outside [0, VPL): another lane's, or none
#pragma unroll
      for (int j = 0; j < VPL; ++j)
        if (e >= 0 && j == j0) {
          if (p.renorm) direct[j] += v;
          else d[j] += v;
        }
    }
    if (p.score == MOE_SCORE_SIGMOID) {
#pragma unroll
      for (int j = 0; j < VPL; ++j) d[j] = d[j] * s[j] / (1.0f + expf(l[j])) + direct[j];
    } else {
      float dot = 0.0f;
#pragma unroll
      for (int j = 0; j < VPL; ++j) dot += s[j] > 0.0f ? d[j] * s[j] : 0.0f;
      dot = warp_add(dot);
#pragma unroll
      for (int j = 0; j < VPL; ++j) d[j] = s[j] * (d[j] - dot) + direct[j];
    }
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (l[j] == -INFINITY) d[j] = 0.0f;
  }
  const int64_t row = t * p.E;
  const int e0 = lane * VPL;
  constexpr int PER = BF16 ? 8 : 4;
  if (VPL >= PER && p.E % PER == 0) {
#pragma unroll
    for (int v = 0; v < (VPL >= PER ? VPL / PER : 0); ++v) {
      if (e0 + v * PER >= p.E) continue;
      if (BF16) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const __nv_bfloat162 b = __floats2bfloat162_rn(d[(v * PER + 2 * j) % VPL], d[(v * PER + 2 * j + 1) % VPL]);
          w[j] = *reinterpret_cast<const uint32_t*>(&b);
        }
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.grad_logits) + row + e0 + v * PER) =
            make_uint4(w[0], w[1], w[2], w[3]);
      } else {
        *reinterpret_cast<float4*>(static_cast<float*>(p.grad_logits) + row + e0 + v * PER) =
            make_float4(d[(v * PER) % VPL], d[(v * PER + 1) % VPL], d[(v * PER + 2) % VPL], d[(v * PER + 3) % VPL]);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      if (e0 + j >= p.E) continue;
      if (BF16) static_cast<__nv_bfloat16*>(p.grad_logits)[row + e0 + j] = __float2bfloat16_rn(d[j]);
      else static_cast<float*>(p.grad_logits)[row + e0 + j] = d[j];
    }
  }
}

// Calls f with the registers per lane for E experts as a constant.
template <typename F>
cudaError_t with_vpl(int E, F f) {
  if (E <= 32) return f(std::integral_constant<int, 1>{});
  if (E <= 64) return f(std::integral_constant<int, 2>{});
  if (E <= 128) return f(std::integral_constant<int, 4>{});
  if (E <= 256) return f(std::integral_constant<int, 8>{});
  if (E <= 512) return f(std::integral_constant<int, 16>{});
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
  L.total = L.nblk > 1 ? L.totals + up(sizeof(int32_t) * E) : 0;
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
  const bool ws = dispatch && L.nblk > 1;
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
    p.status = static_cast<uint32_t*>(workspace);
  }
  const unsigned grid = static_cast<unsigned>(L.nblk);
  const cudaError_t e = with_vpl(a->E, [&](auto v) {
    constexpr int VPL = decltype(v)::value;
    if (a->dtype == MOE_BF16) moe_topk_route_kernel<true, VPL><<<grid, kTopkWarps * 32, 0, s>>>(p);
    else moe_topk_route_kernel<false, VPL><<<grid, kTopkWarps * 32, 0, s>>>(p);
    return cudaGetLastError();
  });
  if (e != cudaSuccess) return MOE_ERR_CUDA;
  if (ws) {
    moe_topk_scan_kernel<<<(a->E + 31) / 32, 1024, 0, s>>>(p);
    if (cudaGetLastError() != cudaSuccess) return MOE_ERR_CUDA;
    moe_topk_dispatch_kernel<<<grid, kTopkWarps * 32, 0, s>>>(p);
    if (cudaGetLastError() != cudaSuccess) return MOE_ERR_CUDA;
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
                   a->k,      a->score,    a->renormalize, a->scale};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const unsigned grid = static_cast<unsigned>((a->T + 7) / 8);
  const cudaError_t e = with_vpl(a->E, [&](auto v) {
    constexpr int VPL = decltype(v)::value;
    if (a->dtype == MOE_BF16) moe_topk_grad_kernel<true, VPL><<<grid, 256, 0, s>>>(p);
    else moe_topk_grad_kernel<false, VPL><<<grid, 256, 0, s>>>(p);
    return cudaGetLastError();
  });
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
