// gemm_int8.cu — products of rows and int8 weights in 8-bit integers with a scale
// per row and per output channel (moe_int8_product), rows grouped by expert.
//
//   y[r, n] = gate[r] * a[r] * s[e, n] * sum_k q[r, k] * w[e, k, n]
//   gated pair: y = gate * act(z_w) * z_w_up, both products in one kernel
//
// The sums run on the 5th-generation tensor cores as kind::i8 (signed 8-bit operands,
// 32-bit integer sums, exact for K < 2^17), at twice the 16-bit rate and on half the
// bytes of the 16-bit forms. The weights are read in the caller's [E, K, N] layout as
// the MN-major operand (one TMA box = 128 K rows of 128 columns, 128-B swizzle), the
// rows as the K-major one.
//
// Launches: a prepare kernel (row scales and quantised rows, tile schedule), then one
// of three product kernels (stream, split, pair form; which one: int8_plan.cuh).
// At the Grok-1 shape with 8 experts: 128 rows, gate/up and down 6.26 and 6.3 TB/s of
// weights (96 % of the measured copy rate); 8192 rows 3020 and 2900 TOP/s in short runs, 2617
// and 2276 over seconds under the 1000 W cap, quantisation included.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "gemm_common.cuh"
#include "int8_plan.cuh"

namespace moe {
namespace i8 {

using namespace moe::sm100;
using tc::kWaitLimitNs;
using tc::pack_bf16x2;
using tc::warp_wait;

constexpr int WBOX = BK * 128;       // 16 KB: [128 K x 128 columns]
constexpr int64_t kEarlyBytes = 32 << 20;  // stream form: weights up to which it starts during the preparation

// ---------------------------------------------------------------- prepare --

// Bulk copy of `bytes` (a multiple of 16, both addresses 16-byte aligned) into this
// CTA's shared memory, its bytes counted on `bar`.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// Named barrier of n threads that tells whether `v` held for all of them.
__device__ __forceinline__ bool barrier_and(int id, int n, bool v) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "barrier.cta.red.and.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(all)
      : "r"(static_cast<uint32_t>(v)), "r"(id), "r"(n)
      : "memory");
  return all != 0;
}

struct PrepParams {
  const void* x;
  const int32_t* index;
  const int32_t* counts;
  int64_t x_rows, R, K;
  int32_t n_experts, tile_rows;
  bool quantise;
  int8_t* q;       // [R, K]
  float* a;        // [R]
  Sched* sched;
  int32_t* counters;  // [kMaxCtas] zeroed
  uint32_t* status;
};

constexpr int kPrepThreads = 256;   // of the schedule

// Prefix sums of the experts' rows and row tiles by one CTA. Counts that are
// negative or run past R are cut off (status bit kStatusBounds), so that no row
// outside [0, R) is ever touched.
__device__ void make_schedule(const PrepParams& p) {
  constexpr int PER = kMaxExperts / kPrepThreads;
  __shared__ long long part_rows[kPrepThreads / 32];
  __shared__ int part_tiles[kPrepThreads / 32];
  __shared__ int any_bad;
  auto sync = [] { asm volatile("bar.sync 15, %0;" ::"n"(kPrepThreads) : "memory"); };  // part of the CTA
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  for (int i = tid; i < kMaxCtas; i += kPrepThreads) p.counters[i] = 0;
  long long c[PER], rows = 0;
  bool bad = false;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int e = tid * PER + j;
    c[j] = 0;
    if (e < p.n_experts) c[j] = p.counts != nullptr ? p.counts[e] : p.R;
    if (c[j] < 0) {
      c[j] = 0;
      bad = true;
    }
    rows += c[j];
  }
  long long inc = rows;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) part_rows[warp] = inc;
  sync();
  long long at = inc - rows;
  for (int w = 0; w < warp; ++w) at += part_rows[w];
  int tiles = 0, mine[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int e = tid * PER + j;
    const long long left = at < p.R ? p.R - at : 0;
    const int cut = static_cast<int>(c[j] < left ? c[j] : left);
    if (cut < c[j]) bad = true;
    if (e < p.n_experts) p.sched->off[e] = static_cast<int32_t>(at < p.R ? at : p.R);
    at += c[j];
    if (e == p.n_experts - 1) p.sched->off[p.n_experts] = static_cast<int32_t>(at < p.R ? at : p.R);
    mine[j] = (cut + p.tile_rows - 1) / p.tile_rows;
    tiles += mine[j];
  }
  int tinc = tiles;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, tinc, o);
    if (lane >= o) tinc += v;
  }
  if (lane == 31) part_tiles[warp] = tinc;
  sync();
  int t = tinc - tiles;
  for (int w = 0; w < warp; ++w) t += part_tiles[w];
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int e = tid * PER + j;
    if (e < p.n_experts) p.sched->pre[e] = t;
    t += mine[j];
    if (e == p.n_experts - 1) p.sched->pre[p.n_experts] = t;
  }
  if (tid == 0) any_bad = 0;
  sync();
  if (bad) any_bad = 1;
  sync();
  if (tid == 0) *p.status = any_bad ? kStatusBounds : 0u;
}

// Eight values of a row as they lie in memory: 16 bytes (bf16) or 32.
template <bool BF16>
struct Raw {
  uint4 v[BF16 ? 1 : 2];
};

template <bool BF16>
__device__ __forceinline__ Raw<BF16> load_raw(const void* row, int v) {
  Raw<BF16> r;
#pragma unroll
  for (int i = 0; i < (BF16 ? 1 : 2); ++i) r.v[i] = static_cast<const uint4*>(row)[v * (BF16 ? 1 : 2) + i];
  return r;
}

template <bool BF16>
__device__ __forceinline__ void unpack(const Raw<BF16>& r, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < (BF16 ? 1 : 2); ++i) {
    const uint32_t w[4] = {r.v[i].x, r.v[i].y, r.v[i].z, r.v[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (BF16) {
        f[2 * j] = __uint_as_float(w[j] << 16);
        f[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
      } else {
        f[4 * i + j] = __uint_as_float(w[j]);
      }
    }
  }
}

// ---- exact quotients --------------------------------------------------------
// q = 127 x / top rounded to nearest, ties to even, as the exact quotient rounds. With
// y0 = a / top approximately, a = 127 x, the residual a - y0 top is exact in fp32 for a
// bf16 row (15 + 8 bits), and y = y0 + residual / top is the quotient within an ulp, and
// exactly the quotient where that has few bits, as every half has. A bf16 quotient
// that is no half is at least 2^-16 of itself away from one (254 m_x and (2 n + 1) m_a are
// integers, m_x < 256), so rounding y decides. Ties are common there (about one value
// in a hundred), so they must cost nothing: sending them to a careful path doubled
// the kernel's time. An fp32 quotient can lie as near as 2^-33 to a half: those within two
// ulp are compared exactly.

// 254 x against (2 low + 1) top, low the integer below: both products in two parts (value
// and exact remainder; 32 bits each, so the parts' differences are exact).
__device__ __forceinline__ int quantise_near_half(float x, float top, float low) {
  const float odd = 2.0f * low + 1.0f;
  const float a = 254.0f * x, b = odd * top;
  const float d = (a - b) + (fmaf(254.0f, x, -a) - fmaf(odd, top, -b));
  const int l = static_cast<int>(low);
  return d > 0.0f ? l + 1 : (d < 0.0f ? l : l + (l & 1));
}

// What the quotients of a row need, from the bits of its largest magnitude.
struct RowScale {
  float inv, scale, top;
  bool zero;  // q = 0; a = NaN or 0
  bool far;   // next to an end of the fp32 range: every vector takes the careful path

  __device__ __forceinline__ explicit RowScale(uint32_t top_bits) {
    const float t = __uint_as_float(top_bits);
    zero = top_bits >= 0x7f800000u || top_bits == 0;
    // moved by a power of two (exact for every value that is not far below the
    // largest), so that no product leaves the range
    scale = t < 1e-30f ? 0x1p80f : (t > 1e30f ? 0x1p-30f : 1.0f);
    far = scale != 1.0f;
    top = t * scale;
    inv = 1.0f / top;
  }
};

constexpr float kNearHalf = 0.5f - 2e-5f;  // two ulp of 127

template <bool BF16>
__device__ __noinline__ uint2 quantise8_near(Raw<BF16> r, float inv, float scale, float top) {
  float f[8];
  unpack<BF16>(r, f);
  uint32_t q[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float x = f[j] * scale, y = 127.0f * x * inv, m = rintf(y);
    int n = static_cast<int>(m);
    if (fabsf(y - m) > 0.4999f) n = quantise_near_half(x, top, y < m ? m - 1.0f : m);
    q[j / 4] |= static_cast<uint32_t>(n & 0xff) << (8 * (j % 4));
  }
  return make_uint2(q[0], q[1]);
}

// Eight quotients to bytes. Adding 1.5 * 2^23 leaves a quotient rounded to an integer
// (ties to even) in the low mantissa bits.
template <bool BF16>
__device__ __forceinline__ uint2 quantise8(Raw<BF16> r, const RowScale& s) {
  if (s.zero) return make_uint2(0, 0);
  if (s.far) return quantise8_near<BF16>(r, s.inv, s.scale, s.top);
  constexpr float kMagic = 12582912.0f;
  float f[8];
  unpack<BF16>(r, f);
  uint32_t t[8];
  float off = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float a = 127.0f * f[j], y0 = a * s.inv;
    const float y = fmaf(fmaf(-y0, s.top, a), s.inv, y0);
    const float m = y + kMagic;
    t[j] = __float_as_uint(m);
    if (!BF16) off = fmaxf(off, fabsf(y - (m - kMagic)));
  }
  if (!BF16 && off > kNearHalf) return quantise8_near<BF16>(r, s.inv, s.scale, s.top);
  return make_uint2(
      __byte_perm(__byte_perm(t[0], t[1], 0x0040), __byte_perm(t[2], t[3], 0x0040), 0x5410),
      __byte_perm(__byte_perm(t[4], t[5], 0x0040), __byte_perm(t[6], t[7], 0x0040), 0x5410));
}

// Largest magnitude of eight values, as fp32 bits (bf16: two 16-bit maxima at a time).
template <bool BF16>
__device__ __forceinline__ void largest(const Raw<BF16>& x, uint32_t& top) {
#pragma unroll
  for (int i = 0; i < (BF16 ? 1 : 2); ++i) {
    const uint32_t w[4] = {x.v[i].x, x.v[i].y, x.v[i].z, x.v[i].w};
    if (BF16) {
      const uint32_t m = __vimax3_u16x2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu, w[2] & 0x7fff7fffu);
      top = __vimax3_u16x2(m, w[3] & 0x7fff7fffu, top);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) top = max(top, w[j] & 0x7fffffffu);
    }
  }
}

// fp32 bits of what largest() gathered.
template <bool BF16>
__device__ __forceinline__ uint32_t largest_bits(uint32_t top) {
  return BF16 ? max(top << 16, top & 0xffff0000u) : top;
}

// The row's scale: the largest magnitude over 127, the correctly rounded quotient.
__device__ __forceinline__ float row_step(uint32_t top_bits) {
  return top_bits < 0x7f800000u ? __uint_as_float(top_bits) / 127.0f : __uint_as_float(0x7fc00000u);
}

// Rows to 8 bits, bound by memory: groups of NT threads take rows in turn; up to kRing
// rows of each group are on their way into shared memory as bulk copies while one is worked
// on, and a row goes from there to registers once (its largest magnitude as bits, so
// that NaN and infinity win; then the quotients). One barrier per row. The schedule is
// made by the last CTA, which has the fewest rows.
constexpr int kPrepCta = 512;
constexpr int kRing = 4;
constexpr int kRingBytes = 200 * 1024;  // shared memory for rows on their way
constexpr int kPrepVec = 8;             // vectors of 8 values per thread: few warps per row, as each has its own overhead

template <bool BF16, int NT>
__global__ void __launch_bounds__(kPrepCta, 1)
    moe_int8_prepare_kernel(const __grid_constant__ PrepParams p, int32_t ring) {
  constexpr int GROUPS = kPrepCta / NT, WARPS = NT / 32;
  extern __shared__ __align__(128) uint8_t rows_smem[];
  __shared__ __align__(8) uint64_t full[GROUPS][kRing];
  __shared__ int real_row[GROUPS][kRing];
  __shared__ uint32_t part[GROUPS][2][WARPS < 32 ? 32 : WARPS];
  launch_dependents();
  if (blockIdx.x == gridDim.x - 1 && threadIdx.x < kPrepThreads) make_schedule(p);
  if (!p.quantise) return;
  const int group = threadIdx.x / NT, tid = threadIdx.x % NT, lane = threadIdx.x % 32, warp = tid / 32;
  const int64_t row_bytes = p.K * (BF16 ? 2 : 4);
  const int nvec = static_cast<int>(p.K / 8);
  uint8_t* mine = rows_smem + group * ring * row_bytes;
  const int64_t step = static_cast<int64_t>(gridDim.x) * GROUPS;
  const int64_t r0 = blockIdx.x + static_cast<int64_t>(group) * gridDim.x;
  auto fetch = [&](int64_t r, int slot) {  // thread 0 of the group
    const int64_t src = p.index != nullptr ? p.index[r] : r;
    const bool real = src >= 0 && src < p.x_rows;
    real_row[group][slot] = real;
    if (real) {
      mbar_arrive_expect_tx(&full[group][slot], static_cast<uint32_t>(row_bytes));
      bulk_load(mine + slot * row_bytes, static_cast<const uint8_t*>(p.x) + src * row_bytes,
                static_cast<uint32_t>(row_bytes), &full[group][slot]);
    } else {
      mbar_arrive(&full[group][slot]);
    }
  };
  if (tid == 0) {
    for (int s = 0; s < ring; ++s) mbar_init(&full[group][s], 1);
    fence_mbar_init();
    for (int s = 0; s < ring; ++s)
      if (r0 + s * step < p.R) fetch(r0 + s * step, s);
  }
  __syncthreads();
  int slot = 0;
  uint32_t phase = 0, flip = 0;
  for (int64_t r = r0; r < p.R; r += step) {
    bool ok = mbar_wait(&full[group][slot], phase, kWaitLimitNs);
    const bool real = ok && real_row[group][slot];
    const uint8_t* row = mine + slot * row_bytes;
    Raw<BF16> raw[kPrepVec];
    uint32_t top_bits = 0;
    if (real) {
#pragma unroll
      for (int i = 0; i < kPrepVec; ++i)
        if (tid + i * NT < nvec) raw[i] = load_raw<BF16>(row, tid + i * NT);
#pragma unroll
      for (int i = 0; i < kPrepVec; ++i)
        if (tid + i * NT < nvec) largest<BF16>(raw[i], top_bits);
    }
    top_bits = __reduce_max_sync(0xffffffffu, largest_bits<BF16>(top_bits));
    if (NT == 32) {
      ok = __all_sync(0xffffffffu, ok);
      __syncwarp();
    } else {
      if (lane == 0) part[group][flip][warp] = top_bits;
      ok = barrier_and(1 + group, NT, ok);  // all or none of the group go on
      top_bits = __reduce_max_sync(0xffffffffu, lane < WARPS ? part[group][flip][lane] : 0u);
    }
    if (!ok) {
      if (tid == 0) {
        atomicOr(p.status, kStatusProducerTimeout);
        // unwinding: no copy may still be on its way into this CTA's memory
        for (int i = 0; i < ring && r + i * step < p.R; ++i) {
          mbar_wait(&full[group][slot], phase, kWaitLimitNs);
          if (++slot == ring) {
            slot = 0;
            phase ^= 1;
          }
        }
      }
      return;
    }
    // the row is in registers: its slot takes the next one
    if (tid == 0 && r + ring * step < p.R) fetch(r + ring * step, slot);
    const RowScale rs(top_bits);
    if (tid == 0) p.a[r] = row_step(top_bits);
    uint2* dst = reinterpret_cast<uint2*>(p.q + r * p.K);
#pragma unroll
    for (int i = 0; i < kPrepVec; ++i)
      if (tid + i * NT < nvec)
        dst[tid + i * NT] = quantise8<BF16>(raw[i], rs);
    flip ^= 1;
    if (++slot == ring) {
      slot = 0;
      phase ^= 1;
    }
  }
}

// Rows too long for two of them to be in shared memory: one row per CTA, read twice
// (the second time from L2).
template <bool BF16>
__global__ void __launch_bounds__(kPrepCta) moe_int8_prepare_long_kernel(const __grid_constant__ PrepParams p) {
  __shared__ uint32_t part[kPrepCta / 32];
  launch_dependents();
  if (blockIdx.x == 0) {
    if (threadIdx.x < kPrepThreads) make_schedule(p);
    return;
  }
  const int64_t r = static_cast<int64_t>(blockIdx.x) - 1;
  const int64_t src = p.index != nullptr ? p.index[r] : r;
  const int nvec = static_cast<int>(p.K / 8);
  uint2* dst = reinterpret_cast<uint2*>(p.q + r * p.K);
  if (src < 0 || src >= p.x_rows) {  // a row of zeros: x may hold no row at all
    for (int v = threadIdx.x; v < nvec; v += kPrepCta) dst[v] = make_uint2(0, 0);
    if (threadIdx.x == 0) p.a[r] = 0.0f;
    return;
  }
  const void* row = static_cast<const uint8_t*>(p.x) + src * p.K * (BF16 ? 2 : 4);
  uint32_t top_bits = 0;
  for (int v = threadIdx.x; v < nvec; v += kPrepCta) largest<BF16>(load_raw<BF16>(row, v), top_bits);
  top_bits = __reduce_max_sync(0xffffffffu, largest_bits<BF16>(top_bits));
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = top_bits;
  __syncthreads();
  top_bits = __reduce_max_sync(0xffffffffu, part[threadIdx.x % (kPrepCta / 32)]);
  const RowScale rs(top_bits);
  if (threadIdx.x == 0) p.a[r] = row_step(top_bits);
  for (int v = threadIdx.x; v < nvec; v += kPrepCta)
    dst[v] = quantise8<BF16>(load_raw<BF16>(row, v), rs);
}

// ---------------------------------------------------------------- product --

struct Params {
  const Sched* sched;
  const int32_t* counts; // [n_experts] or nullptr: all R rows (split form of up to 32 experts)
  const float* a;        // [R] row scales
  const float* gate;     // [R] or nullptr
  const __nv_bfloat16* s0;
  const __nv_bfloat16* s1;
  void* out;
  int32_t* counters;     // stream form: K blocks summed of a tile that several CTAs share
  int32_t* part;         // stream form: their partial sums
  uint32_t* status;
  int64_t R;
  int32_t N, n_experts, nt, kb, act;
  int32_t group_rows, group_limit;  // pair form: row tiles per L2 group (tile_order.cuh)
};

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

// Gate activations of N values in fp32, as z * sigmoid(t): that keeps the relative
// accuracy of large negative z (1 + tanh would cancel), and is two special-function
// instructions. The mode is looked at once for all of them.
//   GELU (tanh form) = z / (1 + e^-t), t = 2 sqrt(2 / pi) (z + 0.044715 z^3); SiLU: t = z
// SiLU has no cubic term at all: one with a factor of 0 would make NaN of 0 * inf, where z
// is +inf or its square leaves the fp32 range. A z of -inf is NaN in every mode (-inf * 0).
template <int N>
__device__ __forceinline__ void activate(float (&z)[N], int mode) {
  constexpr float kLog2e = 1.4426950408889634f;
  constexpr float kTanh = 1.5957691216057308f;
  if (mode == MOE_ACT_GELU_ERF) {
#pragma unroll
    for (int j = 0; j < N; ++j) z[j] *= 0.5f * erfcf(-0.70710678118654752f * z[j]);
  } else if (mode == MOE_ACT_SILU) {
#pragma unroll
    for (int j = 0; j < N; ++j) z[j] *= rcp_fast(1.0f + ex2_fast(-kLog2e * z[j]));
  } else {
    constexpr float c1 = -kLog2e * kTanh, c3 = c1 * 0.044715f;
#pragma unroll
    for (int j = 0; j < N; ++j) z[j] *= rcp_fast(1.0f + ex2_fast(z[j] * fmaf(z[j] * c3, z[j], c1)));
  }
}

// Index of the expert that holds row tile `m` (pre[e] <= m < pre[e + 1]).
__device__ __forceinline__ int expert_of(const int32_t* pre, int n, int m) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (pre[mid] <= m) lo = mid;
    else hi = mid;
  }
  return lo;
}

// ---- stream form ----------------------------------------------------------
// For few rows per expert: the weights' columns are the MMA's M side and the tile's
// tokens (at most ROWS) its N side, so the tensor work follows the tokens there are
// and the kernel is bound by reading each weight byte once. The tiles that do not fill
// a wave are cut into equal runs of K blocks; a tile that the runs cut is summed from its
// parts: every CTA but the one that brings the last part stores its 32-bit sums and counts
// its K blocks, that one adds all parts (integers: any order gives the same sum) and
// finishes the tile. No CTA waits for another.

template <int ROWS>
struct StreamCfg {
  static constexpr int X_BYTES = ROWS * BK;
  static constexpr int STAGE_BYTES = X_BYTES + 2 * WBOX;
  static constexpr int STAGES = ROWS <= 64 ? 5 : 4;
  static constexpr int ACC_COLS = 2 * ROWS;  // two 128-column blocks of weights
  static constexpr int TMEM_COLS = 2 * ACC_COLS;
  static constexpr int PART_INTS = 256 * ROWS;  // of a part: [16-token step][8][column][4], see the epilogue
  static constexpr int SMEM = STAGES * STAGE_BYTES + 1024 + 256;  // alignment slack, barriers; + schedule
};
constexpr int XBOX_ROWS = 32;
constexpr int kMinRun = 4;  // K blocks of a run at least: 512 of K
// What joining the parts of a tile costs, in K blocks; measured, us, whole and cut: 80 gated
// tiles of 24 blocks 25.9 and 28.9, 120 plain ones of 6 14.4 and 18.5; 64 of 57, 32 more than
// a run has, 36.4 and 33.6.
constexpr int kJoin = 16, kJoinHidden = 3;

struct Seg {
  int e, row0, rows, n0, kb0, kb1;
  int64_t tile0;  // cut part: first K block of the tile in its sequence
};

template <int ROWS, bool DUAL, bool OB>
__global__ void __launch_bounds__(256, 1)
    moe_int8_stream_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w0,
                           const __grid_constant__ CUtensorMap tm_w1, const __grid_constant__ Params p) {
  using C = StreamCfg<ROWS>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(smem + C::STAGES * C::STAGE_BYTES);
  uint64_t* empty_bar = full_bar + C::STAGES;
  uint64_t* tfull_bar = empty_bar + C::STAGES;
  uint64_t* tempty_bar = tfull_bar + 2;
  uint64_t* drain_bar = tempty_bar + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* last_flag = abort_flag + 1;
  int32_t* pre = reinterpret_cast<int32_t*>(full_bar) + 64;  // 256 B after the barriers' start
  int32_t* off = pre + p.n_experts + 1;

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull_bar[b], 1);
      mbar_init(&tempty_bar[b], 4);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_x);
    tma_prefetch_desc(&tm_w0);
    if (DUAL) tma_prefetch_desc(&tm_w1);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::TMEM_COLS);
    tmem_relinquish();
  }
  wait_prerequisites();  // the schedule and the quantised rows
  for (int e = threadIdx.x; e <= p.n_experts; e += 256) {
    pre[e] = p.sched->pre[e];
    off[e] = p.sched->off[e];
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  // Tiles: waves of one whole tile per CTA, whose neighbours in the order (next columns of
  // the same weights) run side by side, and a remainder of fewer tiles than CTAs, cut into
  // equal runs of K blocks. The cut part goes first, so that joining its sums hides
  // behind the whole tiles.
  const int64_t tiles = static_cast<int64_t>(pre[p.n_experts]) * p.nt;
  const int64_t waves = tiles / gridDim.x, whole0 = tiles - waves * gridDim.x;
  const int64_t total = whole0 * p.kb;  // K blocks of the cut part
  // Runs of at least kMinRun K blocks: no run is empty, the last CTAs may have none. Whole
  // tiles, one to a CTA, where cutting would shorten the longest run by less than joining
  // costs: kJoin K blocks, or kJoinHidden behind whole tiles.
  int64_t G = min(static_cast<int64_t>(gridDim.x), max(total / kMinRun, int64_t(1)));
  if (p.kb - (total + G - 1) / G <= (waves == 0 ? kJoin : kJoinHidden)) G = whole0;
  const int64_t me = blockIdx.x;
  const int64_t lo = me < G ? total * me / G : total, hi = me < G ? total * (me + 1) / G : total;

  struct Cursor {
    int64_t pos, wave;
  };
  auto next = [&](Cursor& c, Seg& s) -> bool {
    int64_t tile;
    if (c.pos < hi) {
      tile = c.pos / p.kb;
      s.tile0 = tile * p.kb;
      s.kb0 = static_cast<int>(c.pos - s.tile0);
      s.kb1 = static_cast<int>(min(hi - s.tile0, static_cast<int64_t>(p.kb)));
      c.pos = s.tile0 + s.kb1;
    } else if (c.wave < waves) {
      tile = whole0 + c.wave * gridDim.x + me;
      s.tile0 = 0;
      s.kb0 = 0;
      s.kb1 = p.kb;
      ++c.wave;
    } else {
      return false;
    }
    s.e = expert_of(pre, p.n_experts, static_cast<int>(tile / p.nt));
    const int mt = pre[s.e + 1] - pre[s.e];
    const int local = static_cast<int>(tile - static_cast<int64_t>(pre[s.e]) * p.nt);
    const int m = local % mt;  // row tiles run fastest: those that share weights follow one another
    s.n0 = (local / mt) * (DUAL ? 128 : 256);
    s.row0 = off[s.e] + m * ROWS;
    s.rows = min(ROWS, off[s.e + 1] - s.row0);
    return true;
  };

  if (warp == 0 && lane == 0) {
    // ------------------------------------------------------------ producer --
    const uint64_t wpolicy = policy_evict_first();
    int stage = 0, issued = 0;
    uint32_t phase = 0;
    bool ok = true;
    Seg s;
    Cursor cur{lo, 0};
    while (ok && next(cur, s)) {
      const int boxes = (s.rows + XBOX_ROWS - 1) / XBOX_ROWS;
      for (int kb = s.kb0; kb < s.kb1; ++kb) {
        if (!mbar_wait(&empty_bar[stage], phase ^ 1, kWaitLimitNs) || *abort_flag) {
          atomicOr(p.status, kStatusProducerTimeout);
          *abort_flag = 1;
          ok = false;
          break;
        }
        uint8_t* xs = smem + stage * C::STAGE_BYTES;
        uint8_t* ws = xs + C::X_BYTES;
        mbar_arrive_expect_tx(&full_bar[stage], boxes * XBOX_ROWS * BK + 2 * WBOX);
        tma_load_3d_hint(ws, &tm_w0, &full_bar[stage], s.n0, kb * BK, s.e, wpolicy);
        tma_load_3d_hint(ws + WBOX, DUAL ? &tm_w1 : &tm_w0, &full_bar[stage], DUAL ? s.n0 : s.n0 + 128, kb * BK,
                         s.e, wpolicy);
        for (int b = 0; b < boxes; ++b)
          tma_load_2d(xs + b * XBOX_ROWS * BK, &tm_x, &full_bar[stage], kb * BK, s.row0 + b * XBOX_ROWS);
        ++issued;
        if (++stage == C::STAGES) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    if (!ok) {  // unwinding: no copy may still be on its way into this CTA's memory
      for (int i = 0; i < min(issued, C::STAGES); ++i) {
        if (--stage < 0) {
          stage = C::STAGES - 1;
          phase ^= 1;
        }
        mbar_wait(&full_bar[stage], phase, kWaitLimitNs);
      }
    }
  } else if (warp == 1 && lane == 0) {
    // ----------------------------------------------------------------- MMA --
    int stage = 0, acc = 0;
    uint32_t phase = 0, acc_phase = 0;
    bool ok = true;
    Seg s;
    Cursor cur{lo, 0};
    while (ok && next(cur, s)) {
      if (!mbar_wait(&tempty_bar[acc], acc_phase ^ 1, kWaitLimitNs) || *abort_flag) ok = false;
      tc_fence_after();
      const uint32_t d = tmem_base + acc * C::ACC_COLS;
      const uint32_t ntok = (s.rows + 31) / 32 * 32;
      const uint32_t idesc = idesc_s8_s32(128, ntok, 1, 0);
      for (int kb = s.kb0; ok && kb < s.kb1; ++kb) {
        if (!mbar_wait(&full_bar[stage], phase, kWaitLimitNs) || *abort_flag) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t xs = smem_u32(smem + stage * C::STAGE_BYTES);
        const uint32_t ws = xs + C::X_BYTES;
#pragma unroll
        for (int k = 0; k < BK / 32; ++k) {
          // Weights: MN-major, 128 columns to a swizzle row, 8-deep K groups 1024 B
          // apart; a 32-deep step is 4096 B. Tokens: K-major, 8-row groups 1024 B
          // apart; the step is 32 B inside the swizzled row.
          const uint32_t accum = kb > s.kb0 || k > 0;
          const uint64_t xd = smem_desc_sw128(xs + k * 32, 16, 1024);
          umma_s8(d, smem_desc_sw128(ws + k * 4096, WBOX, 1024), xd, idesc, accum);
          umma_s8(d + ROWS, smem_desc_sw128(ws + WBOX + k * 4096, WBOX, 1024), xd, idesc, accum);
        }
        umma_commit(&empty_bar[stage]);
        if (++stage == C::STAGES) {
          stage = 0;
          phase ^= 1;
        }
      }
      if (ok) umma_commit(&tfull_bar[acc]);
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1;
      }
    }
    if (!ok) {
      atomicOr(p.status, kStatusMmaTimeout);
      *abort_flag = 1;
      umma_commit(drain_bar);  // unwinding: the tensor cores are done before TMEM is freed
      mbar_wait(drain_bar, 0, kWaitLimitNs);
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue --
    // Lane = weight column 32 q + lane of each of the two blocks.
    const int q = warp - 4, col = 32 * q + lane;
    int acc = 0;
    uint32_t acc_phase = 0;
    Seg s;
    Cursor cur{lo, 0};
    while (next(cur, s)) {
      // What the finished tile needs besides its sums, on its way before they are: this
      // lane's channel scales, and the scale (with the gate) of rows lane, lane + 32, ...
      const int ca = s.n0 + col, cb = DUAL ? ca : ca + 128;
      const bool va = ca < p.N, vb = cb < p.N;
      const int64_t se = static_cast<int64_t>(s.e) * p.N;
      const float sa = va ? __bfloat162float(p.s0[se + ca]) : 0.0f;
      const float sb = vb ? __bfloat162float((DUAL ? p.s1 : p.s0)[se + cb]) : 0.0f;
      float ra[ROWS / 32], rg[ROWS / 32];
#pragma unroll
      for (int i = 0; i < ROWS / 32; ++i) {
        const int64_t row = s.row0 + 32 * i + lane;
        const bool in = 32 * i + lane < s.rows;
        // the row's scale, and with the gate: of the up product, or of the only one
        ra[i] = in ? p.a[row] : 0.0f;  // may be written while this kernel starts: not a read-only load
        rg[i] = in && p.gate != nullptr ? ra[i] * __ldg(p.gate + row) : ra[i];
        if (!DUAL) ra[i] = rg[i];
      }
      const bool whole = s.kb1 - s.kb0 == p.kb;
      bool ok = warp_wait(&tfull_bar[acc], acc_phase, abort_flag);
      if (!whole) ok = barrier_and(1, 128, ok);  // the warps meet below: all go on, or none
      if (!ok) {
        atomicOr(p.status, kStatusEpilogueTimeout);
        *abort_flag = 1;
        break;
      }
      tc_fence_after();
      const uint32_t tb = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + acc * C::ACC_COLS;
      // Parts of the tile: CTAs first .. last hold its K blocks; the first one's part
      // is the end of its run (slot 1), the others' the start of theirs (slot 0).
      int first = 0, last = 0;
      bool finish = true;
      if (!whole) {
        first = static_cast<int>(((s.tile0 + 1) * G - 1) / total);
        last = static_cast<int>(((s.tile0 + p.kb) * G - 1) / total);
        int32_t* mine = p.part + (2 * me + (me == first ? 1 : 0)) * C::PART_INTS;
#pragma unroll 1
        for (int j0 = 0; j0 < s.rows; j0 += 16) {
          uint32_t u[16], v[16];
          tmem_ld16x2(tb + j0, tb + ROWS + j0, u, v);
          int4* o = reinterpret_cast<int4*>(mine) + (j0 / 16) * 8 * 128 + col;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            __stcg(o + i * 128, make_int4(u[4 * i], u[4 * i + 1], u[4 * i + 2], u[4 * i + 3]));
            __stcg(o + (4 + i) * 128, make_int4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]));
          }
        }
        __threadfence();
        asm volatile("bar.sync 1, 128;" ::: "memory");
        if (threadIdx.x == 128) {
          const int had = tc::atomic_add_acq_rel_gpu(&p.counters[first], s.kb1 - s.kb0);
          *last_flag = had + (s.kb1 - s.kb0) == p.kb;
        }
        asm volatile("bar.sync 1, 128;" ::: "memory");
        finish = *last_flag != 0;
        if (finish) __threadfence();
      }
      if (finish) {
#pragma unroll
        for (int j0 = 0; j0 < ROWS; j0 += 16) {
          if (j0 >= s.rows) break;
          uint32_t u[16], v[16];
          tmem_ld16x2(tb + j0, tb + ROWS + j0, u, v);
          if (!whole) {
            // the other CTAs' parts, two of them on their way at a time
#pragma unroll 2
            for (int c = first; c <= last; ++c) {
              if (c == me) continue;
              const int4* o = reinterpret_cast<const int4*>(p.part + (2 * static_cast<int64_t>(c) + (c == first ? 1 : 0)) *
                                                                         C::PART_INTS) + (j0 / 16) * 8 * 128 + col;
              int4 w[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) w[i] = __ldcg(o + i * 128);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                u[4 * i] += w[i].x; u[4 * i + 1] += w[i].y; u[4 * i + 2] += w[i].z; u[4 * i + 3] += w[i].w;
                v[4 * i] += w[4 + i].x; v[4 * i + 1] += w[4 + i].y; v[4 * i + 2] += w[4 + i].z; v[4 * i + 3] += w[4 + i].w;
              }
            }
          }
          float za[16], zb[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float a = __shfl_sync(0xffffffffu, ra[j0 / 32], j0 % 32 + j);
            const float b = DUAL ? __shfl_sync(0xffffffffu, rg[j0 / 32], j0 % 32 + j) : a;
            za[j] = static_cast<float>(static_cast<int>(u[j])) * sa * a;
            zb[j] = static_cast<float>(static_cast<int>(v[j])) * sb * b;
          }
          if (DUAL) {
            activate(za, p.act);
#pragma unroll
            for (int j = 0; j < 16; ++j) za[j] *= zb[j];
          }
          auto put = [&](auto* out) {
            using T = std::remove_pointer_t<decltype(out)>;
            T* o = out + (static_cast<int64_t>(s.row0) + j0) * p.N;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              if (j0 + j >= s.rows) break;
              if (va) o[static_cast<int64_t>(j) * p.N + ca] = static_cast<T>(za[j]);
              if (!DUAL && vb) o[static_cast<int64_t>(j) * p.N + cb] = static_cast<T>(zb[j]);
            }
          };
          if (OB) put(static_cast<__nv_bfloat16*>(p.out));
          else put(static_cast<float*>(p.out));
        }
      }
      if (!whole) asm volatile("bar.sync 1, 128;" ::: "memory");  // last_flag read by all before the next one
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty_bar[acc]);
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
}

// The schedule of up to 32 experts by one warp, from the counts themselves (a lane
// each), cut off as make_schedule cuts them off. `report`: write the status word, too.
__device__ __forceinline__ void warp_schedule(const Params& p, int tile_rows, int32_t* pre, int32_t* off, bool report) {
  const int lane = threadIdx.x % 32;
  long long c = 0;
  if (lane < p.n_experts) c = p.counts != nullptr ? p.counts[lane] : p.R;
  const bool negative = c < 0;
  if (negative) c = 0;
  long long end = c;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, end, o);
    if (lane >= o) end += v;
  }
  const int first = static_cast<int>(min(end - c, static_cast<long long>(p.R)));
  const int last = static_cast<int>(min(end, static_cast<long long>(p.R)));
  const int tiles = (last - first + tile_rows - 1) / tile_rows;
  int tend = tiles;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, tend, o);
    if (lane >= o) tend += v;
  }
  if (lane < p.n_experts) {
    pre[lane] = tend - tiles;
    off[lane] = first;
  }
  if (lane == p.n_experts - 1) {
    pre[p.n_experts] = tend;
    off[p.n_experts] = last;
  }
  const bool bad = __any_sync(0xffffffffu, negative || last - first < c);
  if (report && lane == 0) *p.status = bad ? kStatusBounds : 0u;
}

// ---- split form --------------------------------------------------------------
// For products with few tiles, where time is latency: a cluster of S CTAs takes one
// tile, each a run of its K blocks; the partial sums meet in shared memory, and every
// CTA adds and finishes each S-th row from its peers' memory. 64 x 4096 x 4096: 10.7 us.
// (In the stream form one CTA joined the parts from L2: 64 x 4096 x 4096 took 20-25 us.)

template <int ROWS, bool DUAL, bool OB>
__global__ void __launch_bounds__(256, 1)
    moe_int8_split_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w0,
                          const __grid_constant__ CUtensorMap tm_w1, const __grid_constant__ Params p, int32_t S) {
  using C = StreamCfg<ROWS>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(smem + C::STAGES * C::STAGE_BYTES);
  uint64_t* empty_bar = full_bar + C::STAGES;
  uint64_t* tfull_bar = empty_bar + C::STAGES;
  uint64_t* drain_bar = tfull_bar + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int32_t* pre = reinterpret_cast<int32_t*>(full_bar) + 64;
  int32_t* off = pre + p.n_experts + 1;
  int32_t* part = reinterpret_cast<int32_t*>(smem);  // [ROWS][256] sums, once the ring is done with

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int rank = static_cast<int>(cluster_ctarank());
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    mbar_init(tfull_bar, 1);
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_x);
    tma_prefetch_desc(&tm_w0);
    if (DUAL) tma_prefetch_desc(&tm_w1);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::ACC_COLS);
    tmem_relinquish();
  }
  if (p.n_experts <= 32) {
    if (warp == 2) warp_schedule(p, ROWS, pre, off, blockIdx.x == 0);
    wait_prerequisites();  // the quantised rows
  } else {
    wait_prerequisites();  // the schedule and the quantised rows
    for (int e = threadIdx.x; e <= p.n_experts; e += 256) {
      pre[e] = p.sched->pre[e];
      off[e] = p.sched->off[e];
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int tile = static_cast<int>(blockIdx.x / S);
  if (tile < pre[p.n_experts] * p.nt) {  // the same for the whole cluster
    const int e = expert_of(pre, p.n_experts, tile / p.nt);
    const int mt = pre[e + 1] - pre[e], local = tile - pre[e] * p.nt;
    const int n0 = (local / mt) * (DUAL ? 128 : 256);
    const int row0 = off[e] + (local % mt) * ROWS;
    const int rows = min(ROWS, off[e + 1] - row0);
    const int kb0 = p.kb * rank / S, kb1 = p.kb * (rank + 1) / S;
    if (warp == 0 && lane == 0) {
      // ---------------------------------------------------------- producer --
      const uint64_t wpolicy = policy_evict_first();
      const int boxes = (rows + XBOX_ROWS - 1) / XBOX_ROWS;
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait(&empty_bar[stage], phase ^ 1, kWaitLimitNs) || *abort_flag) {
          atomicOr(p.status, kStatusProducerTimeout);
          *abort_flag = 1;
          for (int i = 0; i < min(issued, C::STAGES); ++i) {  // no copy may still be on its way
            if (--stage < 0) {
              stage = C::STAGES - 1;
              phase ^= 1;
            }
            mbar_wait(&full_bar[stage], phase, kWaitLimitNs);
          }
          break;
        }
        uint8_t* xs = smem + stage * C::STAGE_BYTES;
        uint8_t* ws = xs + C::X_BYTES;
        mbar_arrive_expect_tx(&full_bar[stage], boxes * XBOX_ROWS * BK + 2 * WBOX);
        tma_load_3d_hint(ws, &tm_w0, &full_bar[stage], n0, kb * BK, e, wpolicy);
        tma_load_3d_hint(ws + WBOX, DUAL ? &tm_w1 : &tm_w0, &full_bar[stage], DUAL ? n0 : n0 + 128, kb * BK, e, wpolicy);
        for (int b = 0; b < boxes; ++b)
          tma_load_2d(xs + b * XBOX_ROWS * BK, &tm_x, &full_bar[stage], kb * BK, row0 + b * XBOX_ROWS);
        ++issued;
        if (++stage == C::STAGES) {
          stage = 0;
          phase ^= 1;
        }
      }
    } else if (warp == 1 && lane == 0) {
      // --------------------------------------------------------------- MMA --
      const uint32_t idesc = idesc_s8_s32(128, (rows + 31) / 32 * 32, 1, 0);
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait(&full_bar[stage], phase, kWaitLimitNs) || *abort_flag) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t xs = smem_u32(smem + stage * C::STAGE_BYTES);
        const uint32_t ws = xs + C::X_BYTES;
#pragma unroll
        for (int k = 0; k < BK / 32; ++k) {  // operand layouts as in the stream form
          const uint32_t accum = kb > kb0 || k > 0;
          const uint64_t xd = smem_desc_sw128(xs + k * 32, 16, 1024);
          umma_s8(tmem_base, smem_desc_sw128(ws + k * 4096, WBOX, 1024), xd, idesc, accum);
          umma_s8(tmem_base + ROWS, smem_desc_sw128(ws + WBOX + k * 4096, WBOX, 1024), xd, idesc, accum);
        }
        umma_commit(&empty_bar[stage]);
        if (++stage == C::STAGES) {
          stage = 0;
          phase ^= 1;
        }
      }
      if (ok) {
        umma_commit(tfull_bar);
      } else {
        atomicOr(p.status, kStatusMmaTimeout);
        *abort_flag = 1;
        umma_commit(drain_bar);  // unwinding: the tensor cores are done before TMEM is freed
        mbar_wait(drain_bar, 0, kWaitLimitNs);
      }
    } else if (warp >= 4) {
      // ---------------------------------------------------- sums to shared --
      // Every load of the ring has been consumed once the last MMA is complete.
      if (warp_wait(tfull_bar, 0, abort_flag)) {
        tc_fence_after();
        const int q = warp - 4, col = 32 * q + lane;
        const uint32_t tb = tmem_base + (static_cast<uint32_t>(32 * q) << 16);
#pragma unroll 1
        for (int j0 = 0; j0 < rows; j0 += 16) {
          uint32_t u[16], v[16];
          tmem_ld16x2(tb + j0, tb + ROWS + j0, u, v);
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            part[(j0 + j) * 256 + col] = static_cast<int>(u[j]);
            part[(j0 + j) * 256 + 128 + col] = static_cast<int>(v[j]);
          }
        }
        tc_fence_before();
      } else {
        atomicOr(p.status, kStatusEpilogueTimeout);
        *abort_flag = 1;
      }
    }
    // What the finish needs besides the sums, on its way meanwhile.
    const int c = threadIdx.x % 128, half = threadIdx.x / 128;
    const int ca = n0 + c, cb = DUAL ? ca : ca + 128;
    const bool va = ca < p.N, vb = cb < p.N;
    const int64_t se = static_cast<int64_t>(e) * p.N;
    const float sa = va ? __bfloat162float(p.s0[se + ca]) : 0.0f;
    const float sb = vb ? __bfloat162float((DUAL ? p.s1 : p.s0)[se + cb]) : 0.0f;
    __syncwarp();
    cluster_sync();  // every CTA's sums are in its shared memory
    constexpr int kAtOnce = 4;  // rows whose remote loads are on their way together
    for (int r0 = rank + S * half; r0 < rows; r0 += 2 * S * kAtOnce) {
      int32_t w[kAtOnce][2] = {};
      float a[kAtOnce], ag[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const int r = min(r0 + 2 * S * k, rows - 1);
        const int64_t row = static_cast<int64_t>(row0) + r;
        a[k] = p.a[row];  // may be written while this kernel starts: not a read-only load
        ag[k] = p.gate != nullptr ? __ldg(p.gate + row) : 1.0f;
      }
      for (int i = 0; i < S; ++i) {
        const uint32_t base = mapa_shared(part, i) + c * 4;
        int32_t t[kAtOnce][2];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
          const uint32_t at = base + min(r0 + 2 * S * k, rows - 1) * 1024;
          t[k][0] = ld_shared_cluster_s32(at);
          t[k][1] = ld_shared_cluster_s32(at + 512);
        }
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
          w[k][0] += t[k][0];
          w[k][1] += t[k][1];
        }
      }
      float za[kAtOnce], zb[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        ag[k] *= a[k];
        za[k] = static_cast<float>(w[k][0]) * sa * (DUAL ? a[k] : ag[k]);
        zb[k] = static_cast<float>(w[k][1]) * sb * ag[k];
      }
      if (DUAL) {
        activate(za, p.act);
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) za[k] *= zb[k];
      }
      auto put = [&](auto* out) {
        using T = std::remove_pointer_t<decltype(out)>;
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
          const int r = r0 + 2 * S * k;
          T* o = out + (static_cast<int64_t>(row0) + r) * p.N;
          if (r < rows && va) o[ca] = static_cast<T>(za[k]);
          if (!DUAL && r < rows && vb) o[cb] = static_cast<T>(zb[k]);
        }
      };
      if (OB) put(static_cast<__nv_bfloat16*>(p.out));
      else put(static_cast<float*>(p.out));
    }
    cluster_sync();  // no CTA leaves while another may read its sums
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, C::ACC_COLS);
  }
}

// ---- pair form --------------------------------------------------------------
// For many rows per expert: a cluster of two CTAs on an SM pair computes 256 rows x 256
// accumulator columns with cta_group::2 (128 gate and 128 up columns of a gated pair).
// Each CTA loads its own 128 rows and 128 weight columns, 32 KB a stage for 512 tensor
// cycles, and keeps its 128 rows of the sums in its own TMEM (two accumulators, so the
// epilogue of one tile runs beside the next one's products). Tiles are handed out in
// order from a counter, row tiles of one weight tile next to one another, so that the
// pairs that run together share weights in L2 (tile_order.cuh).
//
// With 256-row tiles the operands a CTA loads for 512 tensor cycles, 64 B a cycle, are
// more than L2 delivers (about 50): the tensor pipe was busy 72 % of the cycles. Tiles of
// 512 rows (H = 2) use each weight stage for two MMAs, 48 KB for 1024 cycles: 80 % busy
// (4096 rows of 2 experts, 6144 x 8192 gated: 296 us with the former, 271). Their two
// halves are the two accumulators, so the next tile cannot start beside this one's
// epilogue; it starts on the first half as soon as that is in registers, and runs ahead
// on it by up to the ring's stages while the second is fetched.

constexpr int PX_BYTES = 128 * BK;              // 16 KB: this CTA's 128 rows of it
template <int H>
struct PairCfg {
  static constexpr int ROWS = H * PAIR_ROWS;               // of a tile
  static constexpr int STAGE_BYTES = H * PX_BYTES + WBOX;  // 32 or 48 KB
  static constexpr int STAGES = H == 1 ? 6 : 4;
};
constexpr int PQ = 4;             // tile-id queue: the producer leads by at most 3 tiles
// Epilogue warps: sets of four (one per 32 TMEM lanes), each set with its own columns.
constexpr int PSETS = 4;
constexpr int PEPI = 4 * PSETS;
constexpr int PTHREADS = 128 + 32 * PEPI;
constexpr int PQ_READERS = 2 + 2 * PEPI;  // odd producer, MMA thread, the epilogue warps of both CTAs
constexpr int PSCALES = 2 * 128 / PSETS;  // channel scales an epilogue warp keeps in shared memory
constexpr int PSMEM = 6 * 32 * 1024 + 1024 + 256 + PEPI * PSCALES * 4 + 2 * (kMaxExperts + 1) * 4;
static_assert(PSMEM <= 232448, "shared memory above the per-block limit");
static_assert(PairCfg<1>::STAGES * PairCfg<1>::STAGE_BYTES <= 6 * 32 * 1024 &&
                  PairCfg<2>::STAGES * PairCfg<2>::STAGE_BYTES <= 6 * 32 * 1024,
              "ring larger than its share");
static_assert((2 * PairCfg<1>::STAGES + 4 + 2 * PQ + 1) * 8 + 8 + 4 * PQ <= 256, "barrier area too small");

// Waits with cluster-scope acquire (for barriers that the other CTA arrives on): one look,
// and bounded.
__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity) {
  auto once = [&]() { return mbar_try_wait_cluster(bar, parity); };
  if (once()) return true;
  const uint64_t t0 = globaltimer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (once()) return true;
    if (globaltimer_ns() - t0 > kWaitLimitNs) return false;
  }
}

// Columns of one epilogue warp: accumulator columns [c0, c0 + PCOLS) of a plain product
// (its scales in sc[0 .. PCOLS)), or PCOLS / 2 gate columns from c0 and the up columns
// 128 further on (scales of both halves).
constexpr int PCOLS = 256 / PSETS;

template <bool DUAL>
__device__ __forceinline__ void pair_scales(const Params& p, int e, int n0, int c0, int lane, float* sc) {
  const int64_t se = static_cast<int64_t>(e) * p.N;
#pragma unroll
  for (int i = 0; i < PCOLS / 32; ++i) {
    const int j = 32 * i + lane;
    const bool up = DUAL && j >= PCOLS / 2;
    const int c = n0 + c0 + (up ? j - PCOLS / 2 : j);
    sc[j] = c < p.N ? __bfloat162float((up ? p.s1 : p.s0)[se + c]) : 0.0f;
  }
  __syncwarp();
}

// One row (thread) of a tile, its sums in registers (u, v: the gate and up columns, or
// 32 columns and the next 32): scaled, activated and stored as 32 or 64 contiguous
// bytes at a time. a, ag: the row's scale, and that times its gate.
template <bool DUAL, bool OB>
__device__ __forceinline__ void pair_epilogue(const Params& p, int n0, const uint32_t (&u)[32], const uint32_t (&v)[32],
                                              const float* sc, int64_t row, float a, float ag) {
  static_assert(PCOLS == 64, "two registers sets of 32 columns");
  auto put16 = [&](int c, const float (&y)[16]) {
    if (n0 + c >= p.N) return;  // N is a multiple of 16
    if (OB) {
      uint4* d = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + row * p.N + n0 + c);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        d[i] = make_uint4(pack_bf16x2(y[8 * i], y[8 * i + 1]), pack_bf16x2(y[8 * i + 2], y[8 * i + 3]),
                          pack_bf16x2(y[8 * i + 4], y[8 * i + 5]), pack_bf16x2(y[8 * i + 6], y[8 * i + 7]));
    } else {
      float4* d = reinterpret_cast<float4*>(static_cast<float*>(p.out) + row * p.N + n0 + c);
#pragma unroll
      for (int i = 0; i < 4; ++i) d[i] = make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
    }
  };
#pragma unroll
  for (int c = 0; c < 32; c += 16) {
    float y[16], y1[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      y[j] = static_cast<float>(static_cast<int>(u[c + j])) * sc[c + j] * (DUAL ? a : ag);
      y1[j] = static_cast<float>(static_cast<int>(v[c + j])) * sc[32 + c + j] * ag;
    }
    if (DUAL) {
      activate(y, p.act);
#pragma unroll
      for (int j = 0; j < 16; ++j) y[j] *= y1[j];
    }
    put16(c, y);
    if (!DUAL) put16(32 + c, y1);
  }
}

// Arrive on an mbarrier of either CTA, in the default (CTA) scope: what it orders is
// shared-memory and TMEM reads; a release in cluster scope would also wait for the
// epilogue's global stores (measured: 4328 x 352 x 5568 gated 76 us with it).
__device__ __forceinline__ void mbar_arrive_remote(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

template <int H, bool DUAL, bool OB>
__global__ void __launch_bounds__(PTHREADS, 1)
    moe_int8_pair_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w0,
                         const __grid_constant__ CUtensorMap tm_w1, const __grid_constant__ Params p) {
  constexpr int PSTAGES = PairCfg<H>::STAGES, PSTAGE_BYTES = PairCfg<H>::STAGE_BYTES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(smem + PSTAGES * PSTAGE_BYTES);
  uint64_t* empty_bar = full_bar + PSTAGES;
  uint64_t* tfull_bar = empty_bar + PSTAGES;
  uint64_t* tempty_bar = tfull_bar + 2;
  uint64_t* qfull_bar = tempty_bar + 2;
  uint64_t* qempty_bar = qfull_bar + PQ;
  uint64_t* drain_bar = qempty_bar + PQ;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* tile_q = abort_flag + 1;
  float* scales = reinterpret_cast<float*>(full_bar) + 64;
  int32_t* pre = reinterpret_cast<int32_t*>(scales + PEPI * PSCALES);
  int32_t* off = pre + p.n_experts + 1;

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = cluster_ctarank();  // 0: issues the MMAs of the pair
  if (threadIdx.x == 0) {
    for (int s = 0; s < PSTAGES; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull_bar[b], 1);
      mbar_init(&tempty_bar[b], 2 * PEPI);
    }
    for (int i = 0; i < PQ; ++i) {
      mbar_init(&qfull_bar[i], 1);
      mbar_init(&qempty_bar[i], PQ_READERS);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_x);
    tma_prefetch_desc(&tm_w0);
    if (DUAL) tma_prefetch_desc(&tm_w1);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  for (int e = threadIdx.x; e <= p.n_experts; e += PTHREADS) {
    pre[e] = p.sched->pre[e];
    off[e] = p.sched->off[e];
  }
  tc_fence_before();
  cluster_sync();  // barriers of both CTAs initialised, TMEM allocated in both
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int ntiles = pre[p.n_experts] * p.nt;

  struct Tile {
    int e, row0, rows, n0;
  };
  auto decode = [&](int tile) {
    Tile t;
    t.e = expert_of(pre, p.n_experts, tile / p.nt);
    const int mt = pre[t.e + 1] - pre[t.e];
    int m, c, ks;
    tile_coords(tile - pre[t.e] * p.nt, mt, p.nt, group_for(mt, p.group_rows, p.group_limit), m, c, ks);
    t.row0 = off[t.e] + m * PairCfg<H>::ROWS;
    t.rows = min(PairCfg<H>::ROWS, off[t.e + 1] - t.row0);
    t.n0 = c * (DUAL ? 128 : 256);
    return t;
  };
  // Queue operations: the tile id, -1 when none is left, -2 when a wait ran out.
  int ahead = 0;  // even CTA's producer: the tile id taken while the tile before it loads
  auto q_fill = [&](int i) -> int {
    const int slot = i % PQ;
    const uint32_t ph = (i / PQ) & 1;
    if (!mbar_wait_cluster(&qempty_bar[slot], ph ^ 1) || *abort_flag) return -2;
    const int tile = ahead < ntiles ? ahead : -1;
    if (tile >= 0) ahead = atomicAdd(p.counters, 1);
    tile_q[slot] = tile;
    st_shared_cluster_u32(mapa_shared(const_cast<int*>(&tile_q[slot]), 1), static_cast<uint32_t>(tile));
    mbar_arrive(&qfull_bar[slot]);
    mbar_arrive_cluster(mapa_shared(&qfull_bar[slot], 1));
    return tile;
  };
  auto q_take = [&](int i) -> int {  // one thread of any other role
    const int slot = i % PQ;
    const uint32_t ph = (i / PQ) & 1;
    if (!mbar_wait_cluster(&qfull_bar[slot], ph) || *abort_flag) return -2;
    const int tile = tile_q[slot];
    mbar_arrive_remote(mapa_shared(&qempty_bar[slot], 0));
    return tile;
  };
  auto q_take_warp = [&](int i) -> int {  // a whole epilogue warp, one arrive
    const int slot = i % PQ;
    const uint32_t ph = (i / PQ) & 1;
    const bool ok = mbar_wait_cluster(&qfull_bar[slot], ph) && !*abort_flag;
    if (!__all_sync(0xffffffffu, ok)) return -2;
    const int tile = tile_q[slot];
    __syncwarp();
    if (lane == 0) mbar_arrive_remote(mapa_shared(&qempty_bar[slot], 0));
    return tile;
  };

  if (warp == 0 && lane == 0) {
    // ------------------------------------------------------------ producer --
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    if (rank == 0) ahead = atomicAdd(p.counters, 1);
    for (int i = 0; ok; ++i) {
      const int tile = rank == 0 ? q_fill(i) : q_take(i);
      if (tile == -2) ok = false;
      if (tile < 0) break;
      const Tile t = decode(tile);
      const int row = t.row0 + 128 * static_cast<int>(rank);
      const int nh = H == 2 && t.rows > PAIR_ROWS ? 2 : 1;  // halves with rows
      // gated pair: the even CTA holds the gate columns, the odd one the up columns
      const CUtensorMap* wmap = DUAL && rank == 1 ? &tm_w1 : &tm_w0;
      const int n = DUAL ? t.n0 : t.n0 + 128 * static_cast<int>(rank);
      for (int kb = 0; kb < p.kb; ++kb) {
        if (!mbar_wait(&empty_bar[stage], phase ^ 1, kWaitLimitNs) || *abort_flag) {
          ok = false;
          break;
        }
        uint8_t* xs = smem + stage * PSTAGE_BYTES;
        const uint32_t bar0 = mapa_shared(&full_bar[stage], 0);
        if (rank == 0) mbar_arrive_expect_tx(&full_bar[stage], 2 * (nh * PX_BYTES + WBOX));
        tma_load_3d_pair(xs + H * PX_BYTES, wmap, bar0, n, kb * BK, t.e);
        tma_load_2d_pair(xs, &tm_x, bar0, kb * BK, row);
        if (H == 2 && nh == 2) tma_load_2d_pair(xs + PX_BYTES, &tm_x, bar0, kb * BK, row + PAIR_ROWS);
        if (++stage == PSTAGES) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    if (!ok) {
      atomicOr(p.status, kStatusProducerTimeout);
      *abort_flag = 1;
    }
    // Every stage's last release (an arrive of the pair's MMA commit) has landed
    // before this CTA may leave; after a timeout this wait is bounded as well.
    for (int i = 0; i < PSTAGES; ++i) {
      if (!mbar_wait(&empty_bar[stage], phase ^ 1, kWaitLimitNs)) {
        atomicOr(p.status, kStatusProducerTimeout);
        break;
      }
      if (++stage == PSTAGES) {
        stage = 0;
        phase ^= 1;
      }
    }
  } else if (warp == 1 && lane == 0 && rank == 0) {
    // ----------------------------------------------------------------- MMA --
    constexpr uint32_t idesc = idesc_s8_s32(PAIR_ROWS, 256, 0, 1);
    int stage = 0, acc = 0;
    uint32_t phase = 0, acc_phase = 0;
    bool ok = true;
    for (int i = 0; ok; ++i) {
      const int tile = q_take(i);
      if (tile == -2) ok = false;
      if (tile < 0) break;
      // Accumulators take turns, one per half of a tile.
      const int a0 = acc, nh = H == 2 && decode(tile).rows > PAIR_ROWS ? 2 : 1;
      if (!mbar_wait_cluster(&tempty_bar[acc], acc_phase ^ 1) || *abort_flag) ok = false;
      tc_fence_after();
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1;
      }
      auto issue = [&](int st, int half, int a, bool first) {
        const uint32_t xs = smem_u32(smem + st * PSTAGE_BYTES), ws = xs + H * PX_BYTES;
#pragma unroll
        for (int k = 0; k < BK / 32; ++k)
          umma_s8_pair(tmem_base + a * 256, smem_desc_sw128(xs + half * PX_BYTES + k * 32, 16, 1024),
                       smem_desc_sw128(ws + k * 4096, WBOX, 1024), idesc, !first || k > 0);
      };
      auto release = [&] {
        umma_commit_pair(&empty_bar[stage], 0x3);
        if (++stage == PSTAGES) {
          stage = 0;
          phase ^= 1;
        }
      };
      if (nh == 1) {
        for (int kb = 0; ok && kb < p.kb; ++kb) {
          if (!mbar_wait(&full_bar[stage], phase, kWaitLimitNs) || *abort_flag) {
            ok = false;
            break;
          }
          tc_fence_after();
          issue(stage, 0, a0, kb == 0);
          release();
        }
        if (ok) umma_commit_pair(&tfull_bar[a0], 0x3);
      } else if constexpr (H == 2) {
        const int a1 = acc;
        const uint32_t p1 = acc_phase ^ 1;
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1;
        }
        // k0, k1: K blocks issued to the first and the second half; (s0, ph0) is the
        // first half's place in the ring, (stage, phase) the second's.
        bool ready = false;
        int k0 = 0, k1 = 0, s0 = stage;
        uint32_t ph0 = phase;
        auto issue0 = [&] {
          if (!mbar_wait(&full_bar[s0], ph0, kWaitLimitNs) || *abort_flag) return false;
          tc_fence_after();
          issue(s0, 0, a0, k0 == 0);
          if (++s0 == PSTAGES) {
            s0 = 0;
            ph0 ^= 1;
          }
          if (++k0 == p.kb) umma_commit_pair(&tfull_bar[a0], 0x3);
          return true;
        };
        while (ok && k1 < p.kb) {
          if (!ready) {
            ready = mbar_try_wait_cluster(&tempty_bar[a1], p1);
            if (!ready && k0 < p.kb && k0 - k1 < PSTAGES) {
              ok = issue0();
              continue;
            }
            if (!ready && (!mbar_wait_cluster(&tempty_bar[a1], p1) || *abort_flag)) {
              ok = false;
              break;
            }
            ready = true;
            tc_fence_after();
          }
          if (k0 == k1 && !issue0()) {
            ok = false;
            break;
          }
          issue(stage, 1, a1, k1 == 0);
          release();
          ++k1;
        }
        if (ok) umma_commit_pair(&tfull_bar[a1], 0x3);
      }
    }
    if (!ok) {
      atomicOr(p.status, kStatusMmaTimeout);
      *abort_flag = 1;
      umma_commit_pair(drain_bar, 0x1);  // unwinding: the tensor cores are done before TMEM is freed
      mbar_wait(drain_bar, 0, kWaitLimitNs);
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue --
    const int q = warp % 4, set = (warp - 4) / 4;
    const int c0 = set * (DUAL ? PCOLS / 2 : PCOLS);
    float* sc = scales + (warp - 4) * PSCALES;
    const uint32_t tempty0[2] = {mapa_shared(&tempty_bar[0], 0), mapa_shared(&tempty_bar[1], 0)};
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int i = 0;; ++i) {
      const int tile = q_take_warp(i);
      if (tile == -1) break;
      Tile t{};
      int nh = 1;
      float a[H], ag[H];
      const int r0 = 128 * static_cast<int>(rank) + 32 * q + lane;  // row of the tile, and of its second half + 256
      if (tile >= 0) {  // what the tile needs besides its sums, on its way before they are
        t = decode(tile);
        if (H == 2 && t.rows > PAIR_ROWS) nh = 2;
#pragma unroll
        for (int h = 0; h < H; ++h) {
          const int r = r0 + h * PAIR_ROWS;
          const int64_t row = static_cast<int64_t>(t.row0) + r;
          a[h] = r < t.rows ? __ldg(p.a + row) : 0.0f;
          ag[h] = r < t.rows && p.gate != nullptr ? a[h] * __ldg(p.gate + row) : a[h];
        }
        pair_scales<DUAL>(p, t.e, t.n0, c0, lane, sc);
      }
      bool ok = tile != -2;
#pragma unroll
      for (int h = 0; h < H; ++h) {
        if (!ok || h >= nh) break;
        if (!warp_wait(&tfull_bar[acc], acc_phase, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        // The sums go to registers at once, so that the accumulator is free for the next
        // tile before this one is scaled and stored.
        const uint32_t tb = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + acc * 256 + c0;
        uint32_t u[32], v[32];
        tmem_ld32x2(tb, tb + (DUAL ? 128 : 32), u, v);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(tempty0[acc]);
        const int r = r0 + h * PAIR_ROWS;
        if (r < t.rows)
          pair_epilogue<DUAL, OB>(p, t.n0 + c0, u, v, sc, static_cast<int64_t>(t.row0) + r, a[h], ag[h]);
        __syncwarp();  // every lane has read the scales
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1;
        }
      }
      if (!ok) {
        atomicOr(p.status, kStatusEpilogueTimeout);
        *abort_flag = 1;
        break;
      }
    }
  }
  tc_fence_before();
  __syncwarp();
  cluster_sync();  // no CTA leaves while its peer may still signal it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

// ------------------------------------------------------------------- host --

moe_status_t check_sizes(int64_t R, int64_t K, int64_t N, int32_t n_experts, moe_dtype_t x_dtype) {
  if (R < 0 || K <= 0 || N <= 0 || n_experts < 1) return MOE_ERR_INVALID_ARG;
  if (x_dtype != MOE_F32 && x_dtype != MOE_BF16 && x_dtype != MOE_INT8) return MOE_ERR_INVALID_ARG;
  if (K % 16 != 0 || N % 16 != 0 || K >= 131072 || N > (int64_t(1) << 20) || R > (int64_t(1) << 24) ||
      n_experts > kMaxExperts)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool weight_map(CUtensorMap* m, const void* w, const moe_int8_args_t* a) {
  const uint64_t dims[3] = {static_cast<uint64_t>(a->N), static_cast<uint64_t>(a->K),
                            static_cast<uint64_t>(a->n_experts)};
  const uint64_t strides[2] = {dims[0], dims[0] * dims[1]};
  const uint32_t box[3] = {128, BK, 1};
  return encode_tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, w, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

bool row_map(CUtensorMap* m, const void* q, const moe_int8_args_t* a, uint32_t box_rows) {
  const uint64_t dims[2] = {static_cast<uint64_t>(a->K), static_cast<uint64_t>(a->R)};
  const uint64_t strides[1] = {dims[0]};
  const uint32_t box[2] = {BK, box_rows};
  return encode_tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, q, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// Stream form, or split form with `split` CTAs per tile.
template <int ROWS, bool DUAL, bool OB>
cudaError_t launch_stream(const moe_int8_args_t* a, const void* q, Params p, int32_t split, bool dependent,
                          cudaStream_t s) {
  using C = StreamCfg<ROWS>;
  auto kern = moe_int8_stream_kernel<ROWS, DUAL, OB>;
  auto split_kern = moe_int8_split_kernel<ROWS, DUAL, OB>;
  constexpr int kSmem = C::SMEM + 2 * (kMaxExperts + 1) * 4;
  static_assert(kSmem <= 232448, "shared memory above the per-block limit");
  static_assert((2 * C::STAGES + 5) * 8 + 16 <= 256, "barrier area too small");
  const cudaError_t err = set_smem_limit_once(split > 0 ? reinterpret_cast<const void*>(split_kern)
                                                        : reinterpret_cast<const void*>(kern), kSmem);
  if (err != cudaSuccess) return err;
  CUtensorMap tx, tw0, tw1;
  if (!row_map(&tx, q, a, XBOX_ROWS) || !weight_map(&tw0, a->w, a) || !weight_map(&tw1, DUAL ? a->w_up : a->w, a))
    return cudaErrorInvalidValue;
  p.nt = static_cast<int32_t>((a->N + (DUAL ? 127 : 255)) / (DUAL ? 128 : 256));
  if (split > 0) {
    const int64_t tiles = std::min<int64_t>(a->R, (a->R + ROWS - 1) / ROWS + a->n_experts - 1) * p.nt;
    return launch_kernel(split_kern, static_cast<unsigned>(tiles * split), 256, kSmem, s, split, dependent, tx, tw0, tw1, p,
                         split);
  }
  const int64_t most = ((a->R + ROWS - 1) / ROWS + a->n_experts) * p.nt * p.kb;
  const int grid = static_cast<int>(std::min<int64_t>(std::min(device_sm_count(), kMaxCtas), most));
  // Started while the rows are prepared where weights take microseconds; with more of them
  // CTAs that start apart lose the DRAM pages that neighbours share (5 to 8 %).
  const int64_t weights = a->n_experts * a->K * a->N * (DUAL ? 2 : 1);
  return launch_kernel(kern, grid, 256, kSmem, s, 1, dependent && weights <= kEarlyBytes, tx, tw0, tw1, p);
}

template <int H, bool DUAL, bool OB>
cudaError_t launch_pair(const moe_int8_args_t* a, const void* q, Params p, cudaStream_t s) {
  auto kern = moe_int8_pair_kernel<H, DUAL, OB>;
  const cudaError_t err = set_smem_limit_once(reinterpret_cast<const void*>(kern), PSMEM);
  if (err != cudaSuccess) return err;
  // Clusters of two that fit at once on this device (queried once per device).
  const int max_pairs = once_per_device(reinterpret_cast<const void*>(&launch_pair<H, DUAL, OB>), [](const void*) {
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = 2;
    at.val.clusterDim.y = 1;
    at.val.clusterDim.z = 1;
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3(2 * (device_sm_count() / 2), 1, 1);
    c.blockDim = dim3(PTHREADS, 1, 1);
    c.dynamicSmemBytes = PSMEM;
    c.attrs = &at;
    c.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, moe_int8_pair_kernel<H, DUAL, OB>, &c) != cudaSuccess || n <= 0)
      n = device_sm_count() / 2;
    return n;
  });
  CUtensorMap tx, tw0, tw1;
  if (!row_map(&tx, q, a, 128) || !weight_map(&tw0, a->w, a) || !weight_map(&tw1, DUAL ? a->w_up : a->w, a))
    return cudaErrorInvalidValue;
  p.nt = static_cast<int32_t>((a->N + (DUAL ? 127 : 255)) / (DUAL ? 128 : 256));
  constexpr int ROWS = PairCfg<H>::ROWS;
  p.group_rows = row_group_size(ROWS, (a->K + 1) / 2, tc::kL2GroupBytes);
  p.group_limit = row_group_size(ROWS, (a->K + 1) / 2, tc::kL2UngroupedBytes);
  const int64_t most = ((a->R + ROWS - 1) / ROWS + a->n_experts) * p.nt;
  return launch_kernel(kern, 2 * static_cast<unsigned>(std::min<int64_t>(most, max_pairs)), PTHREADS, PSMEM, s, 2, false,
                       tx, tw0, tw1, p);
}

template <bool BF16, int NT>
cudaError_t launch_prepare_ring(const PrepParams& p, int32_t ring, cudaStream_t s) {
  auto kern = moe_int8_prepare_kernel<BF16, NT>;
  const cudaError_t err = set_smem_limit_once(reinterpret_cast<const void*>(kern), kRingBytes);
  if (err != cudaSuccess) return err;
  const size_t smem = p.quantise ? static_cast<size_t>(kPrepCta / NT) * ring * p.K * (BF16 ? 2 : 4) : 0;
  const int64_t grid = p.quantise ? std::min<int64_t>(p.R, device_sm_count()) : 1;
  kern<<<static_cast<unsigned>(grid), kPrepCta, smem, s>>>(p, ring);
  return cudaGetLastError();
}

// Threads per row: the fewest whose registers hold it (a warp for K <= 2048, 128 threads
// for K <= 8192, 256 for K <= 16384, 512 for K <= 32768), as long as two rows of every group fit in
// shared memory.
template <bool BF16>
cudaError_t launch_prepare(const PrepParams& p, cudaStream_t s) {
  auto ring = [&](int nt) -> int32_t {
    if (p.K > static_cast<int64_t>(nt) * 8 * kPrepVec) return 0;
    const int64_t rows = kRingBytes / (p.K * (BF16 ? 2 : 4)) / (kPrepCta / nt);
    return rows < 2 ? 0 : static_cast<int32_t>(std::min<int64_t>(rows, kRing));
  };
  if (!p.quantise) return launch_prepare_ring<BF16, 512>(p, 0, s);
  if (const int32_t n = ring(32)) return launch_prepare_ring<BF16, 32>(p, n, s);
  if (const int32_t n = ring(128)) return launch_prepare_ring<BF16, 128>(p, n, s);
  if (const int32_t n = ring(256)) return launch_prepare_ring<BF16, 256>(p, n, s);
  if (const int32_t n = ring(512)) return launch_prepare_ring<BF16, 512>(p, n, s);
  moe_int8_prepare_long_kernel<BF16><<<static_cast<unsigned>(1 + p.R), kPrepCta, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace i8
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_int8_workspace_size(int64_t R, int64_t K, int64_t N, int32_t n_experts, moe_dtype_t x_dtype,
                               int32_t with_up) {
  if (R <= 0 || (with_up != 0 && with_up != 1) || i8::check_sizes(R, K, N, n_experts, x_dtype) != MOE_OK) return 0;
  return i8::plan(R, K, N, n_experts, x_dtype, with_up == 1).total;
}

moe_status_t moe_int8_product(const moe_int8_args_t* a, void* workspace, size_t ws_bytes, moe_stream_t stream) {
  if (!a) return MOE_ERR_INVALID_ARG;
  const moe_status_t st = i8::check_sizes(a->R, a->K, a->N, a->n_experts, a->x_dtype);
  if (st != MOE_OK) return st;
  if (a->out_dtype != MOE_F32 && a->out_dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
  const bool rows8 = a->x_dtype == MOE_INT8, dual = a->w_up != nullptr;
  if (dual && (a->activation < MOE_ACT_GELU_TANH || a->activation > MOE_ACT_SILU)) return MOE_ERR_INVALID_ARG;
  if (a->x_rows < 0 || a->x_rows > (int64_t(1) << 31) || (!a->index && a->x_rows != a->R)) return MOE_ERR_INVALID_ARG;
  if (a->R == 0) return MOE_OK;
  if ((!a->x && a->x_rows > 0) || !a->w || !a->s || !a->out || (dual != (a->s_up != nullptr))) return MOE_ERR_INVALID_ARG;
  if (rows8 != (a->x_scale != nullptr) || (rows8 && a->index) || (!a->counts && a->n_experts != 1))
    return MOE_ERR_INVALID_ARG;
  const void* const all[] = {a->x, a->x_scale, a->index, a->counts, a->w, a->w_up, a->s, a->s_up, a->gate, a->out};
  for (const void* q : all)
    if (!i8::aligned16(q)) return MOE_ERR_MISALIGNED;
  const i8::Layout L = i8::plan(a->R, a->K, a->N, a->n_experts, a->x_dtype, dual);
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 || ws_bytes < L.total)
    return MOE_ERR_WORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  cudaStream_t s = static_cast<cudaStream_t>(stream);

  i8::PrepParams pp{};
  pp.x = a->x;
  pp.index = a->index;
  pp.counts = a->counts;
  pp.x_rows = a->x_rows;
  pp.R = a->R;
  pp.K = a->K;
  pp.n_experts = a->n_experts;
  pp.tile_rows = L.tile_rows;
  pp.quantise = !rows8;
  pp.q = reinterpret_cast<int8_t*>(ws + L.q);
  pp.a = reinterpret_cast<float*>(ws + L.a);
  pp.sched = reinterpret_cast<i8::Sched*>(ws + L.sched);
  pp.counters = reinterpret_cast<int32_t*>(ws + L.counters);
  pp.status = reinterpret_cast<uint32_t*>(ws + L.status);
  // Rows that are 8-bit already need nothing prepared where the product kernel makes
  // its own schedule.
  const bool prepared = !rows8 || L.split == 0 || a->n_experts > 32;
  if (prepared &&
      (a->x_dtype == MOE_F32 ? i8::launch_prepare<false>(pp, s) : i8::launch_prepare<true>(pp, s)) != cudaSuccess)
    return MOE_ERR_CUDA;

  i8::Params p{};
  p.sched = pp.sched;
  p.counts = a->counts;
  p.a = rows8 ? a->x_scale : pp.a;
  p.gate = a->gate;
  p.s0 = static_cast<const __nv_bfloat16*>(a->s);
  p.s1 = static_cast<const __nv_bfloat16*>(a->s_up);
  p.out = a->out;
  p.counters = pp.counters;
  p.part = reinterpret_cast<int32_t*>(ws + L.part);
  p.status = pp.status;
  p.R = a->R;
  p.N = static_cast<int32_t>(a->N);
  p.n_experts = a->n_experts;
  p.kb = static_cast<int32_t>((a->K + i8::BK - 1) / i8::BK);
  p.act = a->activation;
  const void* q = rows8 ? a->x : static_cast<const void*>(pp.q);
  const bool ob = a->out_dtype == MOE_BF16;
  auto form = [&](auto rows) {
    constexpr int ROWS = decltype(rows)::value;
    if (dual)
      return ob ? i8::launch_stream<ROWS, true, true>(a, q, p, L.split, prepared, s)
                : i8::launch_stream<ROWS, true, false>(a, q, p, L.split, prepared, s);
    return ob ? i8::launch_stream<ROWS, false, true>(a, q, p, L.split, prepared, s)
              : i8::launch_stream<ROWS, false, false>(a, q, p, L.split, prepared, s);
  };
  auto pair = [&](auto h) {
    constexpr int H = decltype(h)::value;
    if (dual) return ob ? i8::launch_pair<H, true, true>(a, q, p, s) : i8::launch_pair<H, true, false>(a, q, p, s);
    return ob ? i8::launch_pair<H, false, true>(a, q, p, s) : i8::launch_pair<H, false, false>(a, q, p, s);
  };
  cudaError_t e;
  if (L.tile_rows == 64) e = form(std::integral_constant<int, 64>{});
  else if (L.tile_rows == 128) e = form(std::integral_constant<int, 128>{});
  else if (L.tile_rows == 256) e = pair(std::integral_constant<int, 1>{});
  else e = pair(std::integral_constant<int, 2>{});
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
