// combine_topk.cu — out[t] = residual[t] + sum_s weights[t, s] * y[slot_pos[t, s]]
// for any number of slots k (moe_combine_topk).
//
// Bound by memory: every row of y is read once and every row of out written once.
// A thread owns eight columns of one token (16 or 32 bytes of a row per load) and
// walks the token's slots four at a time, their loads issued together. The sum is
// fp32 in slot order and is rounded once.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int kCombineThreads = 128;
constexpr int kSlotsAtOnce = 4;

struct CombineParams {
  const void* y;
  const int32_t* slot_pos;
  const float* weights;
  const void* residual;
  void* out;
  int64_t R, T, d;
  int32_t k;
  int32_t chunks;  // CTAs per token
};

template <bool BF16>
struct Eight {  // eight values as they lie in memory
  uint4 a, b;
};

template <bool BF16>
__device__ __forceinline__ Eight<BF16> load8(const void* base, int64_t at) {
  Eight<BF16> v;
  if (BF16) {
    v.a = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + at);
    v.b = make_uint4(0, 0, 0, 0);
  } else {
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const float*>(base) + at);
    v.a = q[0];
    v.b = q[1];
  }
  return v;
}

template <bool BF16>
__device__ __forceinline__ void add8(float (&o)[8], const Eight<BF16>& v, float w) {
  const uint32_t a[4] = {v.a.x, v.a.y, v.a.z, v.a.w}, b[4] = {v.b.x, v.b.y, v.b.z, v.b.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (BF16) {
      o[2 * j] += w * __uint_as_float(a[j] << 16);
      o[2 * j + 1] += w * __uint_as_float(a[j] & 0xFFFF0000u);
    } else {
      o[j] += w * __uint_as_float(a[j]);
      o[4 + j] += w * __uint_as_float(b[j]);
    }
  }
}

template <bool YB, bool OB>
__global__ void __launch_bounds__(kCombineThreads) moe_combine_topk_kernel(const CombineParams p) {
  const int64_t t = blockIdx.x / p.chunks;
  const int64_t c = (static_cast<int64_t>(blockIdx.x % p.chunks) * kCombineThreads + threadIdx.x) * 8;
  if (c >= p.d) return;
  float o[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) o[j] = 0.0f;
  if (p.residual != nullptr) add8<OB>(o, load8<OB>(p.residual, t * p.d + c), 1.0f);
  for (int s0 = 0; s0 < p.k; s0 += kSlotsAtOnce) {
    Eight<YB> v[kSlotsAtOnce];
    float w[kSlotsAtOnce];
    bool in[kSlotsAtOnce];
#pragma unroll
    for (int i = 0; i < kSlotsAtOnce; ++i) {
      in[i] = false;
      if (s0 + i >= p.k) continue;
      const int64_t at = t * p.k + s0 + i;
      const int64_t row = __ldg(p.slot_pos + at);
      in[i] = row >= 0 && row < p.R;
      w[i] = 1.0f;
      if (in[i]) {
        if (p.weights != nullptr) w[i] = __ldg(p.weights + at);
        v[i] = load8<YB>(p.y, row * p.d + c);
      }
    }
#pragma unroll
    for (int i = 0; i < kSlotsAtOnce; ++i)
      if (in[i]) add8<YB>(o, v[i], w[i]);
  }
  const int64_t at = t * p.d + c;
  if (OB) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(o[2 * j], o[2 * j + 1]);
      w[j] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + at) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.out) + at);
    dst[0] = make_float4(o[0], o[1], o[2], o[3]);
    dst[1] = make_float4(o[4], o[5], o[6], o[7]);
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_combine_topk(const void* y, moe_dtype_t y_dtype, int64_t R, const int32_t* slot_pos,
                                         const float* weights, int64_t T, int32_t k, int64_t d,
                                         const void* residual, void* out, moe_dtype_t out_dtype,
                                         moe_stream_t stream) {
  if (T < 0 || R < 0 || k <= 0 || d <= 0) return MOE_ERR_INVALID_ARG;
  if ((y_dtype != MOE_F32 && y_dtype != MOE_BF16) || (out_dtype != MOE_F32 && out_dtype != MOE_BF16))
    return MOE_ERR_INVALID_ARG;
  if (d % 8 != 0 || d > (int64_t(1) << 20) || k > 32 || T > (int64_t(1) << 24) || R > (int64_t(1) << 29))
    return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!slot_pos || !out || (!y && R > 0)) return MOE_ERR_INVALID_ARG;
  if (!aligned16(y) || !aligned16(out) || !aligned16(residual) || !aligned16(slot_pos) || !aligned16(weights))
    return MOE_ERR_MISALIGNED;
  CombineParams p{y, slot_pos, weights, residual, out, R, T, d, k, 0};
  p.chunks = static_cast<int32_t>((d / 8 + kCombineThreads - 1) / kCombineThreads);
  if (T * p.chunks > 0x7fffffff) return MOE_ERR_UNSUPPORTED;
  const unsigned grid = static_cast<unsigned>(T * p.chunks);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool yb = y_dtype == MOE_BF16, ob = out_dtype == MOE_BF16;
  if (yb && ob) moe_combine_topk_kernel<true, true><<<grid, kCombineThreads, 0, s>>>(p);
  else if (yb) moe_combine_topk_kernel<true, false><<<grid, kCombineThreads, 0, s>>>(p);
  else if (ob) moe_combine_topk_kernel<false, true><<<grid, kCombineThreads, 0, s>>>(p);
  else moe_combine_topk_kernel<false, false><<<grid, kCombineThreads, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
