// moe_common.hpp -- helpers shared by the HIP sources behind
// include/moe_ops.h: bf16 conversion, wave64 reductions and the activations.
#pragma once
#include <hip/hip_runtime.h>
#include <float.h>
#include <stdint.h>

#include "../../../include/moe_ops.h"
#include "../nvfp4_common.hpp"
#include "../nvfp4_numerics.hpp"

namespace moe {

using namespace nvfp4g;

constexpr int kCus = 256;  // compute units of the device

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// One rounding to bf16 (nearest, ties to even), two values a dword.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const bf16x2 v = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, v);
}
__device__ __forceinline__ uint16_t to_bf16(float a) { return __builtin_bit_cast(uint16_t, (__bf16)a); }

// Four int8 codes of four fp32 values below 127.5 in magnitude:
// adding 1.5 * 2^23 rounds to the nearest whole number, ties to even, and
// leaves it in the low byte.
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  constexpr float kMagic = 12582912.0f;
  const uint32_t p = __builtin_amdgcn_perm(__float_as_uint(b + kMagic), __float_as_uint(a + kMagic), 0x0c0c0400u);
  const uint32_t q = __builtin_amdgcn_perm(__float_as_uint(d + kMagic), __float_as_uint(c + kMagic), 0x04000c0cu);
  return p | q;
}

// Reductions over the 64 lanes of a wave, the result in every lane: five
// lane exchanges inside and across 16-lane rows, then the two halves.
template <class Op>
__device__ __forceinline__ uint32_t wave_reduce(uint32_t v, Op op) {
  v = op(v, dpp_x1(v));
  v = op(v, dpp_x2(v));
  v = op(v, dpp_hmirror(v));
  v = op(v, swap8(v));
  const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = op(a[0], a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return op(b[0], b[1]);
}
__device__ __forceinline__ float wave_sum(float v) {
  return __uint_as_float(wave_reduce(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}

// Two fp32 accumulators of neighbouring rows (v, v + 1) in lane pairs that
// hold columns j, j + 1: after the exchange an even lane has row v, an odd one
// row v + 1, each with both columns, so that every store is a whole dword.
__device__ __forceinline__ void pair_columns(float a, float b, bool odd, float* lo, float* hi) {
  const float send = odd ? a : b, keep = odd ? b : a;
  const float got = __uint_as_float(dpp_x1(__float_as_uint(send)));
  *lo = odd ? got : keep;
  *hi = odd ? keep : got;
}

// Gate activation in fp32: act(g) = g * q with a logistic q = 1/(1+e^-v).
// SiLU: v = g.  GELU (tanh form): (1 + tanh(w))/2 = 1/(1+e^-2w), so v = 2w =
// 2 sqrt(2/pi) (g + 0.044715 g^3).  act'(g) = q + g q (1-q) v'.  e^-v overflows
// to inf for very negative v, where q is 0.  GELU's polynomial takes g cut to
// +-30: q is exactly 0 or 1 well inside that, and g^2 stays finite.
template <int ACT>
__device__ __forceinline__ float act_logistic(float g, float* dv) {
  float v = g;
  *dv = 1.0f;
  if (ACT == MOE_ACT_GELU) {
    const float c = fminf(fmaxf(g, -30.0f), 30.0f), c2 = c * c;
    v = 1.5957691216057308f * c * __builtin_fmaf(0.044715f, c2, 1.0f);
    *dv = 1.5957691216057308f * __builtin_fmaf(0.134145f, c2, 1.0f);
  }
  return __builtin_amdgcn_rcpf(1.0f + __expf(-v));
}

// A dimension of a launch holds fewer than 2^32 threads; past that the number
// wraps: with 2^24 + 2^20 work-groups of kThreads 2^20 ran, and the call
// succeeded.
constexpr int64_t kMaxGroups = (1ll << 32) / kThreads - 1;

// Work-groups of kThreads in a line: more than 2^23 take a second dimension.
// Its last row may hold work-groups past the last one asked for.
inline dim3 line_grid(uint32_t groups) {
  constexpr uint32_t kLine = 1u << 23;
  return groups <= kLine ? dim3(groups) : dim3(kLine, (groups - 1) / kLine + 1);
}
__device__ __forceinline__ uint32_t line_index() { return uni(blockIdx.y * gridDim.x + blockIdx.x); }

inline bool valid_type(int32_t t) { return t == MOE_F32 || t == MOE_BF16; }

}  // namespace moe
