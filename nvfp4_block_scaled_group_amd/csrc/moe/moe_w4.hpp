// moe_w4.hpp -- bf16 activations times NVFP4 weights: the operand decode
// shared by the single-token kernels and the adapter projection.
//
// value(code) * value(S) has at most 6 significant bits and lies in
// 2^-10 .. 2688, so it is exact in bf16; the activations stay the bf16 they
// are, and the MFMA's fp32 sum is the only rounding before the line factor
// A / 2688 is applied.
#pragma once
#include "moe_common.hpp"

namespace moe {

typedef float f32x2 __attribute__((ext_vector_type(2)));

// Eight codes of a word times value(S), as bf16.
__device__ __forceinline__ bf16x8 decode8_bf16(uint32_t w, float S) {
  const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0);
  const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
  const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2);
  const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
  const u32x4 r = {pack_bf16(a[0] * S, a[1] * S), pack_bf16(b[0] * S, b[1] * S), pack_bf16(c[0] * S, c[1] * S),
                   pack_bf16(d[0] * S, d[1] * S)};
  return __builtin_bit_cast(bf16x8, r);
}

}  // namespace moe
