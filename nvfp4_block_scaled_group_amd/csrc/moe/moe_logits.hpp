// moe_logits.hpp -- reading a token's logits by a group of lanes, and the
// group's reductions: shared by the selection of experts and the balance loss.
#pragma once
#include "moe_common.hpp"

namespace moe {

constexpr float kNegInf = -__builtin_huge_valf();

// A logit as the operator reads it: NaN and -inf masked, +inf as FLT_MAX.
__device__ __forceinline__ float clean(float l) { return l > kNegInf ? fminf(l, FLT_MAX) : kNegInf; }

template <class T>
__device__ __forceinline__ float logit_at(const T* p, int64_t i);
template <>
__device__ __forceinline__ float logit_at<float>(const float* p, int64_t i) { return p[i]; }
template <>
__device__ __forceinline__ float logit_at<int32_t>(const int32_t* p, int64_t i) { return (float)p[i]; }
template <>
__device__ __forceinline__ float logit_at<uint16_t>(const uint16_t* p, int64_t i) {
  return __uint_as_float((uint32_t)p[i] << 16);
}

// VPL consecutive values of a row of E (experts lane*VPL ..) as fp32, whatever
// is there past E.  With `wide` (E a multiple of VPL and the row aligned to the
// lane's piece) as vector loads.  A lane or an element past E reads one inside
// the row: no branch holds the other loads up.
template <class T, int VPL>
__device__ __forceinline__ void load_row(const T* row, int E, int lane, bool wide, float (&v)[VPL]) {
  const int e0 = lane * VPL;
  constexpr int kPer = 16 / (int)sizeof(T) < VPL ? 16 / (int)sizeof(T) : VPL;  // elements of one load
  if (wide) {
    const T* p = row + (e0 < E ? e0 : 0);
#pragma unroll
    for (int i = 0; i < VPL; i += kPer) {
      typedef T vec_t __attribute__((ext_vector_type(kPer)));
      const vec_t q = *reinterpret_cast<const vec_t*>(p + i);
#pragma unroll
      for (int c = 0; c < kPer; ++c) {
        const T x = q[c];
        v[i + c] = logit_at<T>(&x, 0);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) v[i] = logit_at<T>(row, min(e0 + i, E - 1));
  }
}
template <class T, int VPL>
__device__ __forceinline__ void load_logits(const T* row, int E, int lane, bool wide, float (&l)[VPL]) {
  load_row<T, VPL>(row, E, lane, wide, l);
#pragma unroll
  for (int i = 0; i < VPL; ++i) l[i] = lane * VPL + i < E ? clean(l[i]) : kNegInf;
}

// Value of lane ^ (the step's distance) inside a group of lanes: 1, 2, then
// the mirror of 8 and the rotation of 16, which serve reductions as well.
template <int STEP>
__device__ __forceinline__ uint32_t exchange(uint32_t v) {
  if constexpr (STEP == 0) return dpp_x1(v);
  else if constexpr (STEP == 1) return dpp_x2(v);
  else if constexpr (STEP == 2) return dpp_hmirror(v);
  else if constexpr (STEP == 3) return swap8(v);
  else {
    // the swap gives own and other half; which is which depends on the lane
    const auto r = STEP == 4 ? __builtin_amdgcn_permlane16_swap(v, v, false, false)
                             : __builtin_amdgcn_permlane32_swap(v, v, false, false);
    const bool upper = (threadIdx.x >> STEP) & 1;
    return upper ? r[0] : r[1];
  }
}
template <int LANES, int STEP = 0>
__device__ __forceinline__ float group_fmax(float v) {
  if constexpr ((1 << STEP) >= LANES) return v;
  else return group_fmax<LANES, STEP + 1>(fmaxf(v, __uint_as_float(exchange<STEP>(__float_as_uint(v)))));
}
template <int LANES, int STEP = 0>
__device__ __forceinline__ float group_sum(float v) {
  if constexpr ((1 << STEP) >= LANES) return v;
  else return group_sum<LANES, STEP + 1>(v + __uint_as_float(exchange<STEP>(__float_as_uint(v))));
}

// Vector loads of a lane's experts: a row starts on their alignment and no
// lane's piece is cut by the row's end.
inline bool wide_rows(const void* p, int E, int vpl, int size) {
  const int piece = vpl * size < 16 ? vpl * size : 16;
  return E % vpl == 0 && (int64_t)E * size % piece == 0 && aligned(p, piece);
}

}  // namespace moe
