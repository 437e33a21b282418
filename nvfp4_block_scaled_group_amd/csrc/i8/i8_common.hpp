// i8_common.hpp -- helpers shared by the HIP sources behind
// include/i8_group.h: matrix instruction types, the cast of a row and checks.
#pragma once
#include "../../../include/i8_group.h"
#include "../moe/moe_common.hpp"

namespace i8 {

using namespace moe;

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) void* lds_ptr_t;

// s_waitcnt for at most n outstanding vector-memory operations.
constexpr int waitcnt_vm(int n) { return (n & 15) | (7 << 4) | (15 << 8) | ((n >> 4) << 14); }

// Buffer descriptor over `bytes` bytes (below 2^31): reads past it give zero.
__device__ __forceinline__ rsrc_t range_rsrc(const void* p, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(uni(reinterpret_cast<int64_t>(p))), 0,
                                           uni((uint32_t)bytes), 0x00020000);
}

// 16 bytes a lane from memory to LDS: lane l's land at lds + 16 l.
__device__ __forceinline__ void copy16(rsrc_t r, uint8_t* lds, uint32_t offset, uint32_t uniform_offset) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr_t)lds, 16, offset, uniform_offset, 0, 0);
}

// ------------------------------------------------------------ cast of a row
//
// Magnitudes are compared as bit patterns: infinities and NaN are above every
// finite value, so they reach the maximum.

__device__ __forceinline__ uint32_t abs_max8(u32x4 v) {  // of 8 bf16 values, as bf16 bits
  uint32_t m = pkmax(v[0] & 0x7FFF7FFFu, v[1] & 0x7FFF7FFFu);
  m = pkmax(m, pkmax(v[2] & 0x7FFF7FFFu, v[3] & 0x7FFF7FFFu));
  return hmax(m);
}

// How a row is cast: code = nearest(x * pre * mul).
struct RowCast {
  float scale, pre, mul;
};
__device__ __forceinline__ RowCast row_cast(uint32_t amax_bits) {
  const float a = __uint_as_float(amax_bits << 16);
  RowCast c{a / 127.0f, 1.0f, 0.0f};
  if (amax_bits >= 0x7F80u) {
    c.scale = __uint_as_float(0x7FC00000u);
  } else if (amax_bits) {
    c.pre = a < 0x1p-100f ? 0x1p64f : 1.0f;  // 127 / A stays finite
    c.mul = 127.0f / (a * c.pre);
  }
  return c;
}

// Codes of 8 bf16 values.  A row that is not finite has mul 0, and its
// infinities and NaN would not give code 0 by themselves.
__device__ __forceinline__ u32x2 cast8(u32x4 v, const RowCast& c) {
  float x[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = (bf16lo(v[i]) * c.pre) * c.mul;
    x[2 * i + 1] = (bf16hi(v[i]) * c.pre) * c.mul;
  }
  const u32x2 q = {codes4(x[0], x[1], x[2], x[3]), codes4(x[4], x[5], x[6], x[7])};
  return c.mul > 0.0f ? q : u32x2{0, 0};
}

// ------------------------------------------------------------- host side

inline bool valid_k(int64_t k) { return k > 0 && k % 16 == 0 && k <= I8_MAX_K; }
inline bool valid_n(int64_t n) { return n > 0 && n % 16 == 0 && n <= (1 << 20); }

}  // namespace i8
