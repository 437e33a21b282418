// moe_token.hpp -- the product of a few bf16 rows with a run of NVFP4 lines,
// shared by the single-token expert kernels and the adapter projection.
#pragma once
#include "moe_w4.hpp"

namespace moe {

constexpr int kModeGlu = 0;     // tiles alternate: 16 gate lines, the 16 up lines of the same columns
constexpr int kModeLinear = 1;  // tiles of 16 consecutive lines
constexpr int kStepK = 128;     // contraction step of a wave

// The NL tiles of 16 lines a wave multiplies.  Lines past the end are read as
// the last tile's first line and their results dropped by the caller, tile by
// tile (the number of columns is a multiple of 16).
template <int MODE, int NL>
struct TileLines {
  const uint8_t *data[NL], *scale[NL];  // this lane's line of each tile, its 16-byte granule / two scale bytes of step 0

  __device__ __forceinline__ void init(const uint8_t* b_data, const uint8_t* b_scale, int64_t line0, int64_t col0,
                                       int64_t ocols, int64_t k, int lane) {
#pragma unroll
    for (int t = 0; t < NL; ++t) {
      const int c = MODE == kModeGlu ? t / 2 : t;
      const int64_t first = min<int64_t>(col0 + 16 * c, ocols - 16);
      const int64_t line = line0 + (MODE == kModeGlu && (t & 1) ? ocols : 0) + first + (lane & 15);
      data[t] = b_data + line * (k / 2) + 16 * (lane >> 4);
      scale[t] = b_scale + line * (k / 16) + 2 * (lane >> 4);
    }
  }
};

template <int MT, int NL>
struct StepLoads {
  u32x4 codes[NL];
  uint32_t scales[NL];
  u32x4 x[MT][4];

  // Step s: codes 128 s + 32 g .. + 31 of each line (g = lane / 16), the same
  // elements of each token.  `tail`: elements at or past k are left out
  // (k is a multiple of 32, so a lane's 32 are all in or all out).
  template <class W>
  __device__ __forceinline__ void load(const W& w, const uint16_t* const (&xr)[MT], int64_t s, int64_t k, int lane,
                                       bool tail) {
    const int64_t e0 = s * kStepK + 32 * (lane >> 4);
    if (tail && e0 >= k) {
#pragma unroll
      for (int t = 0; t < NL; ++t) {
        codes[t] = u32x4{0, 0, 0, 0};
        scales[t] = 0;
      }
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int q = 0; q < 4; ++q) x[m][q] = u32x4{0, 0, 0, 0};
      return;
    }
#pragma unroll
    for (int t = 0; t < NL; ++t) {
      codes[t] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(w.data[t] + s * (kStepK / 2)));
      scales[t] = *reinterpret_cast<const uint16_t*>(w.scale[t] + s * (kStepK / 16));
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int q = 0; q < 4; ++q) x[m][q] = *reinterpret_cast<const u32x4*>(xr[m] + e0 + 8 * q);
  }
};

// acc[m][t] = x rows of token tile m times the lines of tile t, over the
// steps of this wave: a contiguous share of one KS-th of them.
template <int MT, int NL, int KS, class W>
__device__ __forceinline__ void token_multiply(const W& w, const uint16_t* const (&xr)[MT], int64_t k, int part,
                                               int lane, f32x4 (&acc)[MT][NL]) {
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < NL; ++t) acc[m][t] = f32x4{0, 0, 0, 0};
  const int64_t steps = (k + kStepK - 1) / kStepK, share = (steps + KS - 1) / KS;
  const int64_t s0 = min<int64_t>(part * share, steps), s1 = min<int64_t>(s0 + share, steps);
  if (s0 >= s1) return;
  const bool tail = k % kStepK != 0;
  auto use = [&](const StepLoads<MT, NL>& c) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int t = 0; t < NL; ++t) {
        const bf16x8 b = decode8_bf16(c.codes[t][q], e4m3_value((c.scales[t] >> (8 * (q >> 1))) & 0xFFu));
#pragma unroll
        for (int m = 0; m < MT; ++m)
          acc[m][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, c.x[m][q]), b, acc[m][t], 0,
                                                              0, 0);
      }
  };
  StepLoads<MT, NL> cur, nxt;
  cur.load(w, xr, s0, k, lane, tail && s0 + 1 == steps);
  for (int64_t s = s0 + 1; s < s1; ++s) {
    nxt.load(w, xr, s, k, lane, tail && s + 1 == steps);
    use(cur);
    cur = nxt;
  }
  use(cur);
}

// Partial sums of the KS waves through LDS; joined() adds them in wave order.
template <int MT, int NL, int KS>
__device__ __forceinline__ void join_waves(const f32x4 (&acc)[MT][NL], f32x4* red, int wave, int lane) {
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < NL; ++t) red[((wave * MT + m) * NL + t) * 64 + lane] = acc[m][t];
  __syncthreads();
}
template <int MT, int NL, int KS>
__device__ __forceinline__ f32x4 joined(const f32x4* red, int m, int t, int lane) {
  f32x4 s = red[(m * NL + t) * 64 + lane];
#pragma unroll
  for (int w = 1; w < KS; ++w) s += red[((w * MT + m) * NL + t) * 64 + lane];
  return s;
}

}  // namespace moe
