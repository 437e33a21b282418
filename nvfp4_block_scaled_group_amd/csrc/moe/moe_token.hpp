// moe_token.hpp -- the product of a few bf16 rows with a run of NVFP4 lines,
// shared by the single-token expert kernels and the adapter projection.
//
// MFMA 16x16x32: rows are tokens, columns are weight lines, so a tile costs
// the same for 1 token as for 16.  What bounds it is reading the weights
// (0.5625 byte an element); the work per CU that has to stay under that is
// the decode (2 VALU operations an element) and the loads' addresses: in the
// MFMA layout neighbouring lanes hold different lines, so every lane of a load
// is a request of its own.  Hence
//  * a lane takes 64 consecutive elements of its line a step: two 16-byte
//    loads of codes and one of four scale bytes, two steps in flight; the
//    loads share cache lines, so the codes are not streamed past the caches
//    (8 tokens, 5568 x 1504, 32 experts: 60 us instead of 76);
//  * the tokens' rows are staged in LDS (loads in the MFMA layout from memory
//    cost four times the weights' requests: 25 us instead of 22 for 8 rows of a
//    7168 x 7168 projection with adapters);
//  * the eight waves of a work-group split the contraction KS ways and the
//    lines 8 / KS ways, and join their sums in LDS in a fixed order.
#pragma once
#include "moe_w4.hpp"

namespace moe {

constexpr int kModeGlu = 0;     // tiles alternate: 16 gate lines, the 16 up lines of the same columns
constexpr int kModeLinear = 1;  // tiles of 16 consecutive lines
constexpr int kStepK = 256;     // contraction step of a wave
constexpr int kTokenThreads = 512;
constexpr int kTokenWaves = kTokenThreads / 64;
constexpr int kTokenLds = 72 * 1024;  // of the 160 KB of a CU, so that two work-groups fit; twice that where one is enough

typedef __attribute__((address_space(3))) void* lds_ptr_t;
// s_waitcnt for at most n outstanding vector-memory operations.
constexpr int waitcnt_vm(int n) { return (n & 15) | (7 << 4) | (15 << 8) | ((n >> 4) << 14); }

// Waves on a SIMD that the registers leave room for.
constexpr int token_waves(int mt) { return mt >= 4 ? 2 : 4; }

// Buffer descriptor over `bytes` bytes (below 2^31): reads past it give zero.
__device__ __forceinline__ rsrc_t range_rsrc(const void* p, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(uni(reinterpret_cast<int64_t>(p))), 0,
                                           uni((uint32_t)bytes), 0x00020000);
}

// How the contraction runs: chunks of KS * per steps whose x is staged
// together; in each, wave part p takes `per` steps (an even number).
struct TokenPlan {
  int32_t ks;      // waves that split the contraction: 1, 2, 4 or 8
  int32_t per;     // steps of a wave in a chunk
  int32_t chunks;
  int32_t rows;    // rows of a pass at most
  int32_t pitch;   // bytes of a staged row
  int32_t shared;  // bytes of the staged rows, then of the waves' sums
  int32_t lds;     // bytes of dynamic LDS
};

// rows: the most rows of a pass; ks: waves that should split the contraction
// (fewer where their staged rows would not fit or a wave would have no step:
// 23 tokens, 384 elements in two steps, 4 ways 24 us, 1 way 13); tiles: MFMA
// tiles a wave joins through LDS; extra: bytes the caller wants beside them;
// groups: the work-groups of the launch.
inline TokenPlan token_plan(int64_t k, int rows, int ks, int tiles, int64_t extra, int64_t groups) {
  const int64_t limit = (rows <= 16 && groups > kCus ? kTokenLds : 2 * kTokenLds) - extra, steps = (k + kStepK - 1) / kStepK;
  while (ks > 1 && (rows * (ks * 4 * kStepK + 16) > limit || 2 * ks > steps + 1)) ks /= 2;
  const int64_t want = ((steps + ks - 1) / ks + 1) / 2 * 2;
  const int64_t room = (limit / rows - 16) / (2 * kStepK) / ks / 2 * 2;
  TokenPlan p;
  p.ks = ks;
  p.rows = rows;
  p.per = (int32_t)(want < room ? want : room);
  p.chunks = (int32_t)((steps + (int64_t)p.per * ks - 1) / ((int64_t)p.per * ks));
  p.pitch = p.per * ks * 2 * kStepK + 16;
  const int64_t x = (int64_t)rows * p.pitch, join = kTokenWaves * tiles * 1024;
  p.shared = (int32_t)((x > join ? x : join) + 15) / 16 * 16;
  p.lds = (int32_t)(p.shared + extra);
  return p;
}

// The NL tiles of 16 lines a wave multiplies.  Tiles past the last column
// repeat the last one and their results are dropped by the caller, tile by
// tile (the number of columns is a multiple of 16).
template <int MODE, int NL>
struct TileLines {
  rsrc_t data[NL], scale[NL];
  uint32_t doff, soff;  // this lane's line; its 32 bytes of codes / four scale bytes of step 0
  bool dwords;          // scale bytes of every line start on a dword

  __device__ __forceinline__ void init(const uint8_t* b_data, const uint8_t* b_scale, int64_t line0, int64_t col0,
                                       int64_t ocols, int64_t k, int lane) {
#pragma unroll
    for (int t = 0; t < NL; ++t) {
      const int c = MODE == kModeGlu ? t / 2 : t;
      const int64_t line = line0 + (MODE == kModeGlu && (t & 1) ? ocols : 0) + min<int64_t>(col0 + 16 * c, ocols - 16);
      data[t] = range_rsrc(b_data + line * (k / 2), 8 * k);
      scale[t] = range_rsrc(b_scale + line * (k / 16), k);
    }
    doff = (lane & 15) * (uint32_t)(k / 2) + 32 * (lane >> 4);
    soff = (lane & 15) * (uint32_t)(k / 16) + 4 * (lane >> 4);
    dwords = k % 64 == 0;
  }
};

// Codes and scales of step s: elements 256 s + 64 g .. + 63 of each line (g =
// lane / 16).  Granules of 32 elements past k (a multiple of 32), and steps
// past the last, read as zero codes.
template <int NL>
struct StepCodes {
  u32x4 codes[NL][2];
  uint32_t scales[NL];

  template <class W>
  __device__ __forceinline__ void load(const W& w, uint32_t s, uint32_t steps, const uint32_t (&cut)[2]) {
    const uint32_t past = s >= steps ? kOutOfRange : 0u;
    s = min(s, steps - 1);
    const uint32_t o0 = past | (s + 1 == steps ? cut[0] : 0u), o1 = past | (s + 1 == steps ? cut[1] : 0u);
#pragma unroll
    for (int t = 0; t < NL; ++t) {
      codes[t][0] = __builtin_amdgcn_raw_buffer_load_b128(w.data[t], w.doff | o0, s * (kStepK / 2), 0);
      codes[t][1] = __builtin_amdgcn_raw_buffer_load_b128(w.data[t], (w.doff + 16) | o1, s * (kStepK / 2), 0);
      if (w.dwords)
        scales[t] = __builtin_amdgcn_raw_buffer_load_b32(w.scale[t], w.soff | o0, s * (kStepK / 16), 0);
      else
        scales[t] = __builtin_amdgcn_raw_buffer_load_b16(w.scale[t], w.soff | o0, s * (kStepK / 16), 0) |
                    (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(w.scale[t], (w.soff + 2) | o1, s * (kStepK / 16), 0)
                        << 16;
    }
  }
};

// acc[m][t] = the rows of token tile m times the lines of tile t, over this
// wave's part of the contraction.  row_of(i): x's row of the i-th of `rows`
// rows; beside(): work of the caller while the first x is on its way.  All
// threads of the work-group; xlds is free again on return only after the
// caller's next barrier.
template <int MT, int NL, class W, class RowOf, class Beside>
__device__ __forceinline__ void token_multiply(const W& w, const TokenPlan& P, const uint16_t* x, int64_t k,
                                               int rows, int wave, int lane, uint8_t* xlds, RowOf row_of,
                                               f32x4 (&acc)[MT][NL], Beside beside) {
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < NL; ++t) acc[m][t] = f32x4{0, 0, 0, 0};
  const uint32_t steps = (uint32_t)((k + kStepK - 1) / kStepK);
  const int part = wave % P.ks;
  const uint32_t span = P.ks * P.per;  // steps of a chunk
  const int e0 = (int)(k - (int64_t)(steps - 1) * kStepK) - 64 * (lane >> 4);  // this lane's elements in the last step
  const uint32_t cut[2] = {e0 > 0 ? 0u : kOutOfRange, e0 > 32 ? 0u : kOutOfRange};
  StepCodes<NL> ring[2];
  uint32_t at = part * P.per, done = 0;  // the wave's next step to load, and how many of the chunk's it has loaded
  auto load_next = [&](StepCodes<NL>& r) {
    r.load(w, at, steps, cut);
    at += 1;
    if (++done == (uint32_t)P.per) {
      done = 0;
      at += span - P.per;
    }
  };
  load_next(ring[0]);
  load_next(ring[1]);
  const int xrow[4] = {(lane & 15), 16 + (lane & 15), 32 + (lane & 15), 48 + (lane & 15)};
  uint32_t xoff[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) xoff[m] = (xrow[m] < rows ? xrow[m] : 0) * P.pitch + 128 * (lane >> 4);
  auto use = [&](const StepCodes<NL>& c, const uint8_t* xs) {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      bf16x8 xf[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) xf[m] = *reinterpret_cast<const bf16x8*>(xs + xoff[m] + 16 * q);
#pragma unroll
      for (int t = 0; t < NL; ++t) {
        const bf16x8 b = decode8_bf16(c.codes[t][q >> 2][q & 3], e4m3_value((c.scales[t] >> (8 * (q >> 1))) & 0xFFu));
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[m][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[m], b, acc[m][t], 0, 0, 0);
      }
    }
  };
  for (int c = 0; c < P.chunks; ++c) {
    if (c) __syncthreads();
    // stage the chunk's x by direct copies, 1 KB of a row each (past k, out of
    // the row's range, they write zeros)
    const int64_t k0 = (int64_t)c * span * kStepK;
    const int pieces = span / 2;
    for (int i = wave; i < rows * pieces; i += kTokenWaves) {
      const int r = i / pieces, p = i - r * pieces;
      const rsrc_t xs = range_rsrc(x + row_of(r) * k + k0, 2 * (k > k0 ? k - k0 : 0));
      __builtin_amdgcn_raw_ptr_buffer_load_lds(xs, (lds_ptr_t)(xlds + r * P.pitch + 1024 * p), 16, 16 * lane + 1024 * p, 0, 0,
                                               0);
    }
    if (c == 0) beside();
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
    __syncthreads();
    const uint8_t* xs = xlds + part * P.per * (2 * kStepK);
#pragma unroll 1
    for (int p = 0; p < P.per; p += 2, xs += 4 * kStepK) {
      use(ring[0], xs);
      load_next(ring[0]);
      use(ring[1], xs + 2 * kStepK);
      load_next(ring[1]);
    }
  }
}

// Partial sums of the waves through LDS (join_waves between two barriers);
// joined() adds those of the KS waves of a group in wave order.
template <int MT, int NL>
__device__ __forceinline__ void join_waves(const f32x4 (&acc)[MT][NL], f32x4* red, int wave, int lane) {
  __syncthreads();
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < NL; ++t) red[((wave * MT + m) * NL + t) * 64 + lane] = acc[m][t];
  __syncthreads();
}
template <int MT, int NL>
__device__ __forceinline__ f32x4 joined(const f32x4* red, int group, int ks, int m, int t, int lane) {
  f32x4 s = red[((group * ks * MT + m) * NL + t) * 64 + lane];
  for (int w = 1; w < ks; ++w) s += red[(((group * ks + w) * MT + m) * NL + t) * 64 + lane];
  return s;
}

}  // namespace moe
