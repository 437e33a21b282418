// i8_token.hpp -- a few rows times a run of 8-bit lines: the kernel behind the
// experts' single-token products and behind a projection of few rows.
//
// MFMA 16x16x64: rows are tokens, columns are weight lines, so a tile costs
// the same for 1 token as for 16.  Reading the weights bounds it (1 byte an
// element, no decode: 24 tokens of 6 among 64 experts, 2048 x 7168, 844 MB in 131 us,
// 6.4 TB/s; 1 token of 8, 7168 x 2 x 2048, 235 MB in 38 us, 6.2 TB/s, where a quarter
// of the time is the start, the cast of the row and the join; 8 rows of one 2048 x
// 7168 projection 5.9 us, 2.5 TB/s, most of it start and one round of latency).  A lane takes 16 bytes of its line at a time, four
// neighbouring lanes 64 in a row; the eight waves of a work-group split the
// contraction KS ways and the lines 8 / KS ways, and join their int32 sums,
// which are exact in any order, in LDS.  The rows are staged in LDS as codes:
// copied, or cast from bf16 by every work-group that needs them, which saves
// the launch of a cast.
#pragma once
#include <algorithm>

#include "i8_common.hpp"

namespace i8 {

constexpr int kModeGlu = 0;     // tiles alternate: 16 gate lines, the 16 up lines of the same columns
constexpr int kModeLinear = 1;  // tiles of 16 consecutive lines
constexpr int kStepK = 256;     // contraction step of a wave
constexpr int kTokenThreads = 512;
constexpr int kTokenWaves = kTokenThreads / 64;
constexpr int kTokenLds = 72 * 1024;  // of the 160 KB of a CU, so that two work-groups fit; twice that where one is enough

// Waves on a SIMD that the registers leave room for.
constexpr int token_waves(int mt) { return mt >= 2 ? 2 : 4; }

// How the contraction runs: chunks of KS * per steps whose rows are staged
// together; in each, wave part p takes `per` steps (an even number).
struct TokenPlan {
  int32_t ks;      // waves that split the contraction: 1, 2, 4 or 8
  int32_t per;     // steps of a wave in a chunk
  int32_t chunks;
  int32_t rows;    // rows of a pass at most
  int32_t pitch;   // bytes of a staged row
  int32_t lds;     // bytes of dynamic LDS: the staged rows, then the waves' sums
};

inline TokenPlan token_plan(int64_t k, int rows, int ks, int tiles, int64_t groups) {
  const int64_t limit = rows <= 16 && groups > kCus ? kTokenLds : 2 * kTokenLds, steps = (k + kStepK - 1) / kStepK;
  while (ks > 1 && (rows * (ks * 2 * kStepK + 16) > limit || 2 * ks > steps + 1)) ks /= 2;
  const int64_t want = ((steps + ks - 1) / ks + 1) / 2 * 2;
  const int64_t room = (limit / rows - 16) / kStepK / ks / 2 * 2;
  TokenPlan p;
  p.ks = ks;
  p.rows = rows;
  p.per = (int32_t)std::min(want, room);
  p.chunks = (int32_t)((steps + (int64_t)p.per * ks - 1) / ((int64_t)p.per * ks));
  p.pitch = p.per * ks * kStepK + 16;
  p.lds = (int32_t)std::max<int64_t>((int64_t)rows * p.pitch, kTokenWaves * tiles * 1024);
  return p;
}

// The NL tiles of 16 lines a wave multiplies.  Tiles past the last column
// repeat the last one and their results are dropped by the caller, tile by
// tile (the number of columns is a multiple of 16).
template <int MODE, int NL>
struct TileLines {
  rsrc_t data[NL];
  uint32_t off;  // this lane's line and its 16 bytes

  __device__ __forceinline__ void init(const int8_t* b, int64_t line0, int64_t col0, int64_t ocols, int64_t k, int lane) {
#pragma unroll
    for (int t = 0; t < NL; ++t) {
      const int c = MODE == kModeGlu ? t / 2 : t;
      const int64_t line = line0 + (MODE == kModeGlu && (t & 1) ? ocols : 0) + min<int64_t>(col0 + 16 * c, ocols - 16);
      data[t] = range_rsrc(b + line * k, 16 * k);
    }
    off = (lane & 15) * (uint32_t)k + 16 * (lane >> 4);
  }
};

// Codes of step s: bytes 256 s + 64 q + 16 g .. + 15 of each line (q = 0 .. 3,
// g = lane / 16).  Pieces past k, and steps past the last, read as zeros.
template <int NL>
struct StepCodes {
  i32x4 codes[NL][4];

  template <class W>
  __device__ __forceinline__ void load(const W& w, uint32_t s, uint32_t steps, int left) {
    const uint32_t past = s >= steps ? kOutOfRange : 0u;
    s = min(s, steps - 1);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t o = w.off + 64 * q | past | (s + 1 == steps && left <= 64 * q ? kOutOfRange : 0u);
#pragma unroll
      for (int t = 0; t < NL; ++t)
        codes[t][q] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(w.data[t], o, s * kStepK, 0));
    }
  }
};

// The rows of x, bf16 to be cast: rc[] of LDS gets how each row is cast.
struct CastRows {
  const uint16_t* x;
  RowCast* rc;
  uint32_t* lmax;  // one word a row
};
// The rows of x as codes with their scales.
struct CodeRows {
  const int8_t* q;
};

// Stages elements k0 .. k0 + len - 1 (len a multiple of 512) of the rows; what
// lies past k stays as it is, since the weights are zero there.
template <int AHEAD, class RowOf>
__device__ __forceinline__ void stage_rows(const CodeRows& X, int rows, int64_t k, int64_t k0, int len, int pitch, int wave,
                                           int lane, uint8_t* xlds, RowOf row_of) {
  const int pieces = (len + 1023) / 1024;  // 1 KB a copy
  for (int i = wave; i < rows * pieces; i += kTokenWaves) {
    const int r = i / pieces, p = i - r * pieces;
    const rsrc_t xs = range_rsrc(X.q + row_of(r) * k + k0, k > k0 ? k - k0 : 0);
    if (1024 * p + 16 * lane < len) copy16(xs, xlds + r * pitch + 1024 * p, 1024 * p + 16 * lane, 0);
  }
}
// Waves that share a row where there are fewer rows than waves.
__device__ __forceinline__ int row_waves(int rows) { return rows >= 8 ? 1 : rows >= 4 ? 2 : rows >= 2 ? 4 : 8; }
// Pieces of a row that a lane has on their way (one by one a row took 0.7 us
// out of the L2); four of them beside the weights' need the registers of two
// work-groups.
constexpr int ahead(int mt) { return mt >= 2 ? 4 : 2; }

template <int AHEAD, class RowOf>
__device__ __forceinline__ void stage_rows(const CastRows& X, int rows, int64_t k, int64_t k0, int len, int pitch, int wave,
                                           int lane, uint8_t* xlds, RowOf row_of) {
  const int granules = (int)(min<int64_t>(len, k - k0) / 16), parts = row_waves(rows);
  for (int r = wave / parts; r < rows; r += kTokenWaves / parts) {
    const u32x4* row = reinterpret_cast<const u32x4*>(X.x + row_of(r) * k + k0);
    const RowCast c = X.rc[r];
    uint8_t* to = xlds + r * pitch;
    for (int g0 = 64 * (wave % parts) + lane; g0 < granules; g0 += 64 * parts * AHEAD) {
      u32x4 lo[AHEAD], hi[AHEAD];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        const int g = min(g0 + 64 * parts * i, granules - 1);
        lo[i] = row[2 * g];
        hi[i] = row[2 * g + 1];
      }
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        const int g = g0 + 64 * parts * i;
        const u32x2 a = cast8(lo[i], c), b = cast8(hi[i], c);
        if (g < granules) *reinterpret_cast<u32x4*>(to + 16 * g) = u32x4{a[0], a[1], b[0], b[1]};
      }
    }
  }
}

// Largest magnitude of each row, from memory, and how it is cast.  All threads;
// ends with a barrier.
template <int AHEAD, class RowOf>
__device__ __forceinline__ void prepare_rows(const CodeRows&, int, int64_t, int, int, RowOf) {}
template <int AHEAD, class RowOf>
__device__ __forceinline__ void prepare_rows(const CastRows& X, int rows, int64_t k, int wave, int lane, RowOf row_of) {
  const int parts = row_waves(rows), pieces = (int)(k / 8);
  if ((int)threadIdx.x < rows) X.lmax[threadIdx.x] = 0;
  __syncthreads();
  for (int r = wave / parts; r < rows; r += kTokenWaves / parts) {
    const u32x4* row = reinterpret_cast<const u32x4*>(X.x + row_of(r) * k);
    uint32_t m = 0;
    for (int g0 = 64 * (wave % parts) + lane; g0 < pieces; g0 += 64 * parts * AHEAD) {
      u32x4 v[AHEAD];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) v[i] = row[min(g0 + 64 * parts * i, pieces - 1)];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) m = max(m, abs_max8(v[i]));
    }
    m = wave_reduce(m, [](uint32_t a, uint32_t b) { return max(a, b); });
    if (lane == 0) atomicMax(&X.lmax[r], m);
  }
  __syncthreads();
  if ((int)threadIdx.x < rows) X.rc[threadIdx.x] = row_cast(X.lmax[threadIdx.x]);
  __syncthreads();
}

// acc[m][t] = the rows of token tile m times the lines of tile t, over this
// wave's part of the contraction.  row_of(i): x's row of the i-th of `rows`
// rows.  All threads of the work-group; xlds is free again on return only
// after the caller's next barrier.
template <int MT, int NL, class W, class X, class RowOf>
__device__ __forceinline__ void token_multiply(const W& w, const TokenPlan& P, const X& x, int64_t k, int rows, int wave,
                                               int lane, uint8_t* xlds, RowOf row_of, i32x4 (&acc)[MT][NL]) {
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < NL; ++t) acc[m][t] = i32x4{0, 0, 0, 0};
  const uint32_t steps = (uint32_t)((k + kStepK - 1) / kStepK);
  const int part = wave % P.ks;
  const uint32_t span = P.ks * P.per;  // steps of a chunk
  const int left = (int)(k - (int64_t)(steps - 1) * kStepK) - 16 * (lane >> 4);  // this lane's bytes in the last step
  StepCodes<NL> ring[2];
  uint32_t at = part * P.per, done = 0;  // the wave's next step to load, and how many of the chunk's it has loaded
  auto load_next = [&](StepCodes<NL>& r) {
    r.load(w, at, steps, left);
    at += 1;
    if (++done == (uint32_t)P.per) {
      done = 0;
      at += span - P.per;
    }
  };
  load_next(ring[0]);
  load_next(ring[1]);
  prepare_rows<ahead(MT)>(x, rows, k, wave, lane, row_of);
  uint32_t xoff[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int r = 16 * m + (lane & 15);
    xoff[m] = (r < rows ? r : 0) * P.pitch + 16 * (lane >> 4);
  }
  auto use = [&](const StepCodes<NL>& c, const uint8_t* xs) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      i32x4 xf[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) xf[m] = *reinterpret_cast<const i32x4*>(xs + xoff[m] + 64 * q);
#pragma unroll
      for (int t = 0; t < NL; ++t)
#pragma unroll
        for (int m = 0; m < MT; ++m)
          acc[m][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(xf[m], c.codes[t][q], acc[m][t], 0, 0, 0);
    }
  };
  for (int c = 0; c < P.chunks; ++c) {
    if (c) __syncthreads();
    stage_rows<ahead(MT)>(x, rows, k, (int64_t)c * span * kStepK, span * kStepK, P.pitch, wave, lane, xlds, row_of);
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
    __syncthreads();
    const uint8_t* xs = xlds + part * P.per * kStepK;
#pragma unroll 1
    for (int p = 0; p < P.per; p += 2, xs += 2 * kStepK) {
      use(ring[0], xs);
      load_next(ring[0]);
      use(ring[1], xs + kStepK);
      load_next(ring[1]);
    }
  }
}

// Partial sums of the waves through LDS (join_waves between two barriers);
// joined() adds those of the KS waves of a group.
template <int MT, int NL>
__device__ __forceinline__ void join_waves(const i32x4 (&acc)[MT][NL], i32x4* red, int wave, int lane) {
  __syncthreads();
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < NL; ++t) red[((wave * MT + m) * NL + t) * 64 + lane] = acc[m][t];
  __syncthreads();
}
template <int MT, int NL>
__device__ __forceinline__ i32x4 joined(const i32x4* red, int group, int ks, int m, int t, int lane) {
  i32x4 s = red[((group * ks * MT + m) * NL + t) * 64 + lane];
  for (int w = 1; w < ks; ++w) s += red[(((group * ks + w) * MT + m) * NL + t) * 64 + lane];
  return s;
}

// A projection of a few rows of codes (i8_token.hip): out [rows, n] fp32 or
// bf16.  It is taken while the rows fit LDS in one or two pieces; past that, and
// where more than 16 rows are short, the 128 x 128 tiles of i8_gemm.hip are
// faster (us, this kernel and the tiles: 32 rows of 2048 x 7168 7.3 and 11.8, 64 rows
// 9.6 and 12.8; 24 rows of 7168 x 2048 11.0 and 14.0, 40 rows 18.0 and 14.5; 16 rows of
// 16384 x 8192 33.7 and 26.6; 32 rows of 512 x 512 5.8 and 5.2).
constexpr int64_t kFewRows = 16;
inline bool few(int64_t rows, int64_t k) {
  return rows <= 64 && rows * k <= 200000 && (rows <= kFewRows || k >= 1024);
}
int few_rows(const int8_t* a_q, const float* a_scale, int64_t rows, int64_t k, const int8_t* b_q, const float* b_scale,
             int64_t n, void* out, int32_t out_type, hipStream_t st);

}  // namespace i8
