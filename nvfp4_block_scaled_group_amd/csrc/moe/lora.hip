// lora.hip -- low-rank adapters of many requests beside one shared NVFP4
// projection, behind the C ABI of include/moe_ops.h:
//
//   y[t] = W x[t] + alpha_a B_a (A_a x[t]),   a = adapter of row t.
//
// The first launch makes v[t] = A_a x[t] (rank values a row): a work-group
// takes 16 rows and multiplies them (MFMA 16x16x32) by one of the adapters
// that any of them has.  Then the shared projection follows, with the adapters
// in its epilogue:
//   few rows (at most 64)  the weight is read once and bounds it; every
//                          16-line tile adds its rows' B_a v in fp32;
//   more rows              128 x 256 tiles, MFMA 32x32x16; each adapter present
//                          in the tile adds rank/16 MFMA steps of v B_a^T to
//                          the scaled accumulators, rows of other adapters 0.
// v is kept in fp32 (few rows), or as two bf16 halves, v = hi + lo, which
// leaves it 16 significant bits: the adapter's part then has the precision of
// the bf16 result to spare.
#include "moe_token.hpp"

namespace {

using namespace moe;

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kFewRows = 64;      // rows of the first form
constexpr int kShrinkRows = 16;   // rows of a work-group of the first launch
constexpr int kMaxSplit = 8;      // parts of the contraction over work-groups (few rows)
constexpr int kShrinkStep = 128;  // contraction step of a wave of the first launch

constexpr int round16(int r) { return (r + 15) / 16 * 16; }

// ---------------------------------------------------------------- A_a x[t]

// blockIdx = (tile of 16 rows, part of the contraction, which of the tile's
// adapters); v [parts][tokens][rank] fp32, rows without an adapter not written.
// The four waves take a share of the part each and join in LDS.  A step's
// loads are in flight together; parts and adapters are work-groups of their
// own because the chain of steps, not the bytes, is what takes the time.
template <int NR>
__global__ __launch_bounds__(kThreads) void shrink_kernel(const uint16_t* __restrict__ x, int tokens, int64_t k,
                                                          const uint16_t* __restrict__ lora_a, int adapters, int rank,
                                                          const int32_t* __restrict__ ids, float* __restrict__ v) {
  __shared__ f32x4 red[4 * NR * 64];
  const int lane = threadIdx.x & 63, wave = uni((int32_t)(threadIdx.x >> 6));
  const int row0 = uni((int32_t)blockIdx.x) * kShrinkRows;
  const int my = lane < kShrinkRows && row0 + lane < tokens ? ids[row0 + lane] : -1;
  uint64_t left = __ballot((uint32_t)my < (uint32_t)adapters && lane < kShrinkRows), rows = 0;
  int a = 0;
  for (int slot = uni((int32_t)blockIdx.z); slot >= 0; --slot) {
    if (!left) return;  // the tile has fewer adapters
    a = __builtin_amdgcn_readlane(my, (int)__builtin_ctzll(left));
    rows = __ballot(my == a) & left;
    left &= ~rows;
  }
  const int parts = uni((int32_t)gridDim.y) * 4, part = uni((int32_t)blockIdx.y) * 4 + wave;
  const int64_t steps = (k + kShrinkStep - 1) / kShrinkStep, share = (steps + parts - 1) / parts;
  const int64_t s0 = min<int64_t>(part * share, steps), s1 = min<int64_t>(s0 + share, steps);
  const uint16_t* xr = x + (int64_t)min(row0 + (lane & 15), tokens - 1) * k;
  f32x4 acc[NR];
  const uint16_t* ar[NR];  // this lane's line of each 16 ranks (a line past the rank reads the last)
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    acc[r] = f32x4{0, 0, 0, 0};
    ar[r] = lora_a + ((int64_t)a * rank + min(16 * r + (lane & 15), rank - 1)) * k;
  }
  for (int64_t s = s0; s < s1; ++s) {
    const int64_t e0 = s * kShrinkStep + 32 * (lane >> 4);
    const bool in = e0 < k;
    u32x4 xq[4], aq[NR][4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      xq[q] = in ? *reinterpret_cast<const u32x4*>(xr + e0 + 8 * q) : u32x4{0, 0, 0, 0};
#pragma unroll
      for (int r = 0; r < NR; ++r)
        aq[r][q] = in ? *reinterpret_cast<const u32x4*>(ar[r] + e0 + 8 * q) : u32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int r = 0; r < NR; ++r)
        acc[r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, xq[q]),
                                                         __builtin_bit_cast(bf16x8, aq[r][q]), acc[r], 0, 0, 0);
  }
#pragma unroll
  for (int r = 0; r < NR; ++r) red[(wave * NR + r) * 64 + lane] = acc[r];
  __syncthreads();
  // thread -> (row, rank column); element (row, col) of a tile is component
  // row % 4 of lane 16 (row / 4) + col
  const int row = threadIdx.x >> 4, col = threadIdx.x & 15;
  if (!((rows >> row) & 1)) return;
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    const float* f = reinterpret_cast<const float*>(red) + (r * 64 + 16 * (row >> 2) + col) * 4 + (row & 3);
    float sum = f[0];
#pragma unroll
    for (int w = 1; w < 4; ++w) sum += f[w * NR * 64 * 4];
    if (16 * r + col < rank) v[((int64_t)blockIdx.y * tokens + row0 + row) * rank + 16 * r + col] = sum;
  }
}

// sum_r b[r] * v[r] in fp32; the loads of 32 ranks are in flight together.
__device__ __forceinline__ float rank_dot(const uint16_t* b, const float* v, int rank) {
  float d = 0.0f;
  for (int i = 0; i < rank; i += 32) {
    u32x4 q[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i + 8 * j < rank) q[j] = *reinterpret_cast<const u32x4*>(b + i + 8 * j);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (i + 8 * j >= rank) break;
      const f32x4 lo = *reinterpret_cast<const f32x4*>(v + i + 8 * j), hi = *reinterpret_cast<const f32x4*>(v + i + 8 * j + 4);
      d = __builtin_fmaf(bf16lo(q[j][0]), lo[0], d);
      d = __builtin_fmaf(bf16hi(q[j][0]), lo[1], d);
      d = __builtin_fmaf(bf16lo(q[j][1]), lo[2], d);
      d = __builtin_fmaf(bf16hi(q[j][1]), lo[3], d);
      d = __builtin_fmaf(bf16lo(q[j][2]), hi[0], d);
      d = __builtin_fmaf(bf16hi(q[j][2]), hi[1], d);
      d = __builtin_fmaf(bf16lo(q[j][3]), hi[2], d);
      d = __builtin_fmaf(bf16hi(q[j][3]), hi[3], d);
    }
  }
  return d;
}

// alpha * v of row t, the parts summed in their order; 0 without an adapter.
__device__ __forceinline__ float row_v(const float* v, int parts, int64_t tokens, int64_t t, int rank, int c, int a,
                                       const float* alpha) {
  float s = 0.0f;
  for (int p = 0; p < parts; ++p) s += v[(p * tokens + t) * rank + c];
  return s * alpha[a];
}

// For many rows: alpha * v, the parts summed in their order, as two bf16
// halves hi and lo [tokens][rank rounded up to 16], zeros past the rank.
__global__ __launch_bounds__(kThreads) void halves_kernel(const float* __restrict__ v, int parts, int64_t tokens,
                                                          int rank, const float* __restrict__ alpha, int adapters,
                                                          const int32_t* __restrict__ ids, uint16_t* __restrict__ out) {
  const int r16 = round16(rank);
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x, t = i / r16, c = i % r16;
  if (t >= tokens) return;
  const int a = ids[t];
  if ((uint32_t)a >= (uint32_t)adapters) return;  // never read
  const float s = c < rank ? row_v(v, parts, tokens, t, rank, (int)c, a, alpha) : 0.0f;
  const uint16_t hi = to_bf16(s);
  out[i] = hi;
  out[tokens * r16 + i] = to_bf16(s - __uint_as_float((uint32_t)hi << 16));
}

// ------------------------------------------------------ projection, few rows

template <int MT, int NL>
__global__ __launch_bounds__(kTokenThreads, token_waves(MT)) void few_rows_kernel(
    const uint16_t* __restrict__ x, int tokens, int64_t k, const uint8_t* __restrict__ w_data,
    const uint8_t* __restrict__ w_scale, const float* __restrict__ w_amax, int64_t n,
    const uint16_t* __restrict__ lora_b, const float* __restrict__ alpha, int adapters, int rank,
    const int32_t* __restrict__ ids, const float* __restrict__ v, int parts, TokenPlan P, uint16_t* __restrict__ y) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int lane = threadIdx.x & 63, wave = uni((int32_t)(threadIdx.x >> 6));
  const int groups = kTokenWaves / P.ks, group = wave / P.ks, part = wave % P.ks;
  const int64_t col0 = ((int64_t)uni(blockIdx.x) * groups + group) * (NL * 16);
  TileLines<kModeLinear, NL> W;
  W.init(w_data, w_scale, 0, col0, n, k, lane);
  f32x4 acc[MT][NL];
  token_multiply<MT, NL>(W, P, x, k, tokens, wave, lane, lds, [](int i) { return (int64_t)i; }, acc);
  f32x4* red = reinterpret_cast<f32x4*>(lds);
  float* lv = reinterpret_cast<float*>(lds + kTokenWaves * MT * NL * 1024);  // [tokens][rank]: alpha * v of every row
  __syncthreads();
  for (int i = threadIdx.x; i < tokens * rank; i += kTokenThreads) {
    const int a = ids[i / rank];
    lv[i] = (uint32_t)a < (uint32_t)adapters ? row_v(v, parts, tokens, i / rank, rank, i % rank, a, alpha) : 0.0f;
  }
  join_waves<MT, NL>(acc, red, wave, lane);
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    if (mt * 16 >= tokens) continue;
#pragma unroll
    for (int c = 0; c < NL; ++c) {
      if ((mt * NL + c) % P.ks != part || col0 + 16 * c >= n) continue;
      const int64_t col = col0 + 16 * c + (lane & 15);
      const f32x4 sum = joined<MT, NL>(red, group, P.ks, mt, c, lane);
      const float s = w_amax[col] / 2688.0f;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int t = mt * 16 + 4 * (lane >> 4) + q;
        if (t >= tokens) continue;
        float r = sum[q] * s;
        const int a = adapters ? ids[t] : -1;
        if ((uint32_t)a < (uint32_t)adapters) {
          r += rank_dot(lora_b + ((int64_t)a * n + col) * rank, lv + t * rank, rank);
        }
        y[(int64_t)t * n + col] = to_bf16(r);
      }
    }
  }
}

// ----------------------------------------------------- projection, many rows

constexpr int kBM = 128, kBN = 256, kBK = 64;
constexpr int kIM = 4, kIN = 2;                     // 32 x 32 tiles of a wave: all 128 rows x 64 lines
constexpr uint32_t kXBytes = kBM * kBK * 2;         // 16 KB: 128 bytes a row
constexpr uint32_t kWBytes = kBN * kBK / 2;         // 8 KB: 32 bytes a line
constexpr uint32_t kStage = kXBytes + kWBytes;


// Tile of 128 rows x 256 lines, or one of gridDim.y parts of its contraction
// (SPLIT: fp32 sums to partial[blockIdx.y], for finish_kernel, which adds the
// adapters).  Copies run one step ahead; with SPLIT, where a CU may
// have one work-group alone and the latency sets the pace (2.3 us a step), two
// (with many tiles the third stage costs 2%).  Wave w takes all rows and lines 64 w .. + 63,
// so no weight is decoded twice in a work-group.  Element granules (8 of x,
// 16 bytes) and code granules are XOR-placed in LDS so that fragment reads of
// 32 consecutive rows or lines spread over the banks.  Rows past the last and
// elements past k read as zero (the weights' codes there, the next line's, are
// finite and meet zeros).
template <bool SPLIT>
__global__ __launch_bounds__(kThreads, 2) void many_rows_kernel(
    const uint16_t* __restrict__ x, int64_t tokens, int64_t k, const uint8_t* __restrict__ w_data,
    const uint8_t* __restrict__ w_scale, const float* __restrict__ w_amax, int64_t n,
    const uint16_t* __restrict__ lora_b, int adapters, int rank, const int32_t* __restrict__ ids,
    const uint16_t* __restrict__ v, uint32_t ntm, uint32_t ntn, uint16_t* __restrict__ y, float* __restrict__ partial) {
  __shared__ __attribute__((aligned(16))) uint8_t lds0[kStage];
  __shared__ __attribute__((aligned(16))) uint8_t lds1[kStage];
  __shared__ __attribute__((aligned(16))) uint8_t lds2[SPLIT ? kStage : 16];
  const int tid = threadIdx.x, wave = uni((int32_t)(tid >> 6)), lane = tid & 63, h = lane >> 5;
  // groups of 8 row tiles sweep the column tiles together, a run of tiles an XCD
  const uint32_t nb = gridDim.x, xcd = blockIdx.x % kNumXcd, q8 = nb / kNumXcd, r8 = nb % kNumXcd;
  const uint32_t lt = xcd * q8 + min(xcd, r8) + blockIdx.x / kNumXcd;
  const uint32_t grp = lt / (8 * ntn), gin = lt % (8 * ntn), gm = min(8u, ntm - 8 * grp);
  const int64_t row0 = (int64_t)uni(8 * grp + gin % gm) * kBM, col0 = (int64_t)uni(gin / gm) * kBN;
  const uint32_t rows = (uint32_t)min<int64_t>(tokens - row0, kBM), cols = (uint32_t)min<int64_t>(n - col0, kBN);
  const uint32_t dp = uni((uint32_t)(k / 2)), sp = uni((uint32_t)(k / 16)), xp = uni((uint32_t)(2 * k));
  const rsrc_t xs = range_rsrc(x + row0 * k, (int64_t)rows * xp);
  const rsrc_t wd = range_rsrc(w_data + col0 * dp, (int64_t)cols * dp);
  const rsrc_t ws = range_rsrc(w_scale + col0 * sp, (int64_t)cols * sp);
  const uint32_t steps = (uint32_t)((k + kBK - 1) / kBK), share = (steps + gridDim.y - 1) / gridDim.y;
  const uint32_t ks0 = SPLIT ? uni(min(blockIdx.y * share, steps)) : 0, nk = SPLIT ? uni(min(ks0 + share, steps)) : steps;

  // x: 32 rows a copy, lane g: slot g % 8 of row g / 8 (rows 32 apart have the
  // same granule); codes: 128 lines a copy, lane g: slot g % 2 of line g / 2.
  // In the last step a granule past k is moved out of the buffer's range.
  const uint32_t xgr = (tid & 7) ^ ((tid >> 3) & 7), xoff = (tid >> 3) * xp + 16 * xgr;
  const uint32_t woff = (tid >> 1) * dp + 16 * ((tid & 1) ^ ((tid >> 3) & 1));
  const uint32_t past = (steps - 1) * kBK + 8 * xgr < (uint32_t)k ? 0u : kOutOfRange;
  auto issue = [&](uint32_t ks, uint8_t* base) {
    const uint32_t off = ks + 1 == steps ? xoff | past : xoff;
#pragma unroll
    for (int c = 0; c < kBM / 32; ++c)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(xs, (lds_ptr_t)(base + 16 * (c * kThreads + wave * 64)), 16,
                                               off + 32 * c * xp, ks * (2 * kBK), 0, 0);
#pragma unroll
    for (int c = 0; c < kBN / 128; ++c)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(wd, (lds_ptr_t)(base + kXBytes + 16 * (c * kThreads + wave * 64)), 16,
                                               woff + 128 * c * dp, ks * (kBK / 2), 0, 0);
  };
  // Scales of a step, two bytes a line for each lane half (blocks 2h, 2h + 1),
  // fetched with the step's copies: a line's scales may start on any even byte.
  uint32_t sc0[kIN], sc1[kIN], sc2[kIN];
  auto fetch_scales = [&](uint32_t ks, uint32_t (&sc)[kIN]) {
#pragma unroll
    for (int in = 0; in < kIN; ++in)
      sc[in] = __builtin_amdgcn_raw_buffer_load_b16(ws, (wave * 64 + in * 32 + (lane & 31)) * sp + 2 * h, ks * (kBK / 16),
                                                    0);
  };

  f32x16 acc[kIM][kIN];
#pragma unroll
  for (int im = 0; im < kIM; ++im)
#pragma unroll
    for (int in = 0; in < kIN; ++in) acc[im][in] = f32x16{};
  constexpr uint32_t kAhead = SPLIT ? 2 : 1;
  constexpr int kCopies = kBM / 32 + kBN / 128 + kIN;  // vector-memory operations of a step
  auto step = [&](uint32_t ks, const uint8_t* base, const uint32_t (&sc)[kIN], uint8_t* next, uint32_t (&next_sc)[kIN]) {
    // this step's own copies: those of the next step, if under way, may go on
    if (SPLIT && ks + 1 < nk) __builtin_amdgcn_s_waitcnt(waitcnt_vm(kCopies));
    else __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
    __syncthreads();
    float sv[kIN][2];
#pragma unroll
    for (int in = 0; in < kIN; ++in) {
      sv[in][0] = e4m3_value(sc[in] & 0xFFu);
      sv[in][1] = e4m3_value((sc[in] >> 8) & 0xFFu);
    }
    if (ks + kAhead < nk) {
      issue(ks + kAhead, next);
      fetch_scales(ks + kAhead, next_sc);
    }
    u32x4 wq[kIN];
#pragma unroll
    for (int in = 0; in < kIN; ++in) {
      const uint32_t line = wave * 64 + in * 32 + (lane & 31);
      wq[in] = *reinterpret_cast<const u32x4*>(base + kXBytes + 32 * line + 16 * (h ^ ((line >> 2) & 1)));
    }
    // Sub-step s, lane half h: the 8 elements of word 4h + s.  The next
    // sub-step's fragments are read and decoded between this one's MFMAs (one
    // MFMA to four VALU instructions: 32 decode a sub-step's two line tiles).
    bf16x8 xf[2][kIM], wf[2][kIN];
    auto fetch = [&](int s) {
#pragma unroll
      for (int im = 0; im < kIM; ++im) {
        const uint32_t row = im * 32 + (lane & 31);
        xf[s & 1][im] = *reinterpret_cast<const bf16x8*>(base + 128 * row + 16 * ((4 * h + s) ^ (row & 7)));
      }
#pragma unroll
      for (int in = 0; in < kIN; ++in) wf[s & 1][in] = decode8_bf16(wq[in][s], sv[in][s >> 1]);
    };
    fetch(0);
#pragma unroll
    for (int s = 0; s < kBK / 16; ++s) {
      if (s + 1 < kBK / 16) fetch(s + 1);
#pragma unroll
      for (int in = 0; in < kIN; ++in)
#pragma unroll
        for (int im = 0; im < kIM; ++im)
          acc[im][in] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(xf[s & 1][im], wf[s & 1][in], acc[im][in], 0, 0, 0);
      if (s + 1 < kBK / 16) {
        __builtin_amdgcn_sched_group_barrier(0x100, kIM, 0);  // the fragment reads
#pragma unroll
        for (int i = 0; i < kIM * kIN; ++i) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // one MFMA
          __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);  // four VALU
        }
      }
    }
  };
  uint32_t ks = ks0;
  if (ks < nk) {
    issue(ks, lds0);
    fetch_scales(ks, sc0);
  }
  if constexpr (SPLIT) {
    if (ks + 1 < nk) {
      issue(ks + 1, lds1);
      fetch_scales(ks + 1, sc1);
    }
#pragma unroll 1
    for (; ks + 2 < nk; ks += 3) {
      step(ks, lds0, sc0, lds2, sc2);
      step(ks + 1, lds1, sc1, lds0, sc0);
      step(ks + 2, lds2, sc2, lds1, sc1);
    }
    if (ks < nk) step(ks, lds0, sc0, lds2, sc2);
    if (ks + 1 < nk) step(ks + 1, lds1, sc1, lds0, sc0);
  } else {
#pragma unroll 1
    for (; ks + 1 < nk; ks += 2) {
      step(ks, lds0, sc0, lds1, sc1);
      step(ks + 1, lds1, sc1, lds0, sc0);
    }
    if (ks < nk) step(ks, lds0, sc0, lds1, sc1);
  }

  const uint32_t jw = wave * 64;  // first line of the wave in the tile
  const uint32_t yp = (uint32_t)(2 * n);
  float lf[kIN];
#pragma unroll
  for (int in = 0; in < kIN; ++in) {
    const uint32_t j = jw + in * 32 + (lane & 31);
    lf[in] = j < cols ? w_amax[col0 + j] / 2688.0f : 0.0f;
  }
  // Rows past the last are out of the output buffer's range, columns past the
  // last are moved out of it.
  if constexpr (SPLIT) {
    const rsrc_t ps = range_rsrc(partial + ((int64_t)blockIdx.y * tokens + row0) * n + col0,
                                 ((int64_t)rows - 1) * 2 * yp + 4 * cols);
#pragma unroll
    for (int in = 0; in < kIN; ++in) {
      const uint32_t j = jw + in * 32 + (lane & 31), off = j < cols ? 8 * h * yp + 4 * j : kOutOfRange;
#pragma unroll
      for (int im = 0; im < kIM; ++im)
#pragma unroll
        for (int q = 0; q < 16; ++q)
          __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(acc[im][in][q] * lf[in]), ps,
                                                off + (im * 32 + 8 * (q >> 2) + (q & 3)) * 2 * yp, 0, 0);
    }
    return;
  }
  // Every adapter that one of 32 rows has adds rank/16 MFMA steps of v B_a^T.
  // Rows of other adapters meet B_a only as zeros, but a B_a that is not finite
  // must not reach them either: each adapter's product is formed apart and
  // added to its own rows alone.  The loads of 32 ranks are in flight together.
  const uint32_t r16 = round16(rank);
  const rsrc_t vh = range_rsrc(v + row0 * r16, (int64_t)rows * r16 * 2);
  const rsrc_t vl = range_rsrc(v + (tokens + row0) * r16, (int64_t)rows * r16 * 2);
  const rsrc_t ys = range_rsrc(y + row0 * n + col0, ((int64_t)rows - 1) * yp + 2 * cols);
  const bool odd = lane & 1;
#pragma unroll
  for (int im = 0; im < kIM; ++im) {
    const uint32_t row = im * 32 + (lane & 31);
    const int my = adapters && row < rows ? ids[row0 + row] : -1;
    uint32_t left = (uint32_t)__ballot((uint32_t)my < (uint32_t)adapters);  // lanes 32-63 repeat lanes 0-31
    f32x16 sum[kIN];
#pragma unroll
    for (int in = 0; in < kIN; ++in) sum[in] = f32x16{};
#pragma unroll 1
    while (left) {
      const int a = __builtin_amdgcn_readlane(my, (int)__builtin_ctz(left));
      const uint32_t own = (uint32_t)__ballot(my == a);
      left &= ~own;
      const rsrc_t bs = range_rsrc(lora_b + ((int64_t)a * n + col0) * rank, (int64_t)cols * rank * 2);
      const uint32_t voff = my == a ? row * r16 * 2 + 16 * h : kOutOfRange;
      f32x16 part[kIN];
#pragma unroll
      for (int in = 0; in < kIN; ++in) part[in] = f32x16{};
#pragma unroll 1
      for (uint32_t r = 0; r < r16; r += 32) {
        u32x4 b[2][kIN], hi[2], lo[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t rr = r + 16 * i, bin = rr + 8 * h < (uint32_t)rank ? 0u : kOutOfRange;
#pragma unroll
          for (int in = 0; in < kIN; ++in)
            b[i][in] = __builtin_amdgcn_raw_buffer_load_b128(
                bs, ((jw + in * 32 + (lane & 31)) * rank * 2 + 16 * h + 2 * rr) | bin, 0, 0);
          const uint32_t vo = rr < r16 ? voff + 2 * rr : kOutOfRange;
          hi[i] = __builtin_amdgcn_raw_buffer_load_b128(vh, vo, 0, 0);
          lo[i] = __builtin_amdgcn_raw_buffer_load_b128(vl, vo, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int in = 0; in < kIN; ++in) {
            const bf16x8 bf = __builtin_bit_cast(bf16x8, b[i][in]);
            part[in] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, hi[i]), bf, part[in], 0, 0, 0);
            part[in] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, lo[i]), bf, part[in], 0, 0, 0);
          }
      }
#pragma unroll
      for (int in = 0; in < kIN; ++in)
#pragma unroll
        for (int q = 0; q < 16; ++q) sum[in][q] += (own >> (8 * (q >> 2) + 4 * h + (q & 3))) & 1 ? part[in][q] : 0.0f;
    }
#pragma unroll
    for (int in = 0; in < kIN; ++in) {
      const uint32_t jp = (jw + in * 32 + (lane & 31)) & ~1u;
      const uint32_t off = jp < cols ? (im * 32 + 4 * h + odd) * yp + 2 * jp : kOutOfRange;
#pragma unroll
      for (int q = 0; q < 16; q += 2) {
        float lo, hi;
        pair_columns(acc[im][in][q] * lf[in] + sum[in][q], acc[im][in][q + 1] * lf[in] + sum[in][q + 1], odd, &lo, &hi);
        __builtin_amdgcn_raw_buffer_store_b32(pack_bf16(lo, hi), ys, off + (8 * (q >> 2) + (q & 3)) * yp, 0, 0);
      }
    }
  }
}

// y[t] = the sum of the parts, in their order, plus the row's adapter, rounded
// once.  A work-group takes kThreads * 8 columns of a row.
__global__ __launch_bounds__(kThreads) void finish_kernel(const float* __restrict__ partial, int parts, int64_t tokens,
                                                          int64_t n, const uint16_t* __restrict__ lora_b,
                                                          const float* __restrict__ alpha, int adapters, int rank,
                                                          const int32_t* __restrict__ ids, const float* __restrict__ v,
                                                          int v_parts, uint16_t* __restrict__ y) {
  __shared__ __attribute__((aligned(16))) float lv[LORA_MAX_RANK];
  const int64_t t = blockIdx.x, c = ((int64_t)blockIdx.y * kThreads + threadIdx.x) * 8;
  const int a = adapters ? uni(ids[t]) : -1;
  const bool adapted = (uint32_t)a < (uint32_t)adapters;
  if (adapted && (int)threadIdx.x < rank) lv[threadIdx.x] = row_v(v, v_parts, tokens, t, rank, threadIdx.x, a, alpha);
  __syncthreads();
  if (c >= n) return;
  const int64_t count = tokens * n, i = t * n + c;
  f32x4 s0 = *reinterpret_cast<const f32x4*>(partial + i), s1 = *reinterpret_cast<const f32x4*>(partial + i + 4);
  for (int p = 1; p < parts; ++p) {
    s0 += *reinterpret_cast<const f32x4*>(partial + p * count + i);
    s1 += *reinterpret_cast<const f32x4*>(partial + p * count + i + 4);
  }
  float o[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    o[q] = q < 4 ? s0[q] : s1[q - 4];
    if (adapted) o[q] += rank_dot(lora_b + ((int64_t)a * n + c + q) * rank, lv, rank);
  }
  *reinterpret_cast<u32x4*>(y + i) = u32x4{pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]), pack_bf16(o[4], o[5]),
                                          pack_bf16(o[6], o[7])};
}

// ------------------------------------------------------------- host side

// Parts of the contraction of the first launch: enough work-groups for the
// device, at least one step a wave.
int shrink_parts(int64_t tokens, int64_t k) {
  const int64_t tiles = (tokens + kShrinkRows - 1) / kShrinkRows, steps = (k + kShrinkStep - 1) / kShrinkStep;
  const int64_t want = (4 * kCus + tiles - 1) / tiles;
  return (int)std::max<int64_t>(1, std::min(std::min(want, (steps + 3) / 4), (int64_t)kMaxSplit));
}

constexpr int64_t round256(int64_t b) { return (b + 255) / 256 * 256; }
// Workspace: the parts of v; for many rows its halves; the parts of the projection.
int64_t v_bytes(int64_t tokens, int64_t k, int32_t rank) { return round256(tokens * rank * 4 * shrink_parts(tokens, k)); }
int64_t half_bytes(int64_t tokens, int32_t rank) { return tokens <= kFewRows ? 0 : round256(tokens * round16(rank) * 4); }

// Parts of the contraction of many rows: as many as give every CU two
// work-groups where the tiles alone do not give it one, at least 8 steps each,
// and their sums within kMaxWorkspace.
constexpr int64_t kMaxWorkspace = 24 << 20;
int project_parts(int64_t tokens, int64_t k, int64_t n) {
  const int64_t tiles = ((tokens + kBM - 1) / kBM) * ((n + kBN - 1) / kBN);
  if (tokens <= kFewRows || tiles >= kCus) return 1;
  const int64_t by_steps = (k + kBK - 1) / kBK / 8, by_room = kMaxWorkspace / (tokens * n * 4);
  return (int)std::max<int64_t>(1, std::min(std::min(2 * kCus / tiles, by_steps), by_room));
}

template <class F>
void with_ranks(int rank, F f) {
  if (rank <= 16) f(std::integral_constant<int, 1>());
  else if (rank <= 32) f(std::integral_constant<int, 2>());
  else if (rank <= 64) f(std::integral_constant<int, 4>());
  else f(std::integral_constant<int, 8>());
}

template <int MT, int NL>
void launch_few(const uint16_t* x, int tokens, int64_t k, const uint8_t* wd, const uint8_t* ws, const float* wa,
                int64_t n, const uint16_t* b, const float* alpha, int adapters, int rank, const int32_t* ids,
                const float* v, int parts, uint16_t* y, hipStream_t st) {
  int ks = 1;
  while (ks < 8 && (n + 16 * NL * (8 / ks) - 1) / (16 * NL * (8 / ks)) < 200) ks *= 2;
  const TokenPlan P = token_plan(k, tokens, ks, MT * NL, adapters ? (int64_t)tokens * rank * 4 : 0,
                                 (n + 16 * NL * (8 / ks) - 1) / (16 * NL * (8 / ks)));
  const int cols = NL * 16 * (kTokenWaves / P.ks);
  hipLaunchKernelGGL((few_rows_kernel<MT, NL>), dim3((uint32_t)((n + cols - 1) / cols)), dim3(kTokenThreads), P.lds, st, x,
                     tokens, k, wd, ws, wa, n, b, alpha, adapters, adapters ? rank : 0, ids, v, parts, P, y);
}

}  // namespace

extern "C" {

int64_t lora_workspace(int64_t tokens, int64_t k, int64_t n, int32_t rank) {
  if (tokens <= 0 || k <= 0 || n <= 0 || rank < 0) return 0;
  const int parts = project_parts(tokens, k, n);
  return v_bytes(tokens, k, rank) + half_bytes(tokens, rank) + (parts > 1 ? parts * tokens * n * 4 : 0);
}

int lora_linear(const uint16_t* x, int64_t tokens, int64_t k, const uint8_t* w_data, const uint8_t* w_scale,
                const float* w_amax, int64_t n, const uint16_t* lora_a, const uint16_t* lora_b, const float* alpha,
                int32_t num_adapters, int32_t rank, const int32_t* adapter_ids, uint16_t* y, void* workspace,
                int64_t workspace_bytes, void* stream) {
  if (k <= 0 || k % 32 != 0 || k > kMaxK || n <= 0 || n % 16 != 0 || n > (1 << 20)) return NVFP4G_EINVAL;
  if (tokens < 0 || tokens > kMaxRows || num_adapters < 0) return NVFP4G_EINVAL;
  if (num_adapters && (rank <= 0 || rank % 8 != 0 || rank > LORA_MAX_RANK)) return NVFP4G_EINVAL;
  if (tokens == 0) return NVFP4G_OK;
  if (!x || !w_data || !w_scale || !w_amax || !y) return NVFP4G_EINVAL;
  if (num_adapters && (!lora_a || !lora_b || !alpha || !adapter_ids)) return NVFP4G_EINVAL;
  if (!aligned(x, 16) || !aligned(w_data, 16) || !aligned(w_scale, 16) || !aligned(w_amax, 4) || !aligned(y, 16) ||
      !aligned(lora_a, 16) || !aligned(lora_b, 16) || !aligned(alpha, 4) || !aligned(adapter_ids, 4) ||
      !aligned(workspace, 16))
    return NVFP4G_EALIGN;
  const int64_t need = lora_workspace(tokens, k, n, num_adapters ? rank : 0);
  if (need && (!workspace || workspace_bytes < need)) return NVFP4G_EINVAL;
  const hipStream_t st = (hipStream_t)stream;
  const int T = (int)tokens, parts = shrink_parts(tokens, k), r = num_adapters ? rank : 0;
  const bool few = tokens <= kFewRows;
  const int split = project_parts(tokens, k, n);
  float* v = (float*)workspace;
  uint16_t* halves = (uint16_t*)((char*)workspace + v_bytes(tokens, k, r));
  float* partial = (float*)((char*)halves + half_bytes(tokens, r));
  if (((tokens + kBM - 1) / kBM) * ((n + kBN - 1) / kBN) > (int64_t)INT32_MAX) return NVFP4G_EINVAL;
  if (num_adapters) {
    const dim3 grid((uint32_t)((T + kShrinkRows - 1) / kShrinkRows), parts, std::min(std::min(T, kShrinkRows), num_adapters));
    with_ranks(rank, [&](auto nr) {
      hipLaunchKernelGGL((shrink_kernel<decltype(nr)::value>), grid, dim3(kThreads), 0, st, x, T, k, lora_a,
                         num_adapters, rank, adapter_ids, v);
    });
    if (split == 1 && !few)
      hipLaunchKernelGGL(halves_kernel, dim3((uint32_t)((tokens * round16(rank) + kThreads - 1) / kThreads)),
                         dim3(kThreads), 0, st, v, parts, tokens, rank, alpha, num_adapters, adapter_ids, halves);
  }
  if (few) {
    // one 16-line tile a work-group: the most work-groups a projection gives
    if (T <= 16) launch_few<1, 1>(x, T, k, w_data, w_scale, w_amax, n, lora_b, alpha, num_adapters, rank, adapter_ids, v, parts, y, st);
    else if (T <= 32) launch_few<2, 1>(x, T, k, w_data, w_scale, w_amax, n, lora_b, alpha, num_adapters, rank, adapter_ids, v, parts, y, st);
    else launch_few<4, 1>(x, T, k, w_data, w_scale, w_amax, n, lora_b, alpha, num_adapters, rank, adapter_ids, v, parts, y, st);
  } else {
    const uint32_t ntm = (uint32_t)((tokens + kBM - 1) / kBM), ntn = (uint32_t)((n + kBN - 1) / kBN);
    if (split > 1) {
      hipLaunchKernelGGL((many_rows_kernel<true>), dim3(ntm * ntn, split), dim3(kThreads), 0, st, x, tokens, k, w_data,
                         w_scale, w_amax, n, lora_b, num_adapters, r, adapter_ids, halves, ntm, ntn, y, partial);
      hipLaunchKernelGGL(finish_kernel, dim3((uint32_t)tokens, (uint32_t)((n + 8 * kThreads - 1) / (8 * kThreads))),
                         dim3(kThreads), 0, st, partial, split, tokens, n, lora_b, alpha, num_adapters, r, adapter_ids,
                         v, parts, y);
    } else {
      hipLaunchKernelGGL((many_rows_kernel<false>), dim3(ntm * ntn), dim3(kThreads), 0, st, x, tokens, k, w_data,
                         w_scale, w_amax, n, lora_b, num_adapters, r, adapter_ids, halves, ntm, ntn, y, partial);
    }
  }
  return hip_status();
}

}  // extern "C"
