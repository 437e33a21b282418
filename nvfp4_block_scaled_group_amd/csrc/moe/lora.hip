// lora.hip -- low-rank adapters of many requests beside one shared NVFP4
// projection, behind the C ABI of include/moe_ops.h:
//
//   y[t] = W x[t] + alpha_a B_a (A_a x[t]),   a = adapter of row t.
//
// The first launch makes v[t] = A_a x[t] (rank values a row): a work-group
// takes 16 rows and multiplies them (MFMA 16x16x32) by one of the adapters
// that any of them has.  Then the shared projection follows, with the adapters
// in its epilogue:
//   few rows (at most 32)  the weight is read once and bounds it; every
//                          16-line tile adds its rows' B_a v in fp32;
//   more rows              128 x 256 tiles, MFMA 32x32x16; each adapter present
//                          in 32 rows of the tile adds rank/16 MFMA steps of
//                          v B_a^T to its own rows of the scaled accumulators;
//                          where tiles are few, parts of the contraction, and
//                          a last launch that adds them and the adapters.
// 32 rows are one pass over the weight in the first form: 17 rows of 7168 x 7168
// take 24 us, 32 rows 28; in the second 36 and 37.
// Measured: 8 rows, 7168 x 7168, 6 adapters of rank 16: 19 us (1.6 TB/s; the
// latency of a wave's seven steps after the first launch's 5 us); 4095 rows,
// 7168 x 2048, 8 adapters of rank 32: 167 to 171 us (0.73 PFLOP/s; MFMA and decode).
// v is kept in fp32, or, where the second launch multiplies it by MFMA, as three
// bf16 pieces of 8 significant bits whose sum is the fp32 value (4096 rows of 32
// adapters of rank 64: 223 us; with two pieces, 16 bits, 214).
#include "moe_token.hpp"

namespace {

using namespace moe;

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kFewRows = 32;      // rows of the first form
constexpr int kShrinkRows = 16;   // rows of a work-group of the first launch
constexpr int kMaxSplit = 8;      // parts of the contraction over work-groups (few rows)
constexpr int kShrinkThreads = 512, kShrinkWaves = kShrinkThreads / 64;
constexpr int kShrinkStep = 128;  // contraction step of a wave of the first launch

constexpr int kPieces = 3;        // bf16 pieces of an fp32 value: 24 significant bits

constexpr int round16(int r) { return (r + 15) / 16 * 16; }

// ------------------------------------------------------------- row order

// Rows in windows of kWindow are put in the order of their adapters (stable,
// no adapter last), so that a tile of the next launches has few of them even
// where every row is another request.  A work-group ranks 64 rows, four lanes
// a row: each compares it with a quarter of the window, in LDS.
constexpr int kWindow = 1024;
constexpr int kOrderRows = kThreads / 4;
__global__ __launch_bounds__(kThreads) void order_kernel(const int32_t* __restrict__ ids, int tokens, int adapters,
                                                         int32_t* __restrict__ order) {
  __shared__ __attribute__((aligned(16))) uint32_t key[kWindow];
  const int tid = threadIdx.x, first = uni((int32_t)blockIdx.x) * kOrderRows, row0 = first / kWindow * kWindow;
  const int count = min(tokens - row0, kWindow), quarter = (count + 15) / 16 * 4;
  // adapter and place in one number: all different, and the rank a count
  for (int j = tid; j < 4 * quarter; j += kThreads) {
    uint32_t v = 0xFFFFFFFFu;  // past the last row
    if (j < count) v = min((uint32_t)ids[row0 + j], (uint32_t)adapters) * kWindow + j;
    key[j] = v;
  }
  __syncthreads();
  const int i = first - row0 + (tid >> 2), part = tid & 3;
  const uint32_t mine = i < count ? key[i] : 0u;
  uint32_t rank = 0;
#pragma unroll 8
  for (int j = part * quarter; j < (part + 1) * quarter; j += 4) {
    const u32x4 q = *reinterpret_cast<const u32x4*>(key + j);
#pragma unroll
    for (int c = 0; c < 4; ++c) rank += q[c] < mine;
  }
  rank += dpp_x1(rank);
  rank += dpp_x2(rank);
  if (part == 0 && i < count) order[row0 + rank] = row0 + i;
}

// ---------------------------------------------------------------- A_a x[t]

// blockIdx = (tile of 16 rows in `order`, or as they are if that is NULL, part
// of the contraction, first of the tile's adapters that it takes).  v [parts][tokens][rank]
// fp32, or with PIECES (one part) alpha * v as kPieces bf16 tables [tokens][rank
// rounded up to 16], zeros past the rank.  Rows without an adapter are not
// written.  The waves take a share of the part each and join
// in LDS.  A step's loads are in flight together; parts and adapters are
// work-groups of their own because the chain of steps, not the bytes, is what
// takes the time: 5 us for 8 rows of 7168, 17 to 19 for 4095 rows of 2048 (two
// bytes an element of x: 0.9 TB/s).
template <int NR, bool PIECES>
__global__ __launch_bounds__(kShrinkThreads) void shrink_kernel(const uint16_t* __restrict__ x, int tokens, int64_t k,
                                                          const uint16_t* __restrict__ lora_a,
                                                          const float* __restrict__ alpha, int adapters, int rank,
                                                          const int32_t* __restrict__ ids,
                                                          const int32_t* __restrict__ order, void* __restrict__ v) {
  __shared__ f32x4 red[kShrinkWaves * NR * 64];
  __shared__ int32_t token[kShrinkRows];
  const int lane = threadIdx.x & 63, wave = uni((int32_t)(threadIdx.x >> 6));
  const int row0 = uni((int32_t)blockIdx.x) * kShrinkRows;
  const int pos = min(row0 + (lane & 15), tokens - 1), t = order ? order[pos] : pos;  // lanes 16 apart share a row
  if (threadIdx.x < kShrinkRows) token[threadIdx.x] = t;
  const int my = lane < kShrinkRows && row0 + lane < tokens ? ids[t] : -1;
  uint64_t left = __ballot((uint32_t)my < (uint32_t)adapters && lane < kShrinkRows);
  const int parts = uni((int32_t)gridDim.y) * kShrinkWaves, part = uni((int32_t)blockIdx.y) * kShrinkWaves + wave;
  const int64_t steps = (k + kShrinkStep - 1) / kShrinkStep, share = (steps + parts - 1) / parts;
  const int64_t s0 = min<int64_t>(part * share, steps), s1 = min<int64_t>(s0 + share, steps);
  const uint16_t* xr = x + (int64_t)t * k;
  for (int slot = 0; left; ++slot) {
    const int a = __builtin_amdgcn_readlane(my, (int)__builtin_ctzll(left));
    const uint64_t rows = __ballot(my == a) & left;
    left &= ~rows;
    if (slot % (int)gridDim.z != (int)blockIdx.z) continue;
    f32x4 acc[NR];
    const uint16_t* ar[NR];  // this lane's line of each 16 ranks (a line past the rank reads the last)
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      acc[r] = f32x4{0, 0, 0, 0};
      ar[r] = lora_a + ((int64_t)a * rank + min(16 * r + (lane & 15), rank - 1)) * k;
    }
    constexpr int D = NR <= 2 ? 2 : 1;  // steps in flight (5883 rows of 2688: 3 us less with two; more ranks fill the registers)
    for (int64_t s = s0; s < s1; s += D) {
      u32x4 xq[D][4], aq[D][NR][4];
#pragma unroll
      for (int d = 0; d < D; ++d) {
        const int64_t e0 = (s + d) * kShrinkStep + 32 * (lane >> 4);
        const bool in = e0 < k && s + d < s1;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          xq[d][q] = in ? *reinterpret_cast<const u32x4*>(xr + e0 + 8 * q) : u32x4{0, 0, 0, 0};
#pragma unroll
          for (int r = 0; r < NR; ++r)
            aq[d][r][q] = in ? *reinterpret_cast<const u32x4*>(ar[r] + e0 + 8 * q) : u32x4{0, 0, 0, 0};
        }
      }
#pragma unroll
      for (int d = 0; d < D; ++d)
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int r = 0; r < NR; ++r)
            acc[r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, xq[d][q]),
                                                             __builtin_bit_cast(bf16x8, aq[d][r][q]), acc[r], 0, 0, 0);
    }
#pragma unroll
    for (int r = 0; r < NR; ++r) red[(wave * NR + r) * 64 + lane] = acc[r];
    __syncthreads();
    // thread -> (row, rank column); element (row, col) of a tile is component
    // row % 4 of lane 16 (row / 4) + col
    const int row = threadIdx.x >> 4, col = threadIdx.x & 15;
    if (row < kShrinkRows && ((rows >> row) & 1)) {
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const float* f = reinterpret_cast<const float*>(red) + (r * 64 + 16 * (row >> 2) + col) * 4 + (row & 3);
        float sum = f[0];
#pragma unroll
        for (int w = 1; w < kShrinkWaves; ++w) sum += f[w * NR * 64 * 4];
        const int c = 16 * r + col;
        if (PIECES) {
          const int r16 = round16(rank);
          if (c >= r16) break;
          float w = c < rank ? sum * alpha[a] : 0.0f;
          uint16_t* o = reinterpret_cast<uint16_t*>(v) + (int64_t)token[row] * r16 + c;
#pragma unroll
          for (int i = 0; i < kPieces; ++i, o += (int64_t)tokens * r16) {
            // cut off, not rounded: the rest is exact and nothing overflows
            const uint32_t top = __float_as_uint(w) & 0xFFFF0000u;
            *o = (uint16_t)(top >> 16);
            w = __builtin_isfinite(w) ? w - __uint_as_float(top) : 0.0f;
          }
        } else if (c < rank) {
          reinterpret_cast<float*>(v)[((int64_t)blockIdx.y * tokens + token[row]) * rank + c] = sum;
        }
      }
    }
    if (left) __syncthreads();  // red is written again
  }
}

// Ranks i .. i + 31 of a line of B (past the rank not read, and not used).
__device__ __forceinline__ void rank_load(const uint16_t* b, int i, int rank, u32x4 (&q)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (i + 8 * j < rank) q[j] = *reinterpret_cast<const u32x4*>(b + i + 8 * j);
}

// d + the sum of up to 32 ranks q[r] * v[r], in their order, in fp32.
__device__ __forceinline__ float rank_sum(const u32x4 (&q)[4], const float* v, int ranks, float d) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (8 * j >= ranks) break;
    const f32x4 lo = *reinterpret_cast<const f32x4*>(v + 8 * j), hi = *reinterpret_cast<const f32x4*>(v + 8 * j + 4);
    d = __builtin_fmaf(bf16lo(q[j][0]), lo[0], d);
    d = __builtin_fmaf(bf16hi(q[j][0]), lo[1], d);
    d = __builtin_fmaf(bf16lo(q[j][1]), lo[2], d);
    d = __builtin_fmaf(bf16hi(q[j][1]), lo[3], d);
    d = __builtin_fmaf(bf16lo(q[j][2]), hi[0], d);
    d = __builtin_fmaf(bf16hi(q[j][2]), hi[1], d);
    d = __builtin_fmaf(bf16lo(q[j][3]), hi[2], d);
    d = __builtin_fmaf(bf16hi(q[j][3]), hi[3], d);
  }
  return d;
}

// d + the ranks from `from` (a multiple of 32) on of a line of B times v; the
// loads of 32 ranks are in flight together.
__device__ __forceinline__ float rank_dot(const uint16_t* b, const float* v, int from, int rank, float d) {
  for (int i = from; i < rank; i += 32) {
    u32x4 q[4];
    rank_load(b, i, rank, q);
    d = rank_sum(q, v + i, rank - i, d);
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

// ------------------------------------------------------ projection, few rows

// The weight is read once (15 us for 7168 x 7168 and 8 rows, 1.9 TB/s: a wave has
// seven steps of it, and the start and the end are half of the time).
// Wave part p of a tile finishes the outputs whose number (token tile, row of
// four) is p, p + ks, ...  What its first one needs of B is loaded before the
// weights, and v of all rows beside them.
template <int MT>
__global__ __launch_bounds__(kTokenThreads, token_waves(MT)) void few_rows_kernel(
    const uint16_t* __restrict__ x, int tokens, int64_t k, const uint8_t* __restrict__ w_data,
    const uint8_t* __restrict__ w_scale, const float* __restrict__ w_amax, int64_t n,
    const uint16_t* __restrict__ lora_b, const float* __restrict__ alpha, int adapters, int rank,
    const int32_t* __restrict__ ids, const float* __restrict__ v, int parts, TokenPlan P, uint16_t* __restrict__ y) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int lane = threadIdx.x & 63, wave = uni((int32_t)(threadIdx.x >> 6));
  const int groups = kTokenWaves / P.ks, group = wave / P.ks, part = wave % P.ks;
  const int64_t col0 = ((int64_t)uni(blockIdx.x) * groups + group) * 16, col = col0 + (lane & 15);
  auto row_of = [&](int item) { return 16 * (item >> 2) + 4 * (lane >> 4) + (item & 3); };
  auto adapter_of = [&](int t) { return adapters && t < tokens && col0 < n ? ids[t] : -1; };
  auto line_of = [&](int a) { return lora_b + ((int64_t)a * n + col) * rank; };
  u32x4 first[4];
  const int first_a = adapter_of(row_of(part));
  if ((uint32_t)first_a < (uint32_t)adapters) rank_load(line_of(first_a), 0, rank, first);
  const float factor = w_amax[min<int64_t>(col, n - 1)];
  TileLines<kModeLinear, 1> W;
  W.init(w_data, w_scale, 0, col0, n, k, lane);
  f32x4 acc[MT][1];
  float* lv = reinterpret_cast<float*>(lds + P.shared);  // [tokens][rank]: alpha * v of every row
  token_multiply<MT, 1>(W, P, x, k, tokens, wave, lane, lds, [](int i) { return (int64_t)i; }, acc, [&] {
    for (int i = threadIdx.x; i < tokens * rank; i += kTokenThreads) {
      const int a = ids[i / rank];
      lv[i] = (uint32_t)a < (uint32_t)adapters ? row_v(v, parts, tokens, i / rank, rank, i % rank, a, alpha) : 0.0f;
    }
  });
  f32x4* red = reinterpret_cast<f32x4*>(lds);
  join_waves<MT, 1>(acc, red, wave, lane);
  if (col0 >= n) return;
  for (int item = part; item < 4 * MT; item += P.ks) {
    const int t = row_of(item);
    if (t >= tokens) continue;
    const float* f = reinterpret_cast<const float*>(red + (group * P.ks * MT + (item >> 2)) * 64 + lane) + (item & 3);
    float r = f[0];
    for (int w = 1; w < P.ks; ++w) r += f[w * MT * 64 * 4];
    r *= factor / 2688.0f;
    const int a = item == part ? first_a : adapter_of(t);
    if ((uint32_t)a < (uint32_t)adapters) {
      const float* l = lv + t * rank;
      r += item == part ? rank_dot(line_of(a), l, 32, rank, rank_sum(first, l, rank, 0.0f))
                        : rank_dot(line_of(a), l, 0, rank, 0.0f);
    }
    y[(int64_t)t * n + col] = to_bf16(r);
  }
}

// ----------------------------------------------------- projection, many rows

constexpr int kBM = 128, kBK = 64;
constexpr int kIM = 4;                              // 32 x 32 tiles of a wave: all 128 rows x kIN blocks of lines
constexpr uint32_t kXBytes = kBM * kBK * 2;         // 16 KB: 128 bytes a row
template <int IN>
constexpr uint32_t kStageOf = kXBytes + 128 * IN * kBK / 2;  // and 32 bytes a line: 24 KB, 20 KB

// Tile of 128 rows x 128 kIN lines, or one of gridDim.y parts of its contraction
// (SPLIT: fp32 sums to partial[blockIdx.y], for finish_kernel, which adds the
// adapters).  Copies run one step ahead.  With SPLIT, where a CU may have one
// work-group alone and the latency sets the pace (2.3 us a step), a third stage
// lets them be asked for two steps ahead; but the barrier of a step waits for
// all copies into LDS that are out, those of the next step too, so that they
// still get one step's time (with many tiles the third stage costs 2%).  Wave w
// takes all rows and 32 kIN lines, so no weight is decoded twice in a work-group.
// What bounds it is the MFMAs and the decode between them: 4095 rows, 7168 x
// 2048 in 152 us, 0.8 PFLOP/s (174 over and over, as the clock falls).
// Element granules (8 of x, 16 bytes) and code granules are XOR-placed in LDS so
// that fragment reads of 32 consecutive rows or lines spread over the banks.
// Rows past the last and elements past k read as zero.  The weights' codes past
// k, in the second half of a last step, are the next line's; their scales, which
// may not be numbers, read as zero.
template <bool SPLIT, int kIN>
__global__ __launch_bounds__(kThreads, 2) void many_rows_kernel(
    const uint16_t* __restrict__ x, int64_t tokens, int64_t k, const uint8_t* __restrict__ w_data,
    const uint8_t* __restrict__ w_scale, const float* __restrict__ w_amax, int64_t n,
    const uint16_t* __restrict__ lora_b, int adapters, int rank, const int32_t* __restrict__ ids,
    const int32_t* __restrict__ order, const uint16_t* __restrict__ v, uint32_t ntm, uint32_t ntn, uint16_t* __restrict__ y, float* __restrict__ partial) {
  __shared__ __attribute__((aligned(16))) uint8_t lds0[kStageOf<kIN>];
  __shared__ __attribute__((aligned(16))) uint8_t lds1[kStageOf<kIN>];
  __shared__ __attribute__((aligned(16))) uint8_t lds2[SPLIT ? kStageOf<kIN> : 16];
  __shared__ int32_t lrow[kBM];  // the tile's rows, counted from base0; past the last: -1
  constexpr int kBN = 128 * kIN, kWave = 32 * kIN;  // lines of the tile, of a wave
  const int tid = threadIdx.x, wave = uni((int32_t)(tid >> 6)), lane = tid & 63, h = lane >> 5;
  // groups of 8 row tiles sweep the column tiles together, a run of tiles an XCD
  const uint32_t nb = gridDim.x, xcd = blockIdx.x % kNumXcd, q8 = nb / kNumXcd, r8 = nb % kNumXcd;
  const uint32_t lt = xcd * q8 + min(xcd, r8) + blockIdx.x / kNumXcd;
  const uint32_t grp = lt / (8 * ntn), gin = lt % (8 * ntn), gm = min(8u, ntm - 8 * grp);
  const int64_t row0 = (int64_t)uni(8 * grp + gin % gm) * kBM, col0 = (int64_t)uni(gin / gm) * kBN;
  const uint32_t rows = (uint32_t)min<int64_t>(tokens - row0, kBM), cols = (uint32_t)min<int64_t>(n - col0, kBN);
  const uint32_t dp = uni((uint32_t)(k / 2)), sp = uni((uint32_t)(k / 16)), xp = uni((uint32_t)(2 * k));
  // Rows are addressed from base0: the window's first row if they are in an
  // order of their own, the tile's first if not.
  const int64_t base0 = order ? row0 / kWindow * kWindow : row0;
  const int64_t span = order ? min<int64_t>(tokens - base0, kWindow) : rows;
  const rsrc_t xs = range_rsrc(x + base0 * k, span * xp);
  if (tid < kBM) lrow[tid] = (uint32_t)tid < rows ? (order ? (int32_t)(order[row0 + tid] - base0) : tid) : -1;
  __syncthreads();
  const rsrc_t wd = range_rsrc(w_data + col0 * dp, (int64_t)cols * dp);
  const rsrc_t ws = range_rsrc(w_scale + col0 * sp, (int64_t)cols * sp);
  const uint32_t steps = (uint32_t)((k + kBK - 1) / kBK), share = (steps + gridDim.y - 1) / gridDim.y;
  const uint32_t ks0 = SPLIT ? uni(min(blockIdx.y * share, steps)) : 0, nk = SPLIT ? uni(min(ks0 + share, steps)) : steps;

  // x: 32 rows a copy, lane g: slot g % 8 of row g / 8 (rows 32 apart have the
  // same granule); codes: 128 lines a copy, lane g: slot g % 2 of line g / 2.
  // In the last step a granule past k is moved out of the buffer's range.
  const uint32_t xgr = (tid & 7) ^ ((tid >> 3) & 7), woff = (tid >> 1) * dp + 16 * ((tid & 1) ^ ((tid >> 3) & 1));
  const uint32_t past = (steps - 1) * kBK + 8 * xgr < (uint32_t)k ? 0u : kOutOfRange;
  uint32_t xoff[kBM / 32];
#pragma unroll
  for (int c = 0; c < kBM / 32; ++c) {
    const int32_t r = lrow[32 * c + (tid >> 3)];
    xoff[c] = r < 0 ? kOutOfRange : r * xp + 16 * xgr;
  }
  auto issue = [&](uint32_t ks, uint8_t* base) {
    const uint32_t cut = ks + 1 == steps ? past : 0u;
#pragma unroll
    for (int c = 0; c < kBM / 32; ++c)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(xs, (lds_ptr_t)(base + 16 * (c * kThreads + wave * 64)), 16,
                                               xoff[c] | cut, ks * (2 * kBK), 0, 0);
#pragma unroll
    for (int c = 0; c < kBN / 128; ++c)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(wd, (lds_ptr_t)(base + kXBytes + 16 * (c * kThreads + wave * 64)), 16,
                                               woff + 128 * c * dp, ks * (kBK / 2), 0, 0);
  };
  // Scales of a step, two bytes a line for each lane half (blocks 2h, 2h + 1),
  // fetched with the step's copies: a line's scales may start on any even byte.
  // In the last step a lane half past k is moved out of the buffer's range.
  const uint32_t spast = (steps - 1) * kBK + 32 * h < (uint32_t)k ? 0u : kOutOfRange;
  uint32_t sc0[kIN], sc1[kIN], sc2[kIN];
  auto fetch_scales = [&](uint32_t ks, uint32_t (&sc)[kIN]) {
    const uint32_t cut = ks + 1 == steps ? spast : 0u;
#pragma unroll
    for (int in = 0; in < kIN; ++in)
      sc[in] = __builtin_amdgcn_raw_buffer_load_b16(ws, ((wave * kWave + in * 32 + (lane & 31)) * sp + 2 * h) | cut,
                                                    ks * (kBK / 16), 0);
  };

  f32x16 acc[kIM][kIN];
#pragma unroll
  for (int im = 0; im < kIM; ++im)
#pragma unroll
    for (int in = 0; in < kIN; ++in) acc[im][in] = f32x16{};
  constexpr uint32_t kAhead = SPLIT ? 2 : 1;
  constexpr int kCopies = kBM / 32 + kBN / 128 + kIN;  // vector-memory operations of a step
  auto step = [&](uint32_t ks, const uint8_t* base, const uint32_t (&sc)[kIN], uint8_t* next, uint32_t (&next_sc)[kIN]) {
    // this step's own copies (the barrier waits for the next step's as well)
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
      const uint32_t line = wave * kWave + in * 32 + (lane & 31);
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

  const uint32_t jw = wave * kWave;  // first line of the wave in the tile
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
    const rsrc_t ps = range_rsrc(partial + ((int64_t)blockIdx.y * tokens + base0) * n + col0,
                                 (span - 1) * 2 * yp + 4 * cols);
#pragma unroll
    for (int im = 0; im < kIM; ++im)
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        const int32_t r = lrow[im * 32 + 8 * (q >> 2) + 4 * h + (q & 3)];
#pragma unroll
        for (int in = 0; in < kIN; ++in) {
          const uint32_t j = jw + in * 32 + (lane & 31);
          __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(acc[im][in][q] * lf[in]), ps,
                                                r >= 0 && j < cols ? r * 2 * yp + 4 * j : kOutOfRange, 0, 0);
        }
      }
    return;
  }
  // Every adapter that one of 32 rows has adds rank/16 MFMA steps of v B_a^T.
  // Rows of other adapters meet B_a only as zeros, but a B_a that is not finite
  // must not reach them either: each adapter's product is formed apart and
  // added to its own rows alone.  The loads of 32 ranks are in flight together.
  const uint32_t r16 = round16(rank);
  rsrc_t vs[kPieces];
#pragma unroll
  for (int p = 0; p < kPieces; ++p) vs[p] = range_rsrc(v + (p * tokens + base0) * r16, span * r16 * 2);
  const rsrc_t ys = range_rsrc(y + base0 * n + col0, (span - 1) * yp + 2 * cols);
  const bool odd = lane & 1;
#pragma unroll
  for (int im = 0; im < kIM; ++im) {
    const int32_t row = lrow[im * 32 + (lane & 31)];
    const int my = adapters && row >= 0 ? ids[base0 + row] : -1;
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
        u32x4 b[2][kIN], vq[2][kPieces];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t rr = r + 16 * i, bin = rr + 8 * h < (uint32_t)rank ? 0u : kOutOfRange;
#pragma unroll
          for (int in = 0; in < kIN; ++in)
            b[i][in] = __builtin_amdgcn_raw_buffer_load_b128(
                bs, ((jw + in * 32 + (lane & 31)) * rank * 2 + 16 * h + 2 * rr) | bin, 0, 0);
          const uint32_t vo = rr < r16 ? voff + 2 * rr : kOutOfRange;
#pragma unroll
          for (int p = 0; p < kPieces; ++p) vq[i][p] = __builtin_amdgcn_raw_buffer_load_b128(vs[p], vo, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int in = 0; in < kIN; ++in) {
            const bf16x8 bf = __builtin_bit_cast(bf16x8, b[i][in]);
#pragma unroll
            for (int p = 0; p < kPieces; ++p)
              part[in] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, vq[i][p]), bf, part[in], 0, 0, 0);
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
#pragma unroll
      for (int q = 0; q < 16; q += 2) {
        const int32_t r = lrow[im * 32 + 8 * (q >> 2) + 4 * h + (q & 3) + odd];
        float lo, hi;
        pair_columns(acc[im][in][q] * lf[in] + sum[in][q], acc[im][in][q + 1] * lf[in] + sum[in][q + 1], odd, &lo, &hi);
        __builtin_amdgcn_raw_buffer_store_b32(pack_bf16(lo, hi), ys, r >= 0 && jp < cols ? r * yp + 2 * jp : kOutOfRange,
                                              0, 0);
      }
    }
  }
}

// y[t] = the sum of the parts, in their order, plus the row's adapter, rounded
// once.  A work-group takes kThreads * 2 columns of a row.
__global__ __launch_bounds__(kThreads) void finish_kernel(const float* __restrict__ partial, int parts, int64_t tokens,
                                                          int64_t n, const uint16_t* __restrict__ lora_b,
                                                          const float* __restrict__ alpha, int adapters, int rank,
                                                          const int32_t* __restrict__ ids, const float* __restrict__ v,
                                                          int v_parts, uint16_t* __restrict__ y) {
  __shared__ __attribute__((aligned(16))) float lv[LORA_MAX_RANK];
  const int64_t t = blockIdx.x, c = ((int64_t)blockIdx.y * kThreads + threadIdx.x) * 2;
  const int a = adapters ? uni(ids[t]) : -1;
  const bool adapted = (uint32_t)a < (uint32_t)adapters;
  if (adapted && (int)threadIdx.x < rank) lv[threadIdx.x] = row_v(v, v_parts, tokens, t, rank, threadIdx.x, a, alpha);
  __syncthreads();
  if (c >= n) return;
  const int64_t count = tokens * n, i = t * n + c;
  f32x2 s = *reinterpret_cast<const f32x2*>(partial + i);
#pragma unroll 4
  for (int p = 1; p < parts; ++p) s += *reinterpret_cast<const f32x2*>(partial + p * count + i);
  if (adapted) {
    const uint16_t* b = lora_b + ((int64_t)a * n + c) * rank;
    s[0] += rank_dot(b, lv, 0, rank, 0.0f);
    s[1] += rank_dot(b + rank, lv, 0, rank, 0.0f);
  }
  *reinterpret_cast<uint32_t*>(y + i) = pack_bf16(s[0], s[1]);
}

// ------------------------------------------------------------- host side

// Parts of the contraction of the first launch: enough work-groups for the
// device, at least one step a wave.
int shrink_parts(int64_t tokens, int64_t k) {
  const int64_t tiles = (tokens + kShrinkRows - 1) / kShrinkRows, steps = (k + kShrinkStep - 1) / kShrinkStep;
  const int64_t want = (4 * kCus + tiles - 1) / tiles;
  return (int)std::max<int64_t>(1, std::min(std::min(want, (steps + kShrinkWaves - 1) / kShrinkWaves), (int64_t)kMaxSplit));
}

constexpr int kWideLines = 256;  // lines of a wide tile of the projection
constexpr int64_t round256(int64_t b) { return (b + 255) / 256 * 256; }
// Parts of the contraction of many rows: as many as give every CU two
// work-groups where the tiles alone do not give it one, at least 4 steps each
// (8 left the 7 tiles of 125 rows of a 1552 x 800 projection alone: 29 us
// instead of 21), and all that is kept between the launches within kMaxWorkspace.
constexpr int64_t kMaxWorkspace = 32 << 20;
int project_parts(int64_t tokens, int64_t k, int64_t n, int rank) {
  const int64_t tiles = ((tokens + kBM - 1) / kBM) * ((n + kWideLines - 1) / kWideLines);
  if (tokens <= kFewRows || tiles >= kCus) return 1;
  const int64_t other = round256(tokens * rank * 4 * shrink_parts(tokens, k)) + round256(tokens * 4);
  const int64_t by_steps = (k + kBK - 1) / kBK / 4, by_room = (kMaxWorkspace - other) / (tokens * n * 4);
  return (int)std::max<int64_t>(1, std::min(std::min(2 * kCus / tiles, by_steps), by_room));
}

// Whether the rows are put in order first: a launch of 6 us where every row is
// another request's (4096 rows of 4 adapters, 7168 x 2048: 192 us instead of
// 266); where they come in order already it is lost (5474 rows of 2 adapters,
// 1376 x 352: 39 us instead of 34), which the host cannot see.  A window's
// rows have to be within 31-bit offsets.
bool ordered(int64_t tokens, int64_t k, int64_t n, int adapters) {
  return tokens > kFewRows && adapters > 1 && adapters < (1 << 21) && kWindow * std::max(2 * k, 2 * n) <= INT32_MAX;
}

// Adapters of a tile of the first launch that are taken side by side: as many
// as a tile of rows in order meets if the adapters are equally frequent.
int shrink_slots(int64_t tokens, int adapters, bool in_order) {
  const int64_t run = std::min<int64_t>(tokens, kWindow);
  const int64_t meets = in_order ? 1 + (kShrinkRows * (int64_t)adapters + run - 1) / run : kShrinkRows;
  return (int)std::min(std::min(meets, (int64_t)adapters), std::min<int64_t>(tokens, kShrinkRows));
}

// Workspace of a call: v (its parts, or its pieces), the order, the projection's
// parts.
struct Workspace {
  int64_t v, order, partial;
  int64_t bytes() const { return v + order + partial; }
};
Workspace workspace_of(int64_t tokens, int64_t k, int64_t n, int32_t rank) {
  const int parts = project_parts(tokens, k, n, rank);
  const bool pieces = tokens > kFewRows && parts == 1;
  return {round256(pieces ? tokens * round16(rank) * 2 * kPieces : tokens * rank * 4 * shrink_parts(tokens, k)),
          tokens > kFewRows && rank ? round256(tokens * 4) : 0, parts > 1 ? parts * tokens * n * 4 : 0};
}

// What any batch of up to `tokens` rows and any rank up to `rank` needs.  Without
// parts of the projection the need grows with both.  With parts it does not, as
// fewer tiles get more of them: the most that the parts of each number of row
// tiles take, which never passes kMaxWorkspace.
int64_t workspace_bound(int64_t tokens, int64_t k, int64_t n, int32_t rank) {
  const int64_t few = std::min<int64_t>(tokens, kFewRows);
  int64_t most = workspace_of(few, k, n, rank).bytes();
  if (tokens <= kFewRows) return most;
  most = std::max(most, round256(tokens * round16(rank) * 2 * kPieces) + (rank ? round256(tokens * 4) : 0));
  const int64_t ntn = (n + kWideLines - 1) / kWideLines, by_steps = (k + kBK - 1) / kBK / 4;
  for (int64_t ntm = 1; ntm * ntn < kCus && (ntm - 1) * kBM < tokens; ++ntm) {
    const int64_t parts = std::min(2 * kCus / (ntm * ntn), by_steps), t = std::min(tokens, ntm * kBM);
    if (parts < 2) continue;
    const int64_t v = round256(t * rank * 4 * shrink_parts(few, k));  // few rows have the most parts of v
    most = std::max(most, std::min(kMaxWorkspace, v + round256(t * 4) + parts * t * n * 4));
  }
  return most;
}

template <class F>
void with_ranks(int rank, F f) {
  if (rank <= 16) f(std::integral_constant<int, 1>());
  else if (rank <= 32) f(std::integral_constant<int, 2>());
  else if (rank <= 64) f(std::integral_constant<int, 4>());
  else f(std::integral_constant<int, 8>());
}

template <int MT>
void launch_few(const uint16_t* x, int tokens, int64_t k, const uint8_t* wd, const uint8_t* ws, const float* wa,
                int64_t n, const uint16_t* b, const float* alpha, int adapters, int rank, const int32_t* ids,
                const float* v, int parts, uint16_t* y, hipStream_t st) {
  // Waves that split the contraction: as few as give most CUs a work-group (8
  // rows, 7168 x 7168: 21 us 4 ways, 25 with 2, 34 not split; 17 rows: 25 us 4
  // ways, 35 with 8).
  auto tiles = [&](int ks) { return (n + 16 * (kTokenWaves / ks) - 1) / (16 * (kTokenWaves / ks)); };
  int ks = 1;
  while (ks < kTokenWaves && tiles(ks) < 200) ks *= 2;
  const TokenPlan P = token_plan(k, tokens, ks, MT, adapters ? (int64_t)tokens * rank * 4 : 0, tiles(ks));
  hipLaunchKernelGGL((few_rows_kernel<MT>), dim3((uint32_t)tiles(P.ks)), dim3(kTokenThreads), P.lds, st, x, tokens, k, wd,
                     ws, wa, n, b, alpha, adapters, adapters ? rank : 0, ids, v, parts, P, y);
}

}  // namespace

extern "C" {

int64_t lora_workspace(int64_t tokens, int64_t k, int64_t n, int32_t rank) {
  if (tokens <= 0 || k <= 0 || n <= 0 || rank < 0) return 0;
  return workspace_bound(tokens, k, n, rank);
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
  if (!aligned(x, 16) || !aligned(w_data, 16) || !aligned(w_scale, 4) || !aligned(w_amax, 4) || !aligned(y, 16) ||
      !aligned(lora_a, 16) || !aligned(lora_b, 16) || !aligned(alpha, 4) || !aligned(adapter_ids, 4) ||
      !aligned(workspace, 16))
    return NVFP4G_EALIGN;
  const Workspace w = workspace_of(tokens, k, n, num_adapters ? rank : 0);
  const int64_t need = w.bytes();
  if (need && (!workspace || workspace_bytes < need)) return NVFP4G_EINVAL;
  const hipStream_t st = (hipStream_t)stream;
  if (((tokens + kBM - 1) / kBM) * ((n + kWideLines - 1) / kWideLines) > kMaxGroups) return NVFP4G_EINVAL;
  const int T = (int)tokens, r = num_adapters ? rank : 0, split = project_parts(tokens, k, n, r);
  const bool few = tokens <= kFewRows, pieces = !few && split == 1;
  const int parts = pieces ? 1 : shrink_parts(tokens, k);
  float* v = (float*)workspace;
  int32_t* order = ordered(tokens, k, n, num_adapters) ? (int32_t*)((char*)workspace + w.v) : nullptr;
  float* partial = (float*)((char*)workspace + w.v + w.order);
  if (num_adapters) {
    if (order)
      hipLaunchKernelGGL(order_kernel, dim3((uint32_t)((tokens + kOrderRows - 1) / kOrderRows)), dim3(kThreads), 0, st,
                         adapter_ids, T, num_adapters, order);
    const dim3 grid((uint32_t)((T + kShrinkRows - 1) / kShrinkRows), parts, shrink_slots(T, num_adapters, order));
    with_ranks(rank, [&](auto nr) {
      constexpr int NR = decltype(nr)::value;
      if (pieces)
        hipLaunchKernelGGL((shrink_kernel<NR, true>), grid, dim3(kShrinkThreads), 0, st, x, T, k, lora_a, alpha, num_adapters,
                           rank, adapter_ids, order, v);
      else
        hipLaunchKernelGGL((shrink_kernel<NR, false>), grid, dim3(kShrinkThreads), 0, st, x, T, k, lora_a, alpha,
                           num_adapters, rank, adapter_ids, order, v);
    });
  }
  if (few) {
    // one 16-line tile a work-group: the most work-groups a projection gives
    if (T <= 16) launch_few<1>(x, T, k, w_data, w_scale, w_amax, n, lora_b, alpha, num_adapters, rank, adapter_ids, v, parts, y, st);
    else launch_few<2>(x, T, k, w_data, w_scale, w_amax, n, lora_b, alpha, num_adapters, rank, adapter_ids, v, parts, y, st);
  } else {
    // Half as wide tiles where neither parts nor the wide ones, two a CU, fill
    // the device: 700 rows, 7168 x 7168 (168 wide tiles) 147 us wide, 128 narrow;
    // 1500 rows, 7168 x 4096 (336) 135 and 128; 2048 rows, 7168 x 2048 (448) 86
    // and 102; parts stay wide.
    const int64_t wide = ((tokens + kBM - 1) / kBM) * ((n + kWideLines - 1) / kWideLines);
    const int lines = split == 1 && wide < 3 * kCus / 2 ? kWideLines / 2 : kWideLines;
    const uint32_t ntm = (uint32_t)((tokens + kBM - 1) / kBM), ntn = (uint32_t)((n + lines - 1) / lines);
    auto project = [&](auto kernel, const int32_t* rows_in) {
      hipLaunchKernelGGL(kernel, dim3(ntm * ntn, split), dim3(kThreads), 0, st, x, tokens, k, w_data, w_scale, w_amax, n,
                         lora_b, num_adapters, r, adapter_ids, rows_in, (const uint16_t*)v, ntm, ntn, y, partial);
    };
    if (split > 1) {
      project(many_rows_kernel<true, 2>, nullptr);
      hipLaunchKernelGGL(finish_kernel, dim3((uint32_t)tokens, (uint32_t)((n + 2 * kThreads - 1) / (2 * kThreads))),
                         dim3(kThreads), 0, st, partial, split, tokens, n, lora_b, alpha, num_adapters, r, adapter_ids,
                         v, parts, y);
    } else if (lines == kWideLines) {
      project(many_rows_kernel<false, 2>, order);
    } else {
      project(many_rows_kernel<false, 1>, order);
    }
  }
  return hip_status();
}

}  // extern "C"
