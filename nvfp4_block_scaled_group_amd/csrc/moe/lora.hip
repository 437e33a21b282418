// lora.hip -- low-rank adapters of many requests beside one shared NVFP4
// projection, behind the C ABI of include/moe_ops.h:
//
//   y[t] = W x[t] + alpha_a B_a (A_a x[t]),   a = adapter of row t.
//
// Two launches.  The first makes v[t] = A_a x[t] (rank values a row): a
// work-group takes 16 rows and multiplies them (MFMA 16x16x32) by each adapter
// that any of them has.  The second is the shared projection with the
// adapters in its epilogue:
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

// FEW: blockIdx = (row tile, part of the contraction, which of the tile's
// adapters); v [parts][tokens][rank] fp32.  Otherwise blockIdx.x is the row
// tile and the work-group goes through the tile's adapters itself; v is
// hi [tokens][R16], lo [tokens][R16] bf16 (R16: rank rounded up to 16, zeros
// past rank), scaled by alpha.  The four waves take a share of the
// contraction each and join in LDS.
template <bool FEW, int NR>
__global__ __launch_bounds__(kThreads) void shrink_kernel(const uint16_t* __restrict__ x, int tokens, int64_t k,
                                                          const uint16_t* __restrict__ lora_a,
                                                          const float* __restrict__ alpha, int adapters, int rank,
                                                          const int32_t* __restrict__ ids, void* __restrict__ v) {
  __shared__ f32x4 red[4 * NR * 64];
  const int lane = threadIdx.x & 63, wave = uni((int32_t)(threadIdx.x >> 6));
  const int row0 = uni((int32_t)blockIdx.x) * kShrinkRows;
  const int my = lane < kShrinkRows && row0 + lane < tokens ? ids[row0 + lane] : -1;
  uint64_t left = __ballot((uint32_t)my < (uint32_t)adapters && lane < kShrinkRows);
  int slot = FEW ? uni((int32_t)blockIdx.z) : 0;
  const int parts = FEW ? uni((int32_t)gridDim.y) * 4 : 4, part = (FEW ? uni((int32_t)blockIdx.y) * 4 : 0) + wave;
  const int64_t steps = (k + kShrinkStep - 1) / kShrinkStep, share = (steps + parts - 1) / parts;
  const int64_t s0 = min<int64_t>(part * share, steps), s1 = min<int64_t>(s0 + share, steps);
  const int m = min(row0 + (lane & 15), tokens - 1);
  const uint16_t* xr = x + (int64_t)m * k;
  while (left) {
    const int first = (int)__builtin_ctzll(left);
    const int a = __builtin_amdgcn_readlane(my, first);
    const uint64_t rows = __ballot(my == a) & left;
    left &= ~rows;
    if (FEW && slot-- != 0) continue;
    f32x4 acc[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) acc[r] = f32x4{0, 0, 0, 0};
    // this lane's line of each 16 ranks (a line past the rank reads the last)
    const uint16_t* ar[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) ar[r] = lora_a + ((int64_t)a * rank + min(16 * r + (lane & 15), rank - 1)) * k;
    for (int64_t s = s0; s < s1; ++s) {
      const int64_t e0 = s * kShrinkStep + 32 * (lane >> 4);
      u32x4 xq[4], aq[NR][4];
      const bool in = e0 < k;
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
    // thread -> (row, rank column): 16 rows x NR*16 columns in passes of 256
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      // element (row, col) of tile r is component row % 4 of lane 16 (row / 4) + col
      const int row = threadIdx.x >> 4, col = threadIdx.x & 15;
      const float* f = reinterpret_cast<const float*>(red) + (r * 64 + 16 * (row >> 2) + col) * 4 + (row & 3);
      float sum = f[0];
#pragma unroll
      for (int w = 1; w < 4; ++w) sum += f[w * NR * 64 * 4];
      if (!((rows >> row) & 1)) continue;
      const int c = 16 * r + col;
      const int64_t t = row0 + row;
      if (FEW) {
        if (c < rank) reinterpret_cast<float*>(v)[((int64_t)blockIdx.y * tokens + t) * rank + c] = sum;
      } else if (c < round16(rank)) {
        const float s = c < rank ? sum * alpha[a] : 0.0f;
        const uint16_t hi = to_bf16(s);
        uint16_t* o = reinterpret_cast<uint16_t*>(v) + t * round16(rank) + c;
        o[0] = hi;
        o[(int64_t)tokens * round16(rank)] = to_bf16(s - __uint_as_float((uint32_t)hi << 16));
      }
    }
    if (FEW) break;
    __syncthreads();
  }
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
  token_multiply<MT, NL>(W, P, x, k, tokens, part, lane, lds, [](int i) { return (int64_t)i; }, acc);
  f32x4* red = reinterpret_cast<f32x4*>(lds);
  float* lv = reinterpret_cast<float*>(lds + kTokenWaves * MT * NL * 1024);  // [tokens][rank]: alpha * v of every row
  __syncthreads();
  for (int i = threadIdx.x; i < tokens * rank; i += kTokenThreads) {
    const int a = ids[i / rank];
    float s = 0.0f;
    if ((uint32_t)a < (uint32_t)adapters) {
      for (int p = 0; p < parts; ++p) s += v[(int64_t)p * tokens * rank + i];
      s *= alpha[a];
    }
    lv[i] = s;
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
          const uint16_t* b = lora_b + ((int64_t)a * n + col) * rank;
          float d = 0.0f;
          for (int i = 0; i < rank; i += 8) {
            const u32x4 bq = *reinterpret_cast<const u32x4*>(b + i);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              d = __builtin_fmaf(bf16lo(bq[j]), lv[t * rank + i + 2 * j], d);
              d = __builtin_fmaf(bf16hi(bq[j]), lv[t * rank + i + 2 * j + 1], d);
            }
          }
          r += d;
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

typedef __attribute__((address_space(3))) void* lds_ptr_t;
constexpr int waitcnt_vm(int n) { return (n & 15) | (7 << 4) | (15 << 8) | ((n >> 4) << 14); }

// Tile of 128 rows x 256 lines; wave w takes all rows and lines 64 w .. + 63,
// so no weight is decoded twice in a work-group.  Element granules (8 of x,
// 16 bytes) and code granules are XOR-placed in LDS so that fragment reads of
// 32 consecutive rows or lines spread over the banks.  Rows past the last and
// elements past k read as zero (the weights' codes there, the next line's, are
// finite and meet zeros).
__global__ __launch_bounds__(kThreads, 2) void many_rows_kernel(
    const uint16_t* __restrict__ x, int64_t tokens, int64_t k, const uint8_t* __restrict__ w_data,
    const uint8_t* __restrict__ w_scale, const float* __restrict__ w_amax, int64_t n,
    const uint16_t* __restrict__ lora_b, int adapters, int rank, const int32_t* __restrict__ ids,
    const uint16_t* __restrict__ v, uint32_t ntm, uint32_t ntn, uint16_t* __restrict__ y) {
  __shared__ __attribute__((aligned(16))) uint8_t lds0[kStage];
  __shared__ __attribute__((aligned(16))) uint8_t lds1[kStage];
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
  const uint32_t nk = (uint32_t)((k + kBK - 1) / kBK);

  // x: 32 rows a copy, lane g: slot g % 8 of row g / 8 (rows 32 apart have the
  // same granule); codes: 128 lines a copy, lane g: slot g % 2 of line g / 2.
  // In the last step a granule past k is moved out of the buffer's range.
  const uint32_t xgr = (tid & 7) ^ ((tid >> 3) & 7), xoff = (tid >> 3) * xp + 16 * xgr;
  const uint32_t woff = (tid >> 1) * dp + 16 * ((tid & 1) ^ ((tid >> 3) & 1));
  const uint32_t past = (nk - 1) * kBK + 8 * xgr < (uint32_t)k ? 0u : kOutOfRange;
  auto issue = [&](uint32_t ks, uint8_t* base) {
    const uint32_t off = ks + 1 == nk ? xoff | past : xoff;
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
  // fetched a step ahead: a line's scales may start on any even byte.
  uint32_t sc[kIN];
  auto fetch_scales = [&](uint32_t ks) {
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
  auto step = [&](uint32_t ks, const uint8_t* base, uint8_t* next) {
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
    __syncthreads();
    float sv[kIN][2];
#pragma unroll
    for (int in = 0; in < kIN; ++in) {
      sv[in][0] = e4m3_value(sc[in] & 0xFFu);
      sv[in][1] = e4m3_value((sc[in] >> 8) & 0xFFu);
    }
    if (ks + 1 < nk) {
      issue(ks + 1, next);
      fetch_scales(ks + 1);
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
  issue(0, lds0);
  fetch_scales(0);
  uint32_t ks = 0;
#pragma unroll 1
  for (; ks + 1 < nk; ks += 2) {
    step(ks, lds0, lds1);
    step(ks + 1, lds1, lds0);
  }
  if (ks < nk) step(ks, lds0, lds1);

  // Epilogue, one 32 x 32 block after the other: line factor, then every
  // adapter that a row of the block has adds rank/16 MFMA steps of v B_a^T.
  // Rows of other adapters meet B_a only as zeros, but a B_a that is not finite
  // must not reach them either: each adapter's product is formed apart and
  // added to its own rows alone.  Rows past the last are out of the output
  // buffer's range, columns past the last are moved out of it.
  const uint32_t jw = wave * 64;  // first line of the wave in the tile
  const uint32_t r16 = round16(rank), yp = (uint32_t)(2 * n);
  const rsrc_t vh = range_rsrc(v + row0 * r16, (int64_t)rows * r16 * 2);
  const rsrc_t vl = range_rsrc(v + (tokens + row0) * r16, (int64_t)rows * r16 * 2);
  const rsrc_t ys = range_rsrc(y + row0 * n + col0, ((int64_t)rows - 1) * yp + 2 * cols);
  const bool odd = lane & 1;
  float lf[kIN];
#pragma unroll
  for (int in = 0; in < kIN; ++in) {
    const uint32_t j = jw + in * 32 + (lane & 31);
    lf[in] = j < cols ? w_amax[col0 + j] / 2688.0f : 0.0f;
  }
#pragma unroll
  for (int im = 0; im < kIM; ++im) {
    const uint32_t row = im * 32 + (lane & 31);
    const int my = adapters && row < rows ? ids[row0 + row] : -1;
    const uint32_t any = (uint32_t)__ballot((uint32_t)my < (uint32_t)adapters);  // lanes 32-63 repeat lanes 0-31
#pragma unroll
    for (int in = 0; in < kIN; ++in) {
      f32x16 sum = f32x16{};
      const uint32_t boff = (jw + in * 32 + (lane & 31)) * rank * 2 + 16 * h;
#pragma unroll 1
      for (uint32_t left = any; left;) {
        const int a = __builtin_amdgcn_readlane(my, (int)__builtin_ctz(left));
        const uint32_t own = (uint32_t)__ballot(my == a);
        left &= ~own;
        const rsrc_t bs = range_rsrc(lora_b + ((int64_t)a * n + col0) * rank, (int64_t)cols * rank * 2);
        const uint32_t voff = my == a ? row * r16 * 2 + 16 * h : kOutOfRange;
        f32x16 part = f32x16{};
#pragma unroll 1
        for (uint32_t r = 0; r < r16; r += 16) {
          const uint32_t bo = r + 8 * h < (uint32_t)rank ? boff + 2 * r : kOutOfRange;
          const bf16x8 b = __builtin_bit_cast(bf16x8, __builtin_amdgcn_raw_buffer_load_b128(bs, bo, 0, 0));
          const bf16x8 hi = __builtin_bit_cast(bf16x8, __builtin_amdgcn_raw_buffer_load_b128(vh, voff + 2 * r, 0, 0));
          const bf16x8 lo = __builtin_bit_cast(bf16x8, __builtin_amdgcn_raw_buffer_load_b128(vl, voff + 2 * r, 0, 0));
          part = __builtin_amdgcn_mfma_f32_32x32x16_bf16(hi, b, part, 0, 0, 0);
          part = __builtin_amdgcn_mfma_f32_32x32x16_bf16(lo, b, part, 0, 0, 0);
        }
#pragma unroll
        for (int q = 0; q < 16; ++q) sum[q] += (own >> (8 * (q >> 2) + 4 * h + (q & 3))) & 1 ? part[q] : 0.0f;
      }
      const uint32_t jp = (jw + in * 32 + (lane & 31)) & ~1u;
      const uint32_t off = jp < cols ? (im * 32 + 4 * h + odd) * yp + 2 * jp : kOutOfRange;
#pragma unroll
      for (int q = 0; q < 16; q += 2) {
        float lo, hi;
        pair_columns(acc[im][in][q] * lf[in] + sum[q], acc[im][in][q + 1] * lf[in] + sum[q + 1], odd, &lo, &hi);
        __builtin_amdgcn_raw_buffer_store_b32(pack_bf16(lo, hi), ys, off + (8 * (q >> 2) + (q & 3)) * yp, 0, 0);
      }
    }
  }
}

// ------------------------------------------------------------- host side

// Parts of the contraction over work-groups for few rows: enough to spread a
// long contraction, whole steps each.
int shrink_parts(int64_t k) {
  const int64_t steps = (k + kShrinkStep - 1) / kShrinkStep, p = (steps + 3) / 4;
  return (int)(p < 1 ? 1 : p > kMaxSplit ? kMaxSplit : p);
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

int64_t lora_workspace(int64_t tokens, int64_t k, int32_t rank) {
  if (tokens <= 0 || k <= 0 || rank <= 0) return 0;
  return tokens <= kFewRows ? tokens * rank * 4 * shrink_parts(k) : tokens * round16(rank) * 4;
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
  if (num_adapters && (!workspace || workspace_bytes < lora_workspace(tokens, k, rank))) return NVFP4G_EINVAL;
  const hipStream_t st = (hipStream_t)stream;
  const int T = (int)tokens, parts = shrink_parts(k);
  const bool few = tokens <= kFewRows;
  if (num_adapters) {
    const uint32_t tiles = (uint32_t)((T + kShrinkRows - 1) / kShrinkRows);
    with_ranks(rank, [&](auto nr) {
      constexpr int NR = decltype(nr)::value;
      if (few) {
        const uint32_t slots = (uint32_t)std::min(std::min(T, kShrinkRows), num_adapters);
        hipLaunchKernelGGL((shrink_kernel<true, NR>), dim3(tiles, parts, slots), dim3(kThreads), 0, st, x, T, k, lora_a,
                           alpha, num_adapters, rank, adapter_ids, workspace);
      } else {
        hipLaunchKernelGGL((shrink_kernel<false, NR>), dim3(tiles), dim3(kThreads), 0, st, x, T, k, lora_a, alpha,
                           num_adapters, rank, adapter_ids, workspace);
      }
    });
  }
  if (few) {
    const float* v = (const float*)workspace;
    // one 16-line tile a work-group: the most work-groups a projection gives
    if (T <= 16) launch_few<1, 1>(x, T, k, w_data, w_scale, w_amax, n, lora_b, alpha, num_adapters, rank, adapter_ids, v, parts, y, st);
    else if (T <= 32) launch_few<2, 1>(x, T, k, w_data, w_scale, w_amax, n, lora_b, alpha, num_adapters, rank, adapter_ids, v, parts, y, st);
    else launch_few<4, 1>(x, T, k, w_data, w_scale, w_amax, n, lora_b, alpha, num_adapters, rank, adapter_ids, v, parts, y, st);
  } else {
    const uint32_t ntm = (uint32_t)((tokens + kBM - 1) / kBM), ntn = (uint32_t)((n + kBN - 1) / kBN);
    if ((int64_t)ntm * ntn > (int64_t)INT32_MAX) return NVFP4G_EINVAL;
    hipLaunchKernelGGL(many_rows_kernel, dim3(ntm * ntn), dim3(kThreads), 0, st, x, tokens, k, w_data, w_scale, w_amax,
                       n, lora_b, num_adapters, num_adapters ? rank : 0, adapter_ids, (const uint16_t*)workspace, ntm,
                       ntn, y);
  }
  return hip_status();
}

}  // extern "C"
