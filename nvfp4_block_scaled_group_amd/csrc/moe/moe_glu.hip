// moe_glu.hip -- the experts' gated feed-forward block on row-scaled NVFP4
// operands: gate and up projection, activation and product in one kernel, and
// its backward pass, behind the C ABI of include/moe_ops.h.
//
//   forward   g = Xa Wg^T, u = Xa Wu^T, h = act(g) * u
//   backward  dh = dY Wd,  du = dh * act(g),  dg = dh * u * act'(g)
//
// Both are NT products of two NVFP4 operands stored along the contraction
// index.  A line's factor A / 2688 leaves the sum, and value(code) * value(S)
// (at most 6 significant bits, 2^-10 .. 2688) is exact in fp16, so the fp32
// MFMA sum of exact products is the only rounding before the epilogue, which
// stays in fp32 up to its one rounding to bf16.
//
// Work-group: 128 packed rows x 256 weight lines, 4 waves in a 2 x 2 grid of
// 64 x 128 (2 x 4 MFMA tiles of 32 x 32), two work-groups on a CU.  In the
// forward pass the 256 lines are 128 gate lines and the 128 up lines of the
// same columns, laid out in LDS so that each wave holds g and u of the same
// elements in the same lane (its first two MFMA columns are gate lines, the
// other two the matching up lines): the activation and the product need no
// exchange, and neither g nor u goes through memory.
//
// What bounds it: at large sizes the power of MFMAs and decode together
// (forward, 65536 rows, 7168 x 2 x 2048: 3.0 ms, 1.28 PFLOP/s at a clock of
// 1.6 GHz, MFMAs busy 68% of it); with few steps a tile the start and the
// epilogue too (backward, 16384 rows of 64 experts, 2048 x 1040: 112 to 120 us, 0.6
// PFLOP/s; the same with 1024 columns, a whole number of tiles, 91 to 93 us).
#include <algorithm>

#include "moe_common.hpp"

namespace {

using namespace moe;

typedef _Float16 h2_t __attribute__((ext_vector_type(2)));
typedef _Float16 h8_t __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kWavesN = 2;
constexpr int kWM = 2;            // 32 x 32 MFMA tiles of a wave along the rows; NW along the lines
constexpr int kBM = 128;          // rows of a work-group: the expert granule
constexpr int kBK = 128;          // contraction step
constexpr int kGroupRows = 8;     // row tiles that sweep the column tiles together

// One operand: the lines of a tile, `valid` of which exist (others read 0).
struct Lines {
  const uint8_t* data;   // line pitch L/2 bytes
  const uint8_t* scale;  // line pitch L/16 bytes
  uint32_t valid;
};

// LDS: codes of one step, 64 bytes a line, A then B (two stages in separate
// arrays, so that reads of one need not wait for copies into the other);
// scales of four steps at a time, 32 bytes a line, double-buffered.
constexpr uint32_t kRowBytes = kBK / 2, kRowScales = kBK / 16;
constexpr uint32_t kStB = kBM * kRowBytes;
constexpr uint32_t kScSteps = 4, kScLine = kScSteps * kRowScales;
constexpr uint32_t kScB = kBM * kScLine;
template <int NW>
struct Tile {
  static constexpr int kLines = 2 * 32 * NW;                                    // weight lines of a work-group
  static constexpr uint32_t kStageBytes = kStB + kLines * kRowBytes;            // 24 KB (NW 4), 16 KB (NW 2)
  static constexpr uint32_t kScBlockBytes = kScB + kLines * kScLine;            // 12 KB, 8 KB
};

typedef __attribute__((address_space(3))) void* lds_ptr_t;

// 16-byte granule q of a line sits at slot q ^ (line / 4 % 4), so that a
// fragment read of 32 consecutive lines spreads over the banks.
__device__ __forceinline__ uint32_t swz(uint32_t line, uint32_t q) { return q ^ ((line >> 2) & 3u); }

// s_waitcnt for at most n outstanding vector-memory operations.
constexpr int waitcnt_vm(int n) { return (n & 15) | (7 << 4) | (15 << 8) | ((n >> 4) << 14); }

__device__ __forceinline__ h2_t scales_h2(uint32_t two_codes) {
  return __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(two_codes, 1.0f, false);
}

// Eight codes times value(S) as fp16 (exact).
__device__ __forceinline__ h8_t decode8(uint32_t w, _Float16 S) {
  const h2_t ss = {S, S};
  const h2_t p0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0) * ss;
  const h2_t p1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1) * ss;
  const h2_t p2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2) * ss;
  const h2_t p3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3) * ss;
  return h8_t{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

__device__ __forceinline__ rsrc_t lines_rsrc(const uint8_t* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(uni(reinterpret_cast<int64_t>(p))), 0, bytes,
                                           0x00020000);
}

// acc[im][in] += A lines x B lines^T over the contraction length L (a multiple
// of kBK).  PAIR: B's LDS lines are four blocks of 16 NW: the first of B0
// (gate), the first of B1 (up), the second of B0, the second of B1; otherwise
// 64 NW lines of B0.  Each step waits for its own copies, passes one barrier, issues the
// copies of the next step into the other stage and multiplies meanwhile.
// Contraction order: word 8h + s of a line's 64-byte chunk feeds sub-step s of
// lane half h, in A and B alike, so a lane reads its eight sub-steps' words
// with two 16-byte LDS reads.
// A wave whose columns all lie past the last one (`live` false) copies and
// waits with the others but multiplies nothing.
template <bool PAIR, int NW>
__device__ __forceinline__ void multiply(const Lines& A, const Lines& B0, const Lines& B1, uint32_t L, bool live,
                                         f32x16 (&acc)[kWM][NW], uint8_t* lds0, uint8_t* lds1, uint8_t* lsc) {
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const uint32_t dpitch = uni(L / 2), spitch = uni(L / 16);
  const uint32_t av = uni(A.valid), b0v = uni(B0.valid), b1v = uni(B1.valid);
  const rsrc_t ad = lines_rsrc(A.data, av * dpitch), as = lines_rsrc(A.scale, av * spitch);
  const rsrc_t b0d = lines_rsrc(B0.data, b0v * dpitch), b0s = lines_rsrc(B0.scale, b0v * spitch);
  const rsrc_t b1d = PAIR ? lines_rsrc(B1.data, b1v * dpitch) : b0d;
  constexpr uint32_t kScBlockBytes = Tile<NW>::kScBlockBytes;
  constexpr int kLines = Tile<NW>::kLines;
  constexpr uint32_t kBlock = 16 * NW;  // lines of a PAIR block: a wave's copies stay inside one
  const uint32_t uw = uni((uint32_t)wave);
  // a wave's scale copies move 32 lines, its code copies 16
  const rsrc_t bs = PAIR && (32 * uw / kBlock) % 2 ? lines_rsrc(B1.scale, b1v * spitch) : b0s;
  const uint32_t nk = L / kBK;
  if (nk == 0) return;

  // Codes of a step: 64 lines a copy, lane g moves slot g % 4 of line g / 4.
  const uint32_t cl = tid >> 2, cq = tid & 3;
  auto issue = [&](uint32_t ks, uint8_t* base) {
    const uint32_t sd = ks * kRowBytes;
#pragma unroll
    for (int c = 0; c < kBM / 64; ++c)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ad, (lds_ptr_t)(base + 16 * (c * kThreads + wave * 64)), 16,
                                               (64 * c + cl) * dpitch + 16 * swz(cl, cq), sd, 0, 0);
#pragma unroll
    for (int c = 0; c < kLines / 64; ++c) {
      const uint32_t at = 64 * c + cl, blk = at / kBlock;  // LDS line; its block's parity is the wave's
      const bool up = PAIR && ((64 * c + 16 * uw) / kBlock) % 2;
      const uint32_t line = PAIR ? blk / 2 * kBlock + at % kBlock : at;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(up ? b1d : b0d,
                                               (lds_ptr_t)(base + kStB + 16 * (c * kThreads + wave * 64)), 16,
                                               line * dpitch + 16 * swz(cl, cq), sd, 0, 0);
    }
  };
  // Scales of a block of steps: 128 lines a copy, 16 bytes a lane.
  auto issue_scales = [&](uint32_t blk, uint8_t* sbase) {
    const uint32_t so = blk * kScLine, sl = tid >> 1, sq = tid & 1;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(as, (lds_ptr_t)(sbase + 16 * (wave * 64)), 16, sl * spitch + 16 * sq, so,
                                             0, 0);
#pragma unroll
    for (int c = 0; c < kLines / 128; ++c) {
      const uint32_t at = 128 * c + sl;
      const uint32_t line = PAIR ? at / kBlock / 2 * kBlock + at % kBlock : at;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(bs, (lds_ptr_t)(sbase + kScB + 16 * (c * kThreads + wave * 64)), 16,
                                               line * spitch + 16 * sq, so, 0, 0);
    }
  };

  const int wm = wave / kWavesN, wn = wave % kWavesN, h = lane >> 5;
  auto step = [&](uint32_t ks, const uint8_t* base, uint8_t* next) {
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
    __syncthreads();
    h2_t sa[kWM][2], sb[NW][2];
    const uint8_t* scb = lsc + ((ks / kScSteps) & 1) * kScBlockBytes + kRowScales * (ks % kScSteps) + 4 * h;
#pragma unroll
    for (int im = 0; im < kWM; ++im) {
      const uint32_t sc = *reinterpret_cast<const uint32_t*>(scb + kScLine * (wm * (kWM * 32) + im * 32 + (lane & 31)));
      sa[im][0] = scales_h2(sc & 0xFFFFu);
      sa[im][1] = scales_h2(sc >> 16);
    }
#pragma unroll
    for (int in = 0; in < NW; ++in) {
      const uint32_t sc =
          *reinterpret_cast<const uint32_t*>(scb + kScB + kScLine * (wn * (NW * 32) + in * 32 + (lane & 31)));
      sb[in][0] = scales_h2(sc & 0xFFFFu);
      sb[in][1] = scales_h2(sc >> 16);
    }
    if (ks + 1 < nk) {
      issue(ks + 1, next);
      const uint32_t nb = (ks + 1) / kScSteps;
      if ((ks + 1) % kScSteps == 0) issue_scales(nb, lsc + (nb & 1) * kScBlockBytes);
    }
    if (!live) return;
    u32x4 wa[kWM][2], wb[NW][2];
#pragma unroll
    for (int im = 0; im < kWM; ++im) {
      const uint32_t line = wm * (kWM * 32) + im * 32 + (lane & 31);
      wa[im][0] = *reinterpret_cast<const u32x4*>(base + kRowBytes * line + 16 * swz(line, 2 * h));
      wa[im][1] = *reinterpret_cast<const u32x4*>(base + kRowBytes * line + 16 * swz(line, 2 * h + 1));
    }
#pragma unroll
    for (int in = 0; in < NW; ++in) {
      const uint32_t line = wn * (NW * 32) + in * 32 + (lane & 31);
      wb[in][0] = *reinterpret_cast<const u32x4*>(base + kStB + kRowBytes * line + 16 * swz(line, 2 * h));
      wb[in][1] = *reinterpret_cast<const u32x4*>(base + kStB + kRowBytes * line + 16 * swz(line, 2 * h + 1));
    }
    // the next sub-step's fragments are decoded between this one's MFMAs
    h8_t af[2][kWM], bf[2][NW];
#pragma unroll
    for (int im = 0; im < kWM; ++im) af[0][im] = decode8(wa[im][0][0], sa[im][0][0]);
#pragma unroll
    for (int in = 0; in < NW; ++in) bf[0][in] = decode8(wb[in][0][0], sb[in][0][0]);
#pragma unroll
    for (int s = 0; s < kBK / 16; ++s) {
      const int cu = s & 1, nx = cu ^ 1, t = s + 1;
      if (t < kBK / 16) {
#pragma unroll
        for (int im = 0; im < kWM; ++im) af[nx][im] = decode8(wa[im][t >> 2][t & 3], sa[im][t >> 2][(t >> 1) & 1]);
#pragma unroll
        for (int in = 0; in < NW; ++in) bf[nx][in] = decode8(wb[in][t >> 2][t & 3], sb[in][t >> 2][(t >> 1) & 1]);
      }
#pragma unroll
      for (int im = 0; im < kWM; ++im)
#pragma unroll
        for (int in = 0; in < NW; ++in)
          acc[im][in] = __builtin_amdgcn_mfma_f32_32x32x16_f16(af[cu][im], bf[cu][in], acc[im][in], 0, 0, 0);
      if (t < kBK / 16) {
#pragma unroll
        for (int i = 0; i < kWM * NW; ++i) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // one MFMA
          __builtin_amdgcn_sched_group_barrier(0x002, 8 * (kWM + NW) / (kWM * NW), 0);  // and its share of the decode
        }
      }
    }
  };
  issue(0, lds0);
  issue_scales(0, lsc);
#pragma unroll 1
  for (uint32_t ks = 0; ks < nk; ks += 2) {
    step(ks, lds0, lds1);
    if (ks + 1 >= nk) break;
    step(ks + 1, lds1, lds0);
  }
  __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
  __syncthreads();
}

// Logical tile: super-tiles of 64 consecutive tiles dealt round-robin to the
// 8 XCDs, so that each XCD's L2 holds the operand slices its tiles share.
__device__ __forceinline__ uint32_t xcd_tile() {
  const uint32_t id = blockIdx.x, T = gridDim.x;
  const uint32_t round = kNumXcd * 64, full = (T / round) * round;
  if (id >= full) return uni(id);
  const uint32_t j = id / kNumXcd, x = id % kNumXcd;
  return uni((kNumXcd * (j / 64) + x) * 64 + j % 64);
}

__device__ __forceinline__ void grouped_tile(uint32_t t, uint32_t ntm, uint32_t ntn, uint32_t* tm, uint32_t* tn) {
  const uint32_t g = t / (kGroupRows * ntn), in = t % (kGroupRows * ntn);
  const uint32_t first = g * kGroupRows, gm = min((uint32_t)kGroupRows, ntm - first);
  *tm = uni(first + in % gm);
  *tn = uni(in / gm);
}

// A wave's own half of a code stage, which is free in the epilogue: 32 rows x
// BLK blocks of 32 columns of fp32 go in as the MFMA layout holds them (column
// in the lane) and come out as 8 consecutive columns of a row, so that memory
// sees 16 bytes a lane and 64 or 128 contiguous bytes a row.
template <int BLK>
struct Stage {
  static constexpr int kPitch = 32 * BLK + 8;    // floats: the two lane halves, 4 rows apart, on different banks
  static constexpr int kLanes = 4 * BLK;         // of a row on the way out
  static constexpr int kRows = 64 / kLanes;      // rows of one pass
  float* p;
  __device__ __forceinline__ Stage(uint8_t* lds0, uint8_t* lds1, int wave)
      : p(reinterpret_cast<float*>((wave < 2 ? lds0 : lds1) + (wave & 1) * (Tile<2 * BLK>::kStageBytes / 2))) {
    static_assert(32 * kPitch * 4 <= (int)Tile<2 * BLK>::kStageBytes / 2, "two waves share a stage");
  }
  __device__ __forceinline__ void put(int block, int v, int lane, float x) {
    p[(8 * (v >> 2) + 4 * (lane >> 5) + (v & 3)) * kPitch + 32 * block + (lane & 31)] = x;
  }
  __device__ __forceinline__ void get(int row, int col, float (&x)[8]) const {
    const f32x4 a = *reinterpret_cast<const f32x4*>(p + row * kPitch + col);
    const f32x4 b = *reinterpret_cast<const f32x4*>(p + row * kPitch + col + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = a[i];
      x[4 + i] = b[i];
    }
  }
};
// Orders a wave's own LDS writes and reads (they run in issue order).
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}
__device__ __forceinline__ u32x4 pack8(const float (&v)[8]) {
  return u32x4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
}

struct Operands {
  const uint8_t *a_data, *a_scale;
  const float* a_amax;
  const uint8_t *b_data, *b_scale;
  const float* b_amax;
};

template <int ACT>
__device__ __forceinline__ float glu(float g, float u) {
  float dv;
  return g * act_logistic<ACT>(g, &dv) * u;
}

// What the forward pass keeps for the backward one.
enum Keep { kKeepNone, kKeepBf16, kKeep8 };
// g and u in 8 bits: codes [rows, 2f] and scales [2 * ceil(f / 32), rows], so
// that the scales of a tile's rows lie side by side.
struct Kept {
  int8_t* q;
  uint16_t* s;
  int64_t rows;
};
constexpr int kGroup = MOE_KEEP8_GROUP;  // columns of a scale: four lanes hold 8 each
static_assert(kGroup == 32, "the reductions below are over four lanes");

// Codes of a lane's 8 values and the scale (bf16 bits) of its group.  Beside the
// products they cost little: 16384 rows, 7168 x 2 x 2048: 801 to 810 us, 786 to 796 with
// g and u in bf16, 775 to 802 with none kept; the backward pass 428 to 440 us and 425 to
// 432, 441 to 447 where it writes act(g) u again; 8192 rows, 2048 x 2 x 1040: 93 to 95 us,
// 93, 90, and 63.5, 73, 64.  (Sixteen of the large ones in a row pull the clock down to
// 870 and 473 us.)
__device__ __forceinline__ u32x2 keep8(const float (&v)[8], uint16_t* scale) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);  // NaN above inf above the rest
  m = max(m, dpp_x1(m));
  m = max(m, dpp_x2(m));
  if (m >= 0x7F800000u || m < __float_as_uint(0x1p-112f)) {
    *scale = m >= 0x7F800000u ? 0x7FC0 : 0;
    return u32x2{0, 0};
  }
  *scale = to_bf16(__uint_as_float(m) / 127.0f);
  // v / S, correctly rounded: a rounded reciprocal's product is an ulp off at most, and
  // one step on its exact remainder ends there (Markstein).  At most 127 (1 + 2^-8)
  // (1 + 2^-24)^2 < 127.497 (S is the bf16 value nearest to m / 127, which it is below
  // by 2^-8 of itself at most): a code never passes 127.
  const float S = __uint_as_float((uint32_t)*scale << 16), inv = 1.0f / S;
  float t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q = v[i] * inv;
    t[i] = __builtin_fmaf(__builtin_fmaf(-q, S, v[i]), inv, q);
  }
  return u32x2{codes4(t[0], t[1], t[2], t[3]), codes4(t[4], t[5], t[6], t[7])};
}
// The value of byte i of a lane's codes, exact: the code's byte plus 128 is a
// float in one conversion, and the 128 leave it again before the scale comes (128 s
// would pass fp32's range where s is 2^121).
__device__ __forceinline__ float kept(u32x2 q, int i, float s) {
  const uint32_t w = q[i >> 2] ^ 0x80808080u;
  return ((float)((w >> (8 * (i & 3))) & 0xFFu) - 128.0f) * s;
}

// 8 columns of a row as they were kept.
struct KeptRow {
  u32x2 g, u;
  uint32_t gs, us;
};

// Forward: tiles of 128 packed rows x 32 NW columns (64 NW lines).
template <int ACT, Keep KEEP, int NW>
__global__ __launch_bounds__(kThreads, 2) void glu_fwd_kernel(Operands O, int64_t f, int64_t k, Routing R,
                                                              uint32_t ntm, uint32_t ntn, uint16_t* __restrict__ h,
                                                              uint16_t* __restrict__ gu, Kept K8) {
  constexpr int kCols = 32 * NW;
  __shared__ __attribute__((aligned(16))) uint8_t lds0[Tile<NW>::kStageBytes];
  __shared__ __attribute__((aligned(16))) uint8_t lds1[Tile<NW>::kStageBytes];
  __shared__ __attribute__((aligned(16))) uint8_t lsc[2 * Tile<NW>::kScBlockBytes];
  __shared__ float lsa[kBM], lsb[Tile<NW>::kLines];
  if (!routing_ok(R)) return;
  const int32_t total = route_end(R, R.num_experts - 1);
  uint32_t tm, tn;
  grouped_tile(xcd_tile(), ntm, ntn, &tm, &tn);
  const int32_t row0 = (int32_t)(tm * kBM);
  if (row0 >= total) return;
  int32_t rbeg, rend;
  const int e = find_expert(R, row0, &rbeg, &rend);
  const int64_t col0 = (int64_t)tn * kCols;
  const uint32_t cols = (uint32_t)min<int64_t>(f - col0, kCols);
  const int64_t gl = (int64_t)e * 2 * f + col0, ul = gl + f;
  const Lines A{O.a_data + (int64_t)row0 * (k / 2), O.a_scale + (int64_t)row0 * (k / 16), (uint32_t)kBM};
  const Lines G{O.b_data + gl * (k / 2), O.b_scale + gl * (k / 16), cols};
  const Lines U{O.b_data + ul * (k / 2), O.b_scale + ul * (k / 16), cols};
  f32x16 acc[kWM][NW];
#pragma unroll
  for (int im = 0; im < kWM; ++im)
#pragma unroll
    for (int in = 0; in < NW; ++in) acc[im][in] = f32x16{};
  const int tid = threadIdx.x, wave = uni((int32_t)(tid >> 6)), lane = tid & 63;
  const int wm = wave / kWavesN, wn = wave % kWavesN;
  const bool live = (uint32_t)wn * (kCols / 2) < cols;
  multiply<true, NW>(A, G, U, (uint32_t)k, live, acc, lds0, lds1, lsc);

  if (tid < kBM) lsa[tid] = O.a_amax[row0 + tid] / 2688.0f;
  if (tid < 2 * kCols) {
    const uint32_t j = tid % kCols;
    const float* am = O.b_amax + (tid < kCols ? gl : ul);
    lsb[tid] = j < cols ? am[j] / 2688.0f : 0.0f;
  }
  __syncthreads();
  if (!live) return;
  constexpr int BLK = NW / 2;
  Stage<BLK> stage(lds0, lds1, wave);
  const uint32_t j0 = wn * (32 * BLK), c = 8 * (lane % Stage<BLK>::kLanes), srow = lane / Stage<BLK>::kLanes;
  const bool write = j0 + c < cols;
#pragma unroll
  for (int im = 0; im < kWM; ++im) {
    const int64_t out0 = row0 + wm * (kWM * 32) + im * 32 + srow;
    float g[BLK][16], u[BLK][16];
#pragma unroll
    for (int in = 0; in < BLK; ++in) {
      const float sg = lsb[j0 + in * 32 + (lane & 31)], su = lsb[kCols + j0 + in * 32 + (lane & 31)];
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const float sa = lsa[wm * (kWM * 32) + im * 32 + 8 * (v >> 2) + 4 * (lane >> 5) + (v & 3)];
        g[in][v] = (acc[im][in][v] * sa) * sg;
        u[in][v] = (acc[im][in + BLK][v] * sa) * su;
        stage.put(in, v, lane, glu<ACT>(g[in][v], u[in][v]));
      }
    }
    auto put_rows = [&](uint16_t* base, int64_t pitch) {
      wave_sync();
#pragma unroll
      for (int r = 0; r < 32; r += Stage<BLK>::kRows) {
        float v[8];
        stage.get(r + srow, c, v);
        if (write) *reinterpret_cast<u32x4*>(base + (out0 + r) * pitch + col0 + j0 + c) = pack8(v);
      }
      wave_sync();
    };
    put_rows(h, f);
    if (KEEP == kKeep8) {
      const int64_t groups = (f + kGroup - 1) / kGroup;
#pragma unroll
      for (int up = 0; up < 2; ++up) {
#pragma unroll
        for (int in = 0; in < BLK; ++in)
#pragma unroll
          for (int v = 0; v < 16; ++v) stage.put(in, v, lane, up ? u[in][v] : g[in][v]);
        wave_sync();
        uint16_t* scales = K8.s + (up * groups + (col0 + j0 + c) / kGroup) * K8.rows + out0;
#pragma unroll
        for (int r = 0; r < 32; r += Stage<BLK>::kRows) {
          float v[8];
          stage.get(r + srow, c, v);
          uint16_t s;
          const u32x2 q = keep8(v, &s);
          if (write) *reinterpret_cast<u32x2*>(K8.q + (out0 + r) * 2 * f + up * f + col0 + j0 + c) = q;
          if (write && (lane & 3) == 0) scales[r] = s;
        }
        wave_sync();
      }
    }
    if (KEEP == kKeepBf16) {
#pragma unroll
      for (int in = 0; in < BLK; ++in)
#pragma unroll
        for (int v = 0; v < 16; ++v) stage.put(in, v, lane, g[in][v]);
      put_rows(gu, 2 * f);
#pragma unroll
      for (int in = 0; in < BLK; ++in)
#pragma unroll
        for (int v = 0; v < 16; ++v) stage.put(in, v, lane, u[in][v]);
      put_rows(gu + f, 2 * f);
    }
  }
}

// Backward: tiles of 128 packed rows x 64 NW columns of dh.  With KEEP8 g and u
// come from 8 bits, and act(g) * u goes to `again` if that is not null.
template <int ACT, bool KEEP8, int NW>
__global__ __launch_bounds__(kThreads, 2) void glu_bwd_kernel(Operands O, int64_t f, int64_t k, Routing R,
                                                              uint32_t ntm, uint32_t ntn,
                                                              const uint16_t* __restrict__ gu, Kept K8,
                                                              uint16_t* __restrict__ dgu,
                                                              uint16_t* __restrict__ again) {
  constexpr int kCols = Tile<NW>::kLines;
  __shared__ __attribute__((aligned(16))) uint8_t lds0[Tile<NW>::kStageBytes];
  __shared__ __attribute__((aligned(16))) uint8_t lds1[Tile<NW>::kStageBytes];
  __shared__ __attribute__((aligned(16))) uint8_t lsc[2 * Tile<NW>::kScBlockBytes];
  __shared__ float lsa[kBM], lsb[Tile<NW>::kLines];
  if (!routing_ok(R)) return;
  const int32_t total = route_end(R, R.num_experts - 1);
  uint32_t tm, tn;
  grouped_tile(xcd_tile(), ntm, ntn, &tm, &tn);
  const int32_t row0 = (int32_t)(tm * kBM);
  if (row0 >= total) return;
  int32_t rbeg, rend;
  const int e = find_expert(R, row0, &rbeg, &rend);
  const int64_t col0 = (int64_t)tn * kCols;
  const uint32_t cols = (uint32_t)min<int64_t>(f - col0, kCols);
  const int64_t line0 = (int64_t)e * f + col0;
  const Lines A{O.a_data + (int64_t)row0 * (k / 2), O.a_scale + (int64_t)row0 * (k / 16), (uint32_t)kBM};
  const Lines B{O.b_data + line0 * (k / 2), O.b_scale + line0 * (k / 16), cols};
  f32x16 acc[kWM][NW];
#pragma unroll
  for (int im = 0; im < kWM; ++im)
#pragma unroll
    for (int in = 0; in < NW; ++in) acc[im][in] = f32x16{};
  const int tid = threadIdx.x, wave = uni((int32_t)(tid >> 6)), lane = tid & 63;
  const int wm = wave / kWavesN, wn = wave % kWavesN;
  const bool live = (uint32_t)wn * (kCols / 2) < cols;
  multiply<false, NW>(A, B, B, (uint32_t)k, live, acc, lds0, lds1, lsc);

  constexpr int BLK = NW / 2, kRows = Stage<BLK>::kRows, kPasses = 32 / kRows;
  const int c = 8 * (lane % Stage<BLK>::kLanes), srow = lane / Stage<BLK>::kLanes;
  // the kept rows of 32 x 32 BLK blocks, one block ahead
  KeptRow k8[2][KEEP8 ? kPasses : 1];
  auto load8 = [&](int blk) {
    const uint32_t j = wn * (kCols / 2) + blk % (NW / BLK) * (32 * BLK) + c;
    const int64_t row = row0 + wm * (kWM * 32) + blk / (NW / BLK) * 32 + srow;
    const int64_t up = (f + kGroup - 1) / kGroup * K8.rows;  // from a scale of g to that of u
    const uint16_t* scales = K8.s + (col0 + j) / kGroup * K8.rows + row;
    const int8_t* q = K8.q + row * 2 * f + col0 + j;
#pragma unroll
    for (int r = 0; r < (KEEP8 ? kPasses : 0); ++r) {
      KeptRow& o = k8[blk & 1][r];
      o = KeptRow{u32x2{0, 0}, u32x2{0, 0}, 0, 0};
      if (j < cols) {
        o.g = *reinterpret_cast<const u32x2*>(q + 2 * kRows * r * f);
        o.u = *reinterpret_cast<const u32x2*>(q + 2 * kRows * r * f + f);
        o.gs = scales[kRows * r];
        o.us = scales[up + kRows * r];
      }
    }
  };
  if (KEEP8) load8(0);
  if (tid < kBM) lsa[tid] = O.a_amax[row0 + tid] / 2688.0f;
  if (tid < kCols) lsb[tid] = (uint32_t)tid < cols ? O.b_amax[line0 + tid] / 2688.0f : 0.0f;
  __syncthreads();
  if (!live) return;
  Stage<BLK> stage(lds0, lds1, wave);
#pragma unroll
  for (int im = 0; im < kWM; ++im)
#pragma unroll
    for (int in0 = 0; in0 < NW; in0 += BLK) {
      const uint32_t j0 = wn * (kCols / 2) + in0 * 32;
      const bool write = j0 + c < cols;
      const int64_t at0 = (row0 + wm * (kWM * 32) + im * 32 + srow) * 2 * f + col0 + j0 + c;
      // through the caches: rows of 2f columns start inside a cache line (past
      // them 1 to 4% slower); two blocks' loads at once were 8% slower
      u32x4 gq[kPasses], uq[kPasses];
      constexpr int kBlocks = kWM * NW / BLK;
      const int blk = im * (NW / BLK) + in0 / BLK;
      if (KEEP8 && blk + 1 < kBlocks) load8(blk + 1);
#pragma unroll
      for (int r = 0; r < kPasses; ++r) {
        if (KEEP8) break;
        gq[r] = uq[r] = u32x4{0, 0, 0, 0};
        if (write) {
          gq[r] = *reinterpret_cast<const u32x4*>(gu + at0 + 2 * kRows * r * f);
          uq[r] = *reinterpret_cast<const u32x4*>(gu + at0 + 2 * kRows * r * f + f);
        }
      }
#pragma unroll
      for (int in = 0; in < BLK; ++in) {
        const float sb = lsb[j0 + in * 32 + (lane & 31)];
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          const float sa = lsa[wm * (kWM * 32) + im * 32 + 8 * (v >> 2) + 4 * (lane >> 5) + (v & 3)];
          stage.put(in, v, lane, (acc[im][in0 + in][v] * sa) * sb);
        }
      }
      wave_sync();
#pragma unroll
      for (int r = 0; r < kPasses; ++r) {
        float dh[8], dg[8], du[8], hh[8];
        stage.get(kRows * r + srow, c, dh);
        const KeptRow& kr = k8[blk & 1][KEEP8 ? r : 0];
        const float sg = KEEP8 ? __uint_as_float(kr.gs << 16) : 0.0f, su = KEEP8 ? __uint_as_float(kr.us << 16) : 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float g = KEEP8 ? kept(kr.g, i, sg) : i & 1 ? bf16hi(gq[r][i >> 1]) : bf16lo(gq[r][i >> 1]);
          const float u = KEEP8 ? kept(kr.u, i, su) : i & 1 ? bf16hi(uq[r][i >> 1]) : bf16lo(uq[r][i >> 1]);
          float dv;
          const float q = act_logistic<ACT>(g, &dv), a = g * q;
          du[i] = dh[i] * a;
          dg[i] = dh[i] * u * __builtin_fmaf(a * (1.0f - q), dv, q);
          if (KEEP8) hh[i] = a * u;
        }
        if (KEEP8 && again && write)
          *reinterpret_cast<u32x4*>(again + (row0 + wm * (kWM * 32) + im * 32 + srow + kRows * r) * f + col0 + j0 + c) =
              pack8(hh);
        if (write) {
          *reinterpret_cast<u32x4*>(dgu + at0 + 2 * kRows * r * f) = pack8(dg);
          *reinterpret_cast<u32x4*>(dgu + at0 + 2 * kRows * r * f + f) = pack8(du);
        }
      }
      wave_sync();
    }
}

// ------------------------------------------------------------- host side

constexpr int64_t kMaxF = 1 << 19;  // 2f lines within the grouped GEMM's 2^20

// cols_per_tile: the wide tile's columns (narrow ones are for few tiles).
int check_glu(const Operands& O, int64_t rows, int64_t f, int64_t k, int32_t E, int32_t act, int cols_per_tile) {
  if (k <= 0 || k % kBK != 0 || k > kMaxK || f <= 0 || f % 16 != 0 || f > kMaxF) return NVFP4G_EINVAL;
  if (rows < 0 || rows > kMaxRows || E < 1) return NVFP4G_EINVAL;
  if (act != MOE_ACT_SILU && act != MOE_ACT_GELU) return NVFP4G_EINVAL;
  if ((rows / kBM) * ((f + cols_per_tile - 1) / cols_per_tile) > kMaxGroups) return NVFP4G_EINVAL;
  if (!O.b_data || !O.b_scale || !O.b_amax || (rows && (!O.a_data || !O.a_scale || !O.a_amax))) return NVFP4G_EINVAL;
  if (!aligned(O.a_data, 16) || !aligned(O.b_data, 16) || !aligned(O.a_scale, 4) || !aligned(O.b_scale, 4) ||
      !aligned(O.a_amax, 4) || !aligned(O.b_amax, 4))
    return NVFP4G_EALIGN;
  return NVFP4G_OK;
}

// Routing of a host-split call (d_offs NULL) or of a graph-safe one.
int make_routing(const int64_t* h_splits, const int32_t* d_offs, int32_t* d_status, int64_t rows, int32_t E,
                 bool graph, Routing* R) {
  R->num_experts = E;
  R->m_capacity = (int32_t)rows;
  R->d_offs = nullptr;
  R->d_status = nullptr;
  return graph ? graph_routing(d_offs, d_status, E, rows, R) : host_routing(h_splits, rows, E, R);
}

// Half as wide tiles where the wide ones leave at least half of the CUs idle:
// they decode a third more for an MFMA, but there are twice as many.  Forward,
// 7168 x 2 x 2048: 1024 rows (128 wide tiles) 93 us wide, 70 narrow; 2944 rows
// of 4096 x 2 x 1024 (184) 64 and 66; 65536 rows 3.03 and 3.32 ms.  Device
// routing counts the capacity's tiles: the host does not know the rows.
bool narrow(int64_t wide_tiles) { return wide_tiles <= kCus / 2; }

// The same choice for the calls with an 8-bit checkpoint, by the time that each
// kind of tile takes, in rounds of two wide tiles on a CU: one wide tile alone
// on its CU 0.6 of a round; three narrow ones on a CU 0.82, two 0.55, one 0.35.
// Forward and backward together, wide up to the rule above and by this one:
// 8192 rows, 2048 x 1040: 173 and 159 us; 4096, 2048 x 1408: 110 and 103; 8192,
// 7168 x 1280: 492 and 465; 6144, 4096 x 2048: 322 and 312.
bool narrow_by_time(int64_t wide_tiles, int64_t narrow_tiles) {
  const int64_t w = wide_tiles % (2 * kCus), n = narrow_tiles % (3 * kCus);
  const double wide = wide_tiles / (2 * kCus) + (w == 0 ? 0.0 : w <= kCus ? 0.6 : 1.0);
  const double nar = narrow_tiles / (3 * kCus) * 0.82 + (n == 0 ? 0.0 : n <= kCus ? 0.35 : n <= 2 * kCus ? 0.55 : 0.82);
  return nar < wide;
}

template <int ACT, Keep KEEP, int NW>
int launch_fwd(const Operands& O, int64_t rows, int64_t f, int64_t k, const Routing& R, uint16_t* h, uint16_t* gu,
               const Kept& K8, hipStream_t st) {
  const uint32_t ntm = (uint32_t)(rows / kBM), ntn = (uint32_t)((f + 32 * NW - 1) / (32 * NW));
  if (NW == 4 && (KEEP == kKeep8 ? narrow_by_time((int64_t)ntm * ntn, ntm * ((f + 63) / 64)) : narrow((int64_t)ntm * ntn)))
    return launch_fwd<ACT, KEEP, 2>(O, rows, f, k, R, h, gu, K8, st);
  hipLaunchKernelGGL((glu_fwd_kernel<ACT, KEEP, NW>), dim3(ntm * ntn), dim3(kThreads), 0, st, O, f, k, R, ntm, ntn, h,
                     gu, K8);
  return hip_status();
}

template <int ACT, bool KEEP8, int NW>
int launch_bwd(const Operands& O, int64_t rows, int64_t f, int64_t k, const Routing& R, const uint16_t* gu,
               const Kept& K8, uint16_t* dgu, uint16_t* again, hipStream_t st) {
  const uint32_t ntm = (uint32_t)(rows / kBM), ntn = (uint32_t)((f + 64 * NW - 1) / (64 * NW));
  if (NW == 4 && (KEEP8 ? narrow_by_time((int64_t)ntm * ntn, ntm * ((f + 127) / 128)) : narrow((int64_t)ntm * ntn)))
    return launch_bwd<ACT, KEEP8, 2>(O, rows, f, k, R, gu, K8, dgu, again, st);
  hipLaunchKernelGGL((glu_bwd_kernel<ACT, KEEP8, NW>), dim3(ntm * ntn), dim3(kThreads), 0, st, O, f, k, R, ntm, ntn, gu,
                     K8, dgu, again);
  return hip_status();
}

// How a call's rows are routed: by h_splits, or with `graph` by d_offs.
struct Route {
  const int64_t* h_splits;
  const int32_t* d_offs;
  int32_t* d_status;
  bool graph;
};

template <Keep KEEP>
int fwd(const Operands& O, int64_t rows, int64_t f, int64_t k, int32_t E, const Route& W, int32_t act, uint16_t* h,
        uint16_t* gu, const Kept& K8, void* stream) {
  int rc = check_glu(O, rows, f, k, E, act, 128);
  if (rc) return rc;
  if (rows && (!h || (KEEP == kKeep8 && (!K8.q || !K8.s)))) return NVFP4G_EINVAL;
  if (!aligned(h, 16) || !aligned(gu, 16) || !aligned(K8.q, 16) || !aligned(K8.s, 4)) return NVFP4G_EALIGN;
  Routing R;
  if ((rc = make_routing(W.h_splits, W.d_offs, W.d_status, rows, E, W.graph, &R))) return rc;
  if (rows == 0) return NVFP4G_OK;
  const hipStream_t st = (hipStream_t)stream;
  return act == MOE_ACT_SILU ? launch_fwd<MOE_ACT_SILU, KEEP, 4>(O, rows, f, k, R, h, gu, K8, st)
                             : launch_fwd<MOE_ACT_GELU, KEEP, 4>(O, rows, f, k, R, h, gu, K8, st);
}
int fwd_bf16(const Operands& O, int64_t rows, int64_t f, int64_t k, int32_t E, const Route& W, int32_t act,
             uint16_t* h, uint16_t* gu, void* stream) {
  const Kept none{nullptr, nullptr, 0};
  return gu ? fwd<kKeepBf16>(O, rows, f, k, E, W, act, h, gu, none, stream)
            : fwd<kKeepNone>(O, rows, f, k, E, W, act, h, gu, none, stream);
}

template <bool KEEP8>
int bwd(const Operands& O, int64_t rows, int64_t f, int64_t k, int32_t E, const Route& W, const uint16_t* gu,
        const Kept& K8, int32_t act, uint16_t* dgu, uint16_t* again, void* stream) {
  int rc = check_glu(O, rows, f, k, E, act, 256);
  if (rc) return rc;
  if (rows && ((KEEP8 ? !K8.q || !K8.s : !gu) || !dgu)) return NVFP4G_EINVAL;
  if (!aligned(gu, 16) || !aligned(dgu, 16) || !aligned(again, 16) || !aligned(K8.q, 16) || !aligned(K8.s, 4))
    return NVFP4G_EALIGN;
  Routing R;
  if ((rc = make_routing(W.h_splits, W.d_offs, W.d_status, rows, E, W.graph, &R))) return rc;
  if (rows == 0) return NVFP4G_OK;
  const hipStream_t st = (hipStream_t)stream;
  return act == MOE_ACT_SILU ? launch_bwd<MOE_ACT_SILU, KEEP8, 4>(O, rows, f, k, R, gu, K8, dgu, again, st)
                             : launch_bwd<MOE_ACT_GELU, KEEP8, 4>(O, rows, f, k, R, gu, K8, dgu, again, st);
}
int bwd_bf16(const Operands& O, int64_t rows, int64_t f, int64_t k, int32_t E, const Route& W, const uint16_t* gu,
             int32_t act, uint16_t* dgu, void* stream) {
  return bwd<false>(O, rows, f, k, E, W, gu, Kept{nullptr, nullptr, 0}, act, dgu, nullptr, stream);
}
// The backward pass only reads what was kept.
Kept kept_of(const int8_t* q, const uint16_t* s, int64_t rows) {
  return Kept{const_cast<int8_t*>(q), const_cast<uint16_t*>(s), rows};
}

}  // namespace

extern "C" {

int moe_glu(const uint8_t* a_data, const uint8_t* a_scale, const float* a_amax, const uint8_t* b_data,
            const uint8_t* b_scale, const float* b_amax, int64_t sum_m, int64_t f, int64_t k, int32_t num_experts,
            const int64_t* h_splits, int32_t act, uint16_t* h, uint16_t* gu, void* stream) {
  return fwd_bf16({a_data, a_scale, a_amax, b_data, b_scale, b_amax}, sum_m, f, k, num_experts,
                  {h_splits, nullptr, nullptr, false}, act, h, gu, stream);
}

int moe_glu_graphsafe(const uint8_t* a_data, const uint8_t* a_scale, const float* a_amax, const uint8_t* b_data,
                      const uint8_t* b_scale, const float* b_amax, int64_t m_capacity, int64_t f, int64_t k,
                      int32_t num_experts, const int32_t* d_offs, int32_t act, uint16_t* h, uint16_t* gu,
                      int32_t* d_status, void* stream) {
  return fwd_bf16({a_data, a_scale, a_amax, b_data, b_scale, b_amax}, m_capacity, f, k, num_experts,
                  {nullptr, d_offs, d_status, true}, act, h, gu, stream);
}

int moe_glu_bwd(const uint8_t* a_data, const uint8_t* a_scale, const float* a_amax, const uint8_t* b_data,
                const uint8_t* b_scale, const float* b_amax, int64_t sum_m, int64_t f, int64_t k, int32_t num_experts,
                const int64_t* h_splits, const uint16_t* gu, int32_t act, uint16_t* dgu, void* stream) {
  return bwd_bf16({a_data, a_scale, a_amax, b_data, b_scale, b_amax}, sum_m, f, k, num_experts,
                  {h_splits, nullptr, nullptr, false}, gu, act, dgu, stream);
}

int moe_glu_bwd_graphsafe(const uint8_t* a_data, const uint8_t* a_scale, const float* a_amax, const uint8_t* b_data,
                          const uint8_t* b_scale, const float* b_amax, int64_t m_capacity, int64_t f, int64_t k,
                          int32_t num_experts, const int32_t* d_offs, const uint16_t* gu, int32_t act, uint16_t* dgu,
                          int32_t* d_status, void* stream) {
  return bwd_bf16({a_data, a_scale, a_amax, b_data, b_scale, b_amax}, m_capacity, f, k, num_experts,
                  {nullptr, d_offs, d_status, true}, gu, act, dgu, stream);
}

int moe_glu_keep8(const uint8_t* a_data, const uint8_t* a_scale, const float* a_amax, const uint8_t* b_data,
                  const uint8_t* b_scale, const float* b_amax, int64_t sum_m, int64_t f, int64_t k,
                  int32_t num_experts, const int64_t* h_splits, int32_t act, uint16_t* h, int8_t* gu8,
                  uint16_t* gu_scale, void* stream) {
  return fwd<kKeep8>({a_data, a_scale, a_amax, b_data, b_scale, b_amax}, sum_m, f, k, num_experts,
                     {h_splits, nullptr, nullptr, false}, act, h, nullptr, {gu8, gu_scale, sum_m}, stream);
}

int moe_glu_keep8_graphsafe(const uint8_t* a_data, const uint8_t* a_scale, const float* a_amax, const uint8_t* b_data,
                            const uint8_t* b_scale, const float* b_amax, int64_t m_capacity, int64_t f, int64_t k,
                            int32_t num_experts, const int32_t* d_offs, int32_t act, uint16_t* h, int8_t* gu8,
                            uint16_t* gu_scale, int32_t* d_status, void* stream) {
  return fwd<kKeep8>({a_data, a_scale, a_amax, b_data, b_scale, b_amax}, m_capacity, f, k, num_experts,
                     {nullptr, d_offs, d_status, true}, act, h, nullptr, {gu8, gu_scale, m_capacity}, stream);
}

int moe_glu_bwd_keep8(const uint8_t* a_data, const uint8_t* a_scale, const float* a_amax, const uint8_t* b_data,
                      const uint8_t* b_scale, const float* b_amax, int64_t sum_m, int64_t f, int64_t k,
                      int32_t num_experts, const int64_t* h_splits, const int8_t* gu8, const uint16_t* gu_scale,
                      int32_t act, uint16_t* dgu, uint16_t* h, void* stream) {
  return bwd<true>({a_data, a_scale, a_amax, b_data, b_scale, b_amax}, sum_m, f, k, num_experts,
                   {h_splits, nullptr, nullptr, false}, nullptr, kept_of(gu8, gu_scale, sum_m), act, dgu, h, stream);
}

int moe_glu_bwd_keep8_graphsafe(const uint8_t* a_data, const uint8_t* a_scale, const float* a_amax,
                                const uint8_t* b_data, const uint8_t* b_scale, const float* b_amax,
                                int64_t m_capacity, int64_t f, int64_t k, int32_t num_experts, const int32_t* d_offs,
                                const int8_t* gu8, const uint16_t* gu_scale, int32_t act, uint16_t* dgu, uint16_t* h,
                                int32_t* d_status, void* stream) {
  return bwd<true>({a_data, a_scale, a_amax, b_data, b_scale, b_amax}, m_capacity, f, k, num_experts,
                   {nullptr, d_offs, d_status, true}, nullptr, kept_of(gu8, gu_scale, m_capacity), act, dgu, h,
                   stream);
}

}  // extern "C"
