// i8_gemm.hip -- products in 8-bit integers with a scale for each row and each
// channel: one projection, the experts' grouped products and their gated
// block, behind the C ABI of include/i8_group.h.
//
//   out[r, j] = (sum_c qa[r, c] qb[j, c]) * sa[r] * sb[j],   h = act(g) * u
//
// Both operands are stored along the contraction index; the int32 sums of the
// matrix instruction are exact, so the order of the contraction is free: parts
// of it may be added in any order with the same bits.
//
// What bounds it: at large sizes power (8192 x 8192 x 8192 in 410 to 450 us, 2.4 to
// 2.7 POP/s, matrix units 63% busy at a clock of 1.5 GHz; the same launch on
// zeros runs at 3.4; gated block of 65536 rows of 32 experts, 7168 x 2 x 2048: 1.62
// to 1.76 ms, 2.2 to 2.4), with few steps a tile its start and epilogue (32768 rows of
// 64 experts, 2048 x 7168, fp32: 600 to 660 us, 682 with a row of them, 1.4 to 1.6 POP/s), with few rows an
// expert the weights' way from memory (256 rows of each of 32, 7168 x 2 x 2048: 261 us,
// 3.6 TB/s), with few tiles the copies' latency.
#include "i8_choice.hpp"
#include "i8_token.hpp"

namespace {

using namespace i8;

// A work-group's tile: WM x WN waves of TM x TN MFMA tiles (32 x 32 each), BK
// bytes of a line in a stage, NS stages in LDS, OCC waves on a SIMD.
template <int WM_, int WN_, int TM_, int TN_, int BK_, int NS_, int OCC_>
struct Shape {
  static constexpr int WM = WM_, WN = WN_, TM = TM_, TN = TN_, BK = BK_, NS = NS_, OCC = OCC_;
  static constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;
  static constexpr int BM = 32 * WM * TM, BN = 32 * WN * TN;
  static constexpr int kStageBytes = (BM + BN) * BK;
  static constexpr int kSlots = BK / 16;             // 16-byte granules of a line in a stage
  static constexpr int kWaveLines = 64 / kSlots;     // lines of a wave's copy
  static constexpr int kCopyLines = kWaveLines * kWaves;
  static constexpr int kCopiesA = BM / kCopyLines, kCopiesB = BN / kCopyLines, kCopies = kCopiesA + kCopiesB;
  static_assert(BM % kCopyLines == 0 && BN % kCopyLines == 0 && kCopyLines % 16 == 0, "copies are whole");
  static_assert(NS == 2 || NS == 4, "stages");
};

// One operand: the lines of a tile, `valid` (at least 1) of which exist (others read 0).
struct Lines {
  const int8_t* data;
  uint32_t valid;
};

// 16-byte granule q of a line sits at a slot that makes sixteen consecutive
// lines at one granule, which an LDS read serves at once, meet all 64 banks:
// two lines of 128 bytes, or four of 64, go once around them.
template <class S>
__device__ __forceinline__ uint32_t swz(uint32_t line, uint32_t q) {
  return S::BK == 128 ? q ^ ((line >> 1) & 7u) : q ^ ((line >> 2) & 3u);
}

// The stages in LDS: arrays of their own, so that reads of one need not wait
// for copies into the others.
template <class S>
struct Stages {
  uint8_t *p0, *p1, *p2, *p3;
  template <int I>
  __device__ __forceinline__ uint8_t* at() const {
    constexpr int i = I % S::NS;
    return i == 0 ? p0 : i == 1 ? p1 : i == 2 ? p2 : p3;
  }
};

// N products, then one copy, C times.
template <int N, int C, int I = 0>
__device__ __forceinline__ void spread_copies() {
  if constexpr (I < C) {
    __builtin_amdgcn_sched_group_barrier(0x008, (I + 1) * N / C - I * N / C, 0);
    __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);
    spread_copies<N, C, I + 1>();
  }
}
// R reads of a substep's fragments between the N products of the one before.
template <int N, int R, int I = 0>
__device__ __forceinline__ void spread_reads() {
  if constexpr (I < R) {
    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x008, (I + 1) * N / R - I * N / R, 0);
    spread_reads<N, R, I + 1>();
  }
}

// All waves: this wave's LDS reads are done and at most N of its copies are
// still on their way.
template <int N>
__device__ __forceinline__ void stage_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (0 << 8) | ((N >> 4) << 14));
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// acc[im][in] = B lines x A lines^T over steps ks0 .. ks1 - 1 of the
// contraction: a lane has one row of A (lane % 32) and in its sixteen sums the B
// lines 8 (v / 4) + 4 (lane / 32) + v % 4, four neighbours at a time.  PAIR: B's LDS lines are blocks of 16 TN lines, alternately of
// B0 (gate) and of B1 (up), so that a wave's first TN / 2 tiles are gate lines
// and the others the up lines of the same columns.  The granules of a line's
// last step past k are copied as zeros.
//
// Fragments are read one substep ahead.  Before the last substep of a step one
// barrier says that its stage is read by all and that the next one has landed;
// behind it the copies of the step NS ahead go into the free stage, between the
// products, and the next stage's first fragments are read.  Steps past the last
// are copied too, as zeros without a look at memory: the compiler then knows how
// many copies are on their way everywhere in the loop, and adds no waits.
// A wave whose rows or columns are all past the last (`live` false) copies and
// waits with the others but multiplies nothing.
template <class S, bool PAIR>
struct Multiply {
  const Lines &A, &B0, &B1;
  uint32_t k, ks0, ks1;
  Stages<S> L;
  rsrc_t ar, b0r, b1r;
  uint32_t wave, lane, cl, granule, nk, cut;

  __device__ __forceinline__ Multiply(const Lines& a, const Lines& b0, const Lines& b1, uint32_t k_, uint32_t first,
                                      uint32_t end, Stages<S> l)
      : A(a), B0(b0), B1(b1), k(k_), ks0(first), ks1(end), L(l) {
    ar = range_rsrc(A.data, (int64_t)A.valid * k);
    b0r = range_rsrc(B0.data, (int64_t)B0.valid * k);
    b1r = PAIR ? range_rsrc(B1.data, (int64_t)B1.valid * k) : b0r;
    wave = uni((uint32_t)(threadIdx.x >> 6));
    lane = threadIdx.x & 63;
    cl = S::kWaveLines * wave + lane / S::kSlots;  // line of the first copy
    granule = swz<S>(cl, lane % S::kSlots);
    nk = (k + S::BK - 1) / S::BK;
    cut = (nk - 1) * S::BK + 16 * granule >= k ? kOutOfRange : 0u;
  }

  __device__ __forceinline__ void issue(uint32_t ks, uint8_t* base) const {
    constexpr uint32_t kBlock = 16 * S::TN;
    static_assert(!PAIR || kBlock % S::kWaveLines == 0, "a wave's copy stays in a block");
    const uint32_t so = min(ks, nk - 1) * S::BK, past = ks >= ks1 ? kOutOfRange : ks + 1 == nk ? cut : 0u;
#pragma unroll
    for (int c = 0; c < S::kCopiesA; ++c)
      copy16(ar, base + (c * S::kCopyLines + S::kWaveLines * wave) * S::BK,
             ((c * S::kCopyLines + cl) * k + 16 * granule) | past, so);
#pragma unroll
    for (int c = 0; c < S::kCopiesB; ++c) {
      const uint32_t at = c * S::kCopyLines + cl;
      const bool up = PAIR && ((c * S::kCopyLines + S::kWaveLines * wave) / kBlock) % 2;  // the same for a wave's lines
      const uint32_t line = PAIR ? at / kBlock / 2 * kBlock + at % kBlock : at;
      copy16(up ? b1r : b0r, base + (S::BM + c * S::kCopyLines + S::kWaveLines * wave) * S::BK,
             (line * k + 16 * granule) | past, so);
    }
  }

  template <bool LIVE>
  __device__ __forceinline__ void run(i32x16 (&acc)[S::TM][S::TN]) const {
    const uint32_t wm = wave / S::WN, wn = wave % S::WN, h = lane >> 5;
    const uint32_t la = wm * (32 * S::TM) + (lane & 31), lb = S::BM + wn * (32 * S::TN) + (lane & 31);
    constexpr int kSub = S::BK / 32, kReads = S::TM + S::TN, kMul = S::TM * S::TN;
    i32x4 a[2][S::TM], b[2][S::TN];
    auto read = [&](const uint8_t* base, int s, int to) {
      const uint32_t q = 16 * swz<S>(lane, 2 * s + h);
#pragma unroll
      for (int im = 0; im < S::TM; ++im) a[to][im] = *reinterpret_cast<const i32x4*>(base + (la + 32 * im) * S::BK + q);
#pragma unroll
      for (int in = 0; in < S::TN; ++in) b[to][in] = *reinterpret_cast<const i32x4*>(base + (lb + 32 * in) * S::BK + q);
    };
    auto products = [&](int from) {
#pragma unroll
      for (int im = 0; im < S::TM; ++im)
#pragma unroll
        for (int in = 0; in < S::TN; ++in)
          acc[im][in] = __builtin_amdgcn_mfma_i32_32x32x32_i8(b[from][in], a[from][im], acc[im][in], 0, 0, 0);
    };
    auto step = [&](uint32_t ks, uint8_t* base, const uint8_t* next) {
      if (LIVE) {
#pragma unroll
        for (int s = 0; s + 1 < kSub; ++s) {
          read(base, s + 1, (s + 1) & 1);
          products(s & 1);
          spread_reads<kMul, kReads>();
        }
      }
      stage_barrier<(S::NS - 2) * S::kCopies>();
      if (LIVE) {
        read(next, 0, 0);
        products((kSub - 1) & 1);
      }
      issue(ks + S::NS, base);
      if (LIVE) {
        __builtin_amdgcn_sched_group_barrier(0x100, kReads, 0);
        spread_copies<kMul, S::kCopies>();
      }
    };
    issue(ks0, L.template at<0>());
    issue(ks0 + 1, L.template at<1>());
    if (S::NS > 2) issue(ks0 + 2, L.template at<2>());
    if (S::NS > 2) issue(ks0 + 3, L.template at<3>());
    stage_barrier<(S::NS - 1) * S::kCopies>();
    if (LIVE) read(L.template at<0>(), 0, 0);
    uint32_t ks = ks0;
#pragma unroll 1
    for (; ks + S::NS <= ks1; ks += S::NS) {
      step(ks, L.template at<0>(), L.template at<1>());
      step(ks + 1, L.template at<1>(), L.template at<2>());
      if (S::NS == 2) continue;
      step(ks + 2, L.template at<2>(), L.template at<3>());
      step(ks + 3, L.template at<3>(), L.template at<0>());
    }
    if (ks < ks1) step(ks, L.template at<0>(), L.template at<1>());
    if (S::NS > 2 && ks + 1 < ks1) step(ks + 1, L.template at<1>(), L.template at<2>());
    if (S::NS > 2 && ks + 2 < ks1) step(ks + 2, L.template at<2>(), L.template at<3>());
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
    __syncthreads();
  }
};

// Logical tile: super-tiles of 64 consecutive tiles dealt round-robin to the
// 8 XCDs, so that each XCD's L2 holds the operand slices its tiles share.
__device__ __forceinline__ uint32_t xcd_tile() {
  const uint32_t id = blockIdx.x, T = gridDim.x;
  const uint32_t round = kNumXcd * 64, full = (T / round) * round;
  if (id >= full) return uni(id);
  const uint32_t j = id / kNumXcd, x = id % kNumXcd;
  return uni((kNumXcd * (j / 64) + x) * 64 + j % 64);
}
constexpr int kGroupRows = 8;  // row tiles that sweep the column tiles together
__device__ __forceinline__ void grouped_tile(uint32_t t, uint32_t ntm, uint32_t ntn, uint32_t* tm, uint32_t* tn) {
  const uint32_t g = t / (kGroupRows * ntn), in = t % (kGroupRows * ntn);
  const uint32_t first = g * kGroupRows, gm = min((uint32_t)kGroupRows, ntm - first);
  *tm = uni(first + in % gm);
  *tn = uni(in / gm);
}

// Rows of row tile t: BM of one expert, or what is left of it.  One projection
// is an expert that owns all rows (dense).
struct RowTile {
  int32_t expert;
  int64_t row0;
  int32_t rows;
};
template <int BM>
__device__ __forceinline__ bool row_tile(const Routing& R, bool dense, uint32_t t, RowTile* out) {
  if (dense) {
    const int64_t row0 = (int64_t)t * BM;
    *out = RowTile{0, row0, (int32_t)min<int64_t>(BM, R.m_capacity - row0)};
    return out->rows > 0;
  }
  if (BM <= kTileRows) {  // whole tiles: groups are multiples of 128 rows
    const int32_t row0 = (int32_t)(t * BM);
    if (row0 >= route_end(R, R.num_experts - 1)) return false;
    int32_t b, e;
    const int ex = find_expert(R, row0, &b, &e);
    *out = RowTile{ex, row0, BM};
    return true;
  }
  // an expert has ceil(rows / BM) tiles: 64 experts at a time count theirs
  const int lane = threadIdx.x & 63, E = R.num_experts;
  uint32_t before = 0;
  for (int e0 = 0; e0 < E; e0 += 64) {
    const int e = e0 + lane;
    const int32_t end = e < E ? route_end_lane(R, e) : 0, beg = e < E && e ? route_end_lane(R, e - 1) : 0;
    const uint32_t mine = e < E ? (uint32_t)(end - beg + BM - 1) / BM : 0;
    uint32_t upto = mine;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const uint32_t o = __shfl_up(upto, d);
      if (lane >= d) upto += o;
    }
    const uint64_t hit = __ballot(before + upto > t);
    if (hit) {
      const int f = __ffsll((unsigned long long)hit) - 1;
      const int32_t fb = __shfl(beg, f), fe = __shfl(end, f);
      const uint32_t first = before + __shfl(upto - mine, f);
      const int32_t row0 = uni(fb + (int32_t)(t - first) * BM);
      *out = RowTile{uni(e0 + f), row0, uni(min(BM, fe - row0))};
      return true;
    }
    before += __shfl(upto, 63);
  }
  return false;
}

// A wave's own piece of a stage, free in the epilogue: 32 rows x COLS columns go
// in four neighbours at a time, as the sums lie in the lanes, and come out as 16
// bytes a lane of whole row pieces.  Pitches: the rows that an LDS access serves
// at once (32 of 8 bytes, 16 of 16) meet all 64 banks.
template <int COLS, int SIZE>
struct RowStage {
  static constexpr int kPitch = COLS * SIZE + 4 * SIZE;
  static constexpr int kBytes = 32 * kPitch;
  uint8_t* p;
  __device__ __forceinline__ uint8_t* at(int row, int col) const { return p + row * kPitch + SIZE * col; }
};
// Orders a wave's own LDS writes and reads (they run in issue order).
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

struct Operands {
  const int8_t* a_q;
  const float* a_scale;
  const int8_t* b_q;
  const float* b_scale;
};

// n: columns of the output (f of the gated block, whose experts have 2f lines).
// With kParts a work-group sums `per` steps of the contraction: part p of a tile
// writes its int32 sums to out [parts, rows, n].
template <class S, Epilogue EPI>
__global__ __launch_bounds__(S::kThreads, S::OCC) void product_kernel(Operands O, int64_t n, int64_t k, Routing R,
                                                                      bool dense, uint32_t ntm, uint32_t ntn,
                                                                      uint32_t per, void* __restrict__ out) {
  constexpr bool GLU = is_glu(EPI);
  constexpr int kCols = GLU ? S::BN / 2 : S::BN, kWaveCols = kCols / S::WN, BLK = kWaveCols / 32;
  __shared__ __attribute__((aligned(16))) uint8_t lds0[S::kStageBytes];
  __shared__ __attribute__((aligned(16))) uint8_t lds1[S::kStageBytes];
  __shared__ __attribute__((aligned(16))) uint8_t lds2[S::NS > 2 ? S::kStageBytes : 16];
  __shared__ __attribute__((aligned(16))) uint8_t lds3[S::NS > 2 ? S::kStageBytes : 16];
  __shared__ __attribute__((aligned(16))) float lsb[S::BN];
  if (!routing_ok(R)) return;
  uint32_t tm, tn, t = xcd_tile(), part = 0;
  if (EPI == kParts) {  // the parts of a tile side by side
    const uint32_t parts = uni(gridDim.x / (ntm * ntn));
    part = uni(t % parts);
    t = uni(t / parts);
  }
  grouped_tile(t, ntm, ntn, &tm, &tn);
  RowTile T;
  if (!row_tile<S::BM>(R, dense, tm, &T)) return;
  const int64_t col0 = (int64_t)tn * kCols;
  const uint32_t cols = (uint32_t)min<int64_t>(n - col0, kCols);
  const int64_t line0 = (int64_t)T.expert * (GLU ? 2 * n : n) + col0;
  const Lines A{O.a_q + T.row0 * k, (uint32_t)T.rows};
  const Lines B0{O.b_q + line0 * k, cols}, B1{O.b_q + (line0 + (GLU ? n : 0)) * k, cols};
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = uni((int32_t)(tid >> 6)), wm = wave / S::WN, wn = wave % S::WN;
  const bool live = wn * kWaveCols < (int)cols && wm * (32 * S::TM) < T.rows;
  i32x16 acc[S::TM][S::TN];
#pragma unroll
  for (int im = 0; im < S::TM; ++im)
#pragma unroll
    for (int in = 0; in < S::TN; ++in) acc[im][in] = i32x16{};
  // scales are on their way beside the first copies, and wait in registers: a
  // lane has its rows', a thread one line's, in the order of the stage
  static_assert(S::kThreads >= S::BN, "a thread has a line's scale");
  float sa[S::TM], line_scale = 0.0f;
#pragma unroll
  for (int im = 0; im < S::TM; ++im) {
    const int r = wm * (32 * S::TM) + 32 * im + (lane & 31);
    sa[im] = EPI != kParts && r < T.rows ? O.a_scale[T.row0 + r] : 0.0f;
  }
  if (EPI != kParts && tid < S::BN) {
    const int j = GLU ? tid / (32 * S::TN) * kWaveCols + tid % kWaveCols : tid;
    const bool up = GLU && tid % (32 * S::TN) >= kWaveCols;
    if (j < (int)cols) line_scale = O.b_scale[line0 + (up ? n : 0) + j];
  }
  const uint32_t nk = (uint32_t)((k + S::BK - 1) / S::BK);
  const uint32_t ks0 = EPI == kParts ? part * per : 0, ks1 = EPI == kParts ? min(ks0 + per, nk) : nk;
  const Multiply<S, GLU> M(A, B0, B1, (uint32_t)k, ks0, ks1, Stages<S>{lds0, lds1, lds2, lds3});
  if (live) M.template run<true>(acc);
  else M.template run<false>(acc);
  if (EPI != kParts) {
    if (tid < S::BN) lsb[tid] = line_scale;
    __syncthreads();
  }
  if (!live) return;

  constexpr int SIZE = EPI == kOutF32 || EPI == kParts ? 4 : 2;  // bytes of an output
  using Rows = RowStage<kWaveCols, SIZE>;
  constexpr int kShare = (S::kWaves + S::NS - 1) / S::NS;  // waves of a stage
  static_assert(kShare * Rows::kBytes <= S::kStageBytes, "the waves' rows fit the stages");
  const int own = wave / kShare;
  const Rows stage{(own == 0 ? lds0 : own == 1 ? lds1 : own == 2 ? lds2 : lds3) + (wave % kShare) * Rows::kBytes};
  constexpr int kPer = 16 / SIZE, kLanes = kWaveCols / kPer, kRows = 64 / kLanes;  // columns of a lane's store, lanes of a row, rows of a store
  const int c = kPer * (lane % kLanes), srow = lane / kLanes;
  const bool inside = wn * kWaveCols + c < (int)cols;
  f32x4 sb[S::TN][4];
#pragma unroll
  for (int in = 0; in < S::TN; ++in)
#pragma unroll
    for (int q = 0; q < 4; ++q)
      sb[in][q] = *reinterpret_cast<const f32x4*>(&lsb[wn * (32 * S::TN) + 32 * in + 8 * q + 4 * (lane >> 5)]);
  const int64_t first = EPI == kParts ? part * (int64_t)R.m_capacity : 0;
#pragma unroll
  for (int im = 0; im < S::TM; ++im) {
    const int r0 = wm * (32 * S::TM) + 32 * im;
#pragma unroll
    for (int in = 0; in < BLK; ++in)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint8_t* to = stage.at(lane & 31, 32 * in + 8 * q + 4 * (lane >> 5));
        if constexpr (EPI == kParts) {
          *reinterpret_cast<i32x4*>(to) = i32x4{acc[im][in][4 * q], acc[im][in][4 * q + 1], acc[im][in][4 * q + 2], acc[im][in][4 * q + 3]};
        } else {
          f32x4 y;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            y[i] = ((float)acc[im][in][4 * q + i] * sa[im]) * sb[in][q][i];
            if constexpr (GLU) {
              const float u = ((float)acc[im][in + BLK][4 * q + i] * sa[im]) * sb[in + BLK][q][i];
              float dv;
              y[i] = y[i] * act_logistic<EPI == kGluSilu ? MOE_ACT_SILU : MOE_ACT_GELU>(y[i], &dv) * u;
            }
          }
          if constexpr (SIZE == 4) *reinterpret_cast<f32x4*>(to) = y;
          else *reinterpret_cast<u32x2*>(to) = u32x2{pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3])};
        }
      }
    wave_sync();
#pragma unroll
    for (int r = 0; r < 32; r += kRows) {
      const uint8_t* from = stage.at(r + srow, c);
      const u32x2 lo = *reinterpret_cast<const u32x2*>(from), hi = *reinterpret_cast<const u32x2*>(from + 8);
      const int64_t at = (first + T.row0 + r0 + r + srow) * n + col0 + wn * kWaveCols + c;
      if (inside && r0 + r + srow < T.rows) {
        u32x4* to = reinterpret_cast<u32x4*>(reinterpret_cast<uint8_t*>(out) + SIZE * at);
        const u32x4 v = {lo[0], lo[1], hi[0], hi[1]};
        // results past the caches, which keep the operands (in turn, 32768 rows, 2048 x 7168, fp32: 604 us and 614;
        // 2048 x 2048 x 2048: 14.3 and 14.9); parts are read again at once
        if (EPI == kParts) *to = v;
        else __builtin_nontemporal_store(v, to);
      }
    }
    wave_sync();
  }
}

// Adds the parts of a projection and applies the scales: four columns a lane.
template <bool F32OUT>
__global__ __launch_bounds__(kThreads) void join_kernel(const int32_t* __restrict__ parts, int nparts, int64_t rows,
                                                        int64_t n, const float* __restrict__ a_scale,
                                                        const float* __restrict__ b_scale, void* __restrict__ out) {
  const int64_t at = 4 * ((int64_t)line_index() * kThreads + threadIdx.x);
  if (at >= rows * n) return;
  const int64_t r = at / n, c = at - r * n;
  i32x4 s = *reinterpret_cast<const i32x4*>(parts + at);
  for (int p = 1; p < nparts; ++p) s += *reinterpret_cast<const i32x4*>(parts + p * rows * n + at);
  const float sa = a_scale[r];
  float y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = ((float)s[i] * sa) * b_scale[c + i];
  if (F32OUT)
    *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(out) + at) = f32x4{y[0], y[1], y[2], y[3]};
  else
    *reinterpret_cast<u32x2*>(reinterpret_cast<uint16_t*>(out) + at) = u32x2{pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3])};
}

// ------------------------------------------------------------- host side

template <class S, Epilogue EPI>
int launch(const Operands& O, int64_t rows, int64_t n, int64_t k, const Routing& R, bool dense, int parts, int64_t per,
           void* out, hipStream_t st) {
  constexpr int kCols = is_glu(EPI) ? S::BN / 2 : S::BN;
  const int64_t ntm = row_tiles<S::BM>(R, dense, rows), ntn = (n + kCols - 1) / kCols, wgs = ntm * ntn * parts;
  if (wgs > (1ll << 32) / S::kThreads - 1) return NVFP4G_EINVAL;
  hipLaunchKernelGGL((product_kernel<S, EPI>), dim3((uint32_t)wgs), dim3(S::kThreads), 0, st, O, n, k, R, dense,
                     (uint32_t)ntm, (uint32_t)ntn, (uint32_t)per, out);
  return hip_status();
}

// The tiles a call can take (i8_choice.hpp says which and when).
using Big = Shape<2, 4, 4, 2, 128, 2, 2>;
using Mid = Shape<2, 2, 2, 2, 128, 2, 2>;
using Mid4 = Shape<2, 2, 2, 2, 128, 4, 1>;

template <Epilogue EPI>
int product(const Operands& O, int64_t rows, int64_t n, int64_t k, const Routing& R, bool dense, void* out,
            void* workspace, hipStream_t st) {
  const Choice c = choose<EPI>(rows, n, k, R, dense, workspace ? kMaxWorkspace : 0);
  if (c.shape == 0) return launch<Big, EPI>(O, rows, n, k, R, dense, 1, 0, out, st);
  if (c.shape == 1) return launch<Mid, EPI>(O, rows, n, k, R, dense, 1, 0, out, st);
  if (c.parts == 1) return launch<Mid4, EPI>(O, rows, n, k, R, dense, 1, 0, out, st);
  if constexpr (!is_glu(EPI)) {
    const int rc = launch<Mid4, kParts>(O, rows, n, k, R, dense, c.parts, c.per, workspace, st);
    if (rc) return rc;
    hipLaunchKernelGGL((join_kernel<EPI == kOutF32>), line_grid((uint32_t)((rows * n / 4 + kThreads - 1) / kThreads)),
                       dim3(kThreads), 0, st, (const int32_t*)workspace, c.parts, rows, n, O.a_scale, O.b_scale, out);
    return hip_status();
  }
  return NVFP4G_EINVAL;
}

int check(const Operands& O, int64_t rows, int64_t lines, int64_t k, int32_t E, const void* out) {
  if (!valid_k(k) || !valid_n(lines) || rows < 0 || rows > kMaxRows || E < 1) return NVFP4G_EINVAL;
  if (!O.b_q || !O.b_scale || (rows && (!O.a_q || !O.a_scale || !out))) return NVFP4G_EINVAL;
  if (!aligned(O.a_q, 16) || !aligned(O.b_q, 16) || !aligned(out, 16) || !aligned(O.a_scale, 4) ||
      !aligned(O.b_scale, 4))
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

int gemm(const Operands& O, int64_t rows, int64_t n, int64_t k, int32_t E, const int64_t* h_splits,
         const int32_t* d_offs, int32_t* d_status, bool graph, void* out, int32_t out_type, void* stream) {
  int rc = check(O, rows, n, k, E, out);
  if (rc) return rc;
  if (!valid_type(out_type)) return NVFP4G_EINVAL;
  Routing R;
  if ((rc = make_routing(h_splits, d_offs, d_status, rows, E, graph, &R))) return rc;
  if (rows == 0) return NVFP4G_OK;
  return out_type == MOE_F32 ? product<kOutF32>(O, rows, n, k, R, false, out, nullptr, (hipStream_t)stream)
                             : product<kOutBf16>(O, rows, n, k, R, false, out, nullptr, (hipStream_t)stream);
}

int glu(const Operands& O, int64_t rows, int64_t f, int64_t k, int32_t E, const int64_t* h_splits,
        const int32_t* d_offs, int32_t* d_status, bool graph, int32_t act, uint16_t* h, void* stream) {
  if (f <= 0 || f % 16 != 0 || f > (1 << 19)) return NVFP4G_EINVAL;
  if (act != MOE_ACT_SILU && act != MOE_ACT_GELU) return NVFP4G_EINVAL;
  int rc = check(O, rows, 2 * f, k, E, h);
  if (rc) return rc;
  Routing R;
  if ((rc = make_routing(h_splits, d_offs, d_status, rows, E, graph, &R))) return rc;
  if (rows == 0) return NVFP4G_OK;
  return act == MOE_ACT_SILU ? product<kGluSilu>(O, rows, f, k, R, false, h, nullptr, (hipStream_t)stream)
                             : product<kGluGelu>(O, rows, f, k, R, false, h, nullptr, (hipStream_t)stream);
}

}  // namespace

extern "C" {

// Grows with the rows, so that it serves every smaller batch too.
int64_t i8_linear_workspace(int64_t rows, int64_t k, int64_t n) {
  if (rows < 0 || rows > kMaxRows || !valid_k(k) || !valid_n(n)) return NVFP4G_EINVAL;
  return rows <= kFewRows && few(rows, k) ? 0 : std::min<int64_t>(kMaxWorkspace, kMaxParts * rows * n * 4);
}

int i8_linear(const int8_t* a_q, const float* a_scale, int64_t rows, int64_t k, const int8_t* b_q,
              const float* b_scale, int64_t n, void* out, int32_t out_type, void* workspace, int64_t workspace_bytes,
              void* stream) {
  const Operands O{a_q, a_scale, b_q, b_scale};
  const int rc = check(O, rows, n, k, 1, out);
  if (rc) return rc;
  if (!valid_type(out_type)) return NVFP4G_EINVAL;
  const int64_t need = i8_linear_workspace(rows, k, n);
  if (need && (!workspace || workspace_bytes < need)) return NVFP4G_EINVAL;
  if (!aligned(workspace, 16)) return NVFP4G_EALIGN;
  if (rows == 0) return NVFP4G_OK;
  if (few(rows, k)) return few_rows(a_q, a_scale, rows, k, b_q, b_scale, n, out, out_type, (hipStream_t)stream);
  Routing R;
  R.num_experts = 1;
  R.m_capacity = (int32_t)rows;
  R.d_offs = nullptr;
  R.d_status = nullptr;
  return out_type == MOE_F32 ? product<kOutF32>(O, rows, n, k, R, true, out, workspace, (hipStream_t)stream)
                             : product<kOutBf16>(O, rows, n, k, R, true, out, workspace, (hipStream_t)stream);
}

int i8_group_gemm(const int8_t* a_q, const float* a_scale, const int8_t* b_q, const float* b_scale, int64_t sum_m,
                  int64_t n, int64_t k, int32_t num_experts, const int64_t* h_splits, void* out, int32_t out_type,
                  void* stream) {
  return gemm({a_q, a_scale, b_q, b_scale}, sum_m, n, k, num_experts, h_splits, nullptr, nullptr, false, out, out_type,
              stream);
}

int i8_group_gemm_graphsafe(const int8_t* a_q, const float* a_scale, const int8_t* b_q, const float* b_scale,
                            int64_t m_capacity, int64_t n, int64_t k, int32_t num_experts, const int32_t* d_offs,
                            void* out, int32_t out_type, int32_t* d_status, void* stream) {
  return gemm({a_q, a_scale, b_q, b_scale}, m_capacity, n, k, num_experts, nullptr, d_offs, d_status, true, out,
              out_type, stream);
}

int i8_group_glu(const int8_t* a_q, const float* a_scale, const int8_t* b_q, const float* b_scale, int64_t sum_m,
                 int64_t f, int64_t k, int32_t num_experts, const int64_t* h_splits, int32_t act, uint16_t* h,
                 void* stream) {
  return glu({a_q, a_scale, b_q, b_scale}, sum_m, f, k, num_experts, h_splits, nullptr, nullptr, false, act, h,
             stream);
}

int i8_group_glu_graphsafe(const int8_t* a_q, const float* a_scale, const int8_t* b_q, const float* b_scale,
                           int64_t m_capacity, int64_t f, int64_t k, int32_t num_experts, const int32_t* d_offs,
                           int32_t act, uint16_t* h, int32_t* d_status, void* stream) {
  return glu({a_q, a_scale, b_q, b_scale}, m_capacity, f, k, num_experts, nullptr, d_offs, d_status, true, act, h,
             stream);
}

}  // extern "C"
