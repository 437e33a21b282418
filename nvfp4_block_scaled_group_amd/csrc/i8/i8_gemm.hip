// i8_gemm.hip -- products in 8-bit integers with a scale for each row and each
// channel: one projection, the experts' grouped products and their gated
// block, behind the C ABI of include/i8_group.h.
//
//   out[r, j] = (sum_c qa[r, c] qb[j, c]) * sa[r] * sb[j],   h = act(g) * u
//
// Both operands are stored along the contraction index; the int32 sums of the
// matrix instruction are exact, so the order of the contraction is free.
#include <algorithm>

#include "i8_common.hpp"

namespace {

using namespace i8;

constexpr int kBK = 128;  // contraction step: bytes (and elements) of a line in a stage

enum Epilogue { kOutF32, kOutBf16, kGluSilu, kGluGelu };
constexpr bool is_glu(Epilogue e) { return e == kGluSilu || e == kGluGelu; }

// A work-group's tile: WM x WN waves of TM x TN MFMA tiles (32 x 32 each).
template <int WM_, int WN_, int TM_, int TN_>
struct Shape {
  static constexpr int WM = WM_, WN = WN_, TM = TM_, TN = TN_;
  static constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;
  static constexpr int BM = 32 * WM * TM, BN = 32 * WN * TN;
  static constexpr int kStageBytes = (BM + BN) * kBK;
  static constexpr int kCopyLines = 8 * kWaves;  // of one copy: 8 lines of 128 bytes a wave
  static constexpr int kCopiesA = BM / kCopyLines, kCopiesB = BN / kCopyLines;
  static_assert(BM % kCopyLines == 0 && BN % kCopyLines == 0, "copies are whole");
};

// One operand: the lines of a tile, `valid` (at least 1) of which exist (others read 0).
struct Lines {
  const int8_t* data;
  uint32_t valid;
};

// 16-byte granule q of a line sits at slot q ^ (line % 8): a fragment read of
// 32 consecutive lines at one granule then spreads over all banks.
__device__ __forceinline__ uint32_t swz(uint32_t line, uint32_t q) { return q ^ (line & 7u); }

// acc[im][in] = A lines x B lines^T over k.  PAIR: B's LDS lines are blocks of
// 16 TN lines, alternately of B0 (gate) and of B1 (up), so that a wave's first
// TN / 2 tiles are gate lines and the others the up lines of the same columns.
// Each step waits for its own copies, passes one barrier, issues the copies of
// the next step into the other stage and multiplies meanwhile.  The granules of
// a line's last step past k are copied as zeros.
template <class S, bool PAIR>
__device__ __forceinline__ void multiply(const Lines& A, const Lines& B0, const Lines& B1, uint32_t k, bool live,
                                         i32x16 (&acc)[S::TM][S::TN], uint8_t* lds0, uint8_t* lds1) {
  const int tid = threadIdx.x, lane = tid & 63;
  const uint32_t wave = uni((uint32_t)(tid >> 6));
  const rsrc_t ar = range_rsrc(A.data, (int64_t)A.valid * k), b0r = range_rsrc(B0.data, (int64_t)B0.valid * k);
  const rsrc_t b1r = PAIR ? range_rsrc(B1.data, (int64_t)B1.valid * k) : b0r;
  constexpr uint32_t kBlock = 16 * S::TN;
  const uint32_t cl = 8 * wave + (lane >> 3), granule = swz(cl, lane & 7);  // line of the first copy; its granule
  const uint32_t nk = (k + kBK - 1) / kBK;
  const uint32_t cut = (nk - 1) * kBK + 16 * granule >= k ? kOutOfRange : 0u;

  auto issue = [&](uint32_t ks, uint8_t* base) {
    const uint32_t so = ks * kBK, past = ks + 1 == nk ? cut : 0u;
#pragma unroll
    for (int c = 0; c < S::kCopiesA; ++c)
      copy16(ar, base + (c * S::kCopyLines + 8 * wave) * kBK, ((c * S::kCopyLines + cl) * k + 16 * granule) | past, so);
#pragma unroll
    for (int c = 0; c < S::kCopiesB; ++c) {
      const uint32_t at = c * S::kCopyLines + cl;
      const bool up = PAIR && ((c * S::kCopyLines + 8 * wave) / kBlock) % 2;  // the same for a wave's 8 lines
      const uint32_t line = PAIR ? at / kBlock / 2 * kBlock + at % kBlock : at;
      copy16(up ? b1r : b0r, base + (S::BM + c * S::kCopyLines + 8 * wave) * kBK, (line * k + 16 * granule) | past, so);
    }
  };

  const uint32_t wm = wave / S::WN, wn = wave % S::WN, h = lane >> 5;
  const uint32_t la = wm * (32 * S::TM) + (lane & 31), lb = S::BM + wn * (32 * S::TN) + (lane & 31);
  auto step = [&](uint32_t ks, const uint8_t* base, uint8_t* next) {
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
    __syncthreads();
    if (ks + 1 < nk) issue(ks + 1, next);
    if (!live) return;
#pragma unroll
    for (int s = 0; s < kBK / 32; ++s) {
      const uint32_t q = 16 * swz(lane, 2 * s + h);
      i32x4 a[S::TM], b[S::TN];
#pragma unroll
      for (int im = 0; im < S::TM; ++im) a[im] = *reinterpret_cast<const i32x4*>(base + (la + 32 * im) * kBK + q);
#pragma unroll
      for (int in = 0; in < S::TN; ++in) b[in] = *reinterpret_cast<const i32x4*>(base + (lb + 32 * in) * kBK + q);
#pragma unroll
      for (int im = 0; im < S::TM; ++im)
#pragma unroll
        for (int in = 0; in < S::TN; ++in)
          acc[im][in] = __builtin_amdgcn_mfma_i32_32x32x32_i8(a[im], b[in], acc[im][in], 0, 0, 0);
    }
  };
  issue(0, lds0);
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

// A wave's own half of a stage, free in the epilogue: 32 rows x COLS columns of
// fp32 go in as the MFMA layout holds them (column in the lane) and come out as
// consecutive columns of a row, so that memory sees 16 bytes a lane.
template <int COLS>
struct RowStage {
  static constexpr int kPitch = COLS + 8;  // floats: the two lane halves, 4 rows apart, on different banks
  static constexpr int kBytes = 32 * kPitch * 4;
  float* p;
  __device__ __forceinline__ void put(int block, int v, int lane, float x) {
    p[(8 * (v >> 2) + 4 * (lane >> 5) + (v & 3)) * kPitch + 32 * block + (lane & 31)] = x;
  }
  __device__ __forceinline__ f32x4 get4(int row, int col) const {
    return *reinterpret_cast<const f32x4*>(p + row * kPitch + col);
  }
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
template <class S, Epilogue EPI, int OCC>
__global__ __launch_bounds__(S::kThreads, OCC) void product_kernel(Operands O, int64_t n, int64_t k, Routing R,
                                                                   bool dense, uint32_t ntm, uint32_t ntn,
                                                                   void* __restrict__ out) {
  constexpr bool GLU = is_glu(EPI);
  constexpr int kCols = GLU ? S::BN / 2 : S::BN, kWaveCols = kCols / S::WN, BLK = kWaveCols / 32;
  __shared__ __attribute__((aligned(16))) uint8_t lds0[S::kStageBytes];
  __shared__ __attribute__((aligned(16))) uint8_t lds1[S::kStageBytes];
  __shared__ float lsa[S::BM];
  if (!routing_ok(R)) return;
  uint32_t tm, tn;
  grouped_tile(xcd_tile(), ntm, ntn, &tm, &tn);
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
  for (int i = tid; i < S::BM; i += S::kThreads) lsa[i] = i < T.rows ? O.a_scale[T.row0 + i] : 0.0f;
  multiply<S, GLU>(A, B0, B1, (uint32_t)k, live, acc, lds0, lds1);
  if (!live) return;

  constexpr int kHalf = (S::kWaves + 1) / 2;
  static_assert(kHalf * RowStage<kWaveCols>::kBytes <= S::kStageBytes, "half of the waves share a stage");
  RowStage<kWaveCols> stage{reinterpret_cast<float*>((wave < kHalf ? lds0 : lds1) +
                                                     (wave % kHalf) * RowStage<kWaveCols>::kBytes)};
  constexpr int kPer = EPI == kOutF32 ? 4 : 8;              // columns of a lane's store
  constexpr int kLanes = kWaveCols / kPer, kRows = 64 / kLanes;  // lanes of a row, rows of a store
  const int c = kPer * (lane % kLanes), srow = lane / kLanes;
  const bool inside = wn * kWaveCols + c < (int)cols;
  float sb[S::TN];
#pragma unroll
  for (int in = 0; in < S::TN; ++in) {
    const int j = wn * kWaveCols + (in % BLK) * 32 + (lane & 31);
    sb[in] = j < (int)cols ? O.b_scale[line0 + (GLU && in >= BLK ? n : 0) + j] : 0.0f;
  }
#pragma unroll
  for (int im = 0; im < S::TM; ++im) {
    const int r0 = wm * (32 * S::TM) + 32 * im;
#pragma unroll
    for (int in = 0; in < BLK; ++in)
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const float sa = lsa[r0 + 8 * (v >> 2) + 4 * (lane >> 5) + (v & 3)];
        float y = ((float)acc[im][in][v] * sa) * sb[in];
        if constexpr (GLU) {
          const float u = ((float)acc[im][in + BLK][v] * sa) * sb[in + BLK];
          float dv;
          y = y * act_logistic<EPI == kGluSilu ? MOE_ACT_SILU : MOE_ACT_GELU>(y, &dv) * u;
        }
        stage.put(in, v, lane, y);
      }
    wave_sync();
#pragma unroll
    for (int r = 0; r < 32; r += kRows) {
      const f32x4 lo = stage.get4(r + srow, c);
      const int64_t at = (T.row0 + r0 + r + srow) * n + col0 + wn * kWaveCols + c;
      const bool write = inside && r0 + r + srow < T.rows;
      if constexpr (EPI == kOutF32) {
        if (write) *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(out) + at) = lo;
      } else {
        const f32x4 hi = stage.get4(r + srow, c + 4);
        if (write)
          *reinterpret_cast<u32x4*>(reinterpret_cast<uint16_t*>(out) + at) =
              u32x4{pack_bf16(lo[0], lo[1]), pack_bf16(lo[2], lo[3]), pack_bf16(hi[0], hi[1]), pack_bf16(hi[2], hi[3])};
      }
    }
    wave_sync();
  }
}

// ------------------------------------------------------------- host side

// Row tiles of BM rows that the routing can need at most.
template <int BM>
int64_t row_tiles(const Routing& R, bool dense, int64_t rows) {
  if (dense) return (rows + BM - 1) / BM;
  if (BM <= kTileRows) return rows / BM;
  if (R.d_offs) return std::min<int64_t>(rows / kTileRows, rows / BM + R.num_experts);
  int64_t t = 0;
  for (int e = 0; e < R.num_experts; ++e) t += (R.h_offs[e] - (e ? R.h_offs[e - 1] : 0) + BM - 1) / BM;
  return t;
}

template <class S, Epilogue EPI, int OCC>
int launch(const Operands& O, int64_t rows, int64_t n, int64_t k, const Routing& R, bool dense, void* out,
           hipStream_t st) {
  constexpr int kCols = is_glu(EPI) ? S::BN / 2 : S::BN;
  const int64_t ntm = row_tiles<S::BM>(R, dense, rows), ntn = (n + kCols - 1) / kCols;
  if (ntm * ntn > (1ll << 32) / S::kThreads - 1) return NVFP4G_EINVAL;
  hipLaunchKernelGGL((product_kernel<S, EPI, OCC>), dim3((uint32_t)(ntm * ntn)), dim3(S::kThreads), 0, st, O, n, k, R,
                     dense, (uint32_t)ntm, (uint32_t)ntn, out);
  return hip_status();
}

template <Epilogue EPI>
int product(const Operands& O, int64_t rows, int64_t n, int64_t k, const Routing& R, bool dense, void* out,
            hipStream_t st) {
  return launch<Shape<2, 2, 2, 4>, EPI, 1>(O, rows, n, k, R, dense, out, st);
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
  return out_type == MOE_F32 ? product<kOutF32>(O, rows, n, k, R, false, out, (hipStream_t)stream)
                             : product<kOutBf16>(O, rows, n, k, R, false, out, (hipStream_t)stream);
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
  return act == MOE_ACT_SILU ? product<kGluSilu>(O, rows, f, k, R, false, h, (hipStream_t)stream)
                             : product<kGluGelu>(O, rows, f, k, R, false, h, (hipStream_t)stream);
}

}  // namespace

extern "C" {

int64_t i8_linear_workspace(int64_t rows, int64_t k, int64_t n) { return 0; }

int i8_linear(const int8_t* a_q, const float* a_scale, int64_t rows, int64_t k, const int8_t* b_q,
              const float* b_scale, int64_t n, void* out, int32_t out_type, void* workspace, int64_t workspace_bytes,
              void* stream) {
  const Operands O{a_q, a_scale, b_q, b_scale};
  const int rc = check(O, rows, n, k, 1, out);
  if (rc) return rc;
  if (!valid_type(out_type)) return NVFP4G_EINVAL;
  if (rows == 0) return NVFP4G_OK;
  Routing R;
  R.num_experts = 1;
  R.m_capacity = (int32_t)rows;
  R.d_offs = nullptr;
  R.d_status = nullptr;
  return out_type == MOE_F32 ? product<kOutF32>(O, rows, n, k, R, true, out, (hipStream_t)stream)
                             : product<kOutBf16>(O, rows, n, k, R, true, out, (hipStream_t)stream);
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
