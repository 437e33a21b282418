// i8_token.hip -- products in 8-bit integers for single tokens: the experts'
// projections, and a projection of few rows, behind the C ABI of
// include/i8_group.h.
//
// A work-group takes one expert (the first pair that chose it is its leader;
// the work-groups of later pairs with the same expert end at once) and a run
// of weight lines, and multiplies them by all pairs of that expert, 16 * MT at
// a time, so each chosen expert's weights are read once.
#include "i8_token.hpp"

namespace {

using namespace i8;

// Whether no pair before `lead` has its expert (each wave finds out by
// itself).  mine: ids[lane], loaded beside e.
__device__ __forceinline__ bool leads(const int32_t* ids, int lead, int e, int lane, int mine) {
  bool earlier = lane < lead && mine == e;
  for (int p = lane + 64; p < lead; p += 64) earlier |= ids[p] == e;
  return !__any(earlier);
}

// Pairs of expert e, in pair order, into list[]; returns their number.  All
// threads of the work-group; the list is there after the last barrier inside.
__device__ __forceinline__ int gather_pairs(const int32_t* ids, int pairs, int e, int own, int32_t* list, int32_t* wcnt) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int at = 0;
  for (int p0 = 0; p0 < pairs; p0 += kTokenThreads) {
    const int p = p0 + tid;
    const bool mine = p < pairs && (p0 ? ids[p] : own) == e;
    const uint64_t b = __ballot(mine);
    if (lane == 0) wcnt[wave] = __popcll(b);
    __syncthreads();
    int before = at;
    for (int w = 0; w < kTokenWaves; ++w) {
      if (w < wave) before += wcnt[w];
      at += wcnt[w];
    }
    if (mine) list[before + __popcll(b & ((1ull << lane) - 1))] = p;
    __syncthreads();
  }
  return at;
}

// x rows: pair / per (per = topk: the token's row is shared by its choices).
template <int MODE, int ACT, int MT, int NL>
__global__ __launch_bounds__(kTokenThreads, token_waves(MT)) void token_kernel(
    const uint16_t* __restrict__ x, int64_t k, int per, const int32_t* __restrict__ ids, int pairs,
    const int8_t* __restrict__ b_q, const float* __restrict__ b_scale, int64_t n, int E, TokenPlan P,
    void* __restrict__ out) {
  __shared__ int32_t list[MOE_MAX_TOKEN_PAIRS];
  __shared__ int32_t wcnt[kTokenWaves];
  __shared__ RowCast lcast[16 * MT];
  __shared__ uint32_t lmax[16 * MT];
  extern __shared__ __attribute__((aligned(16))) uint8_t xlds[];
  constexpr int kCols = MODE == kModeGlu ? NL / 2 * 16 : NL * 16;   // output columns of a wave
  const int lane = threadIdx.x & 63, wave = uni((int32_t)(threadIdx.x >> 6));
  const int lead = uni((int32_t)blockIdx.y);
  const int mine = ids[min(lane, pairs - 1)], own = ids[min((int)threadIdx.x, pairs - 1)], e = uni(ids[lead]);
  const int64_t ocols = MODE == kModeGlu ? n / 2 : n;
  const int groups = kTokenWaves / P.ks, group = wave / P.ks, part = wave % P.ks;
  const int64_t first_col = (int64_t)blockIdx.x * groups * kCols, col0 = first_col + group * kCols;
  if ((uint32_t)e >= (uint32_t)E) {  // no expert: a row of zeros
    const int64_t c1 = min<int64_t>(first_col + groups * kCols, ocols);
    for (int64_t c = first_col + threadIdx.x; c < c1; c += kTokenThreads) {
      if (MODE == kModeGlu) reinterpret_cast<uint16_t*>(out)[lead * ocols + c] = 0;
      else reinterpret_cast<float*>(out)[lead * ocols + c] = 0.0f;
    }
    return;
  }
  // The choices of a lone token are taken one by one (a token that names an
  // expert twice reads its weights twice), with nothing to gather.
  const bool lone = pairs <= per;
  if (!lone && !leads(ids, lead, e, lane, mine)) return;
  const int cnt = lone ? 1 : gather_pairs(ids, pairs, e, own, list, wcnt);
  auto pair_at = [&](int i) { return lone ? lead : list[i]; };
  const int64_t line0 = (int64_t)e * n;
  TileLines<MODE, NL> W;
  W.init(b_q, line0, col0, ocols, k, lane);
  i32x4* red = reinterpret_cast<i32x4*>(xlds);
  float sg[kCols / 16], su[kCols / 16];  // scales of this lane's columns, loaded before anything waits
#pragma unroll
  for (int c = 0; c < kCols / 16; ++c) {
    const int64_t col = min<int64_t>(col0 + 16 * c, ocols - 16) + (lane & 15);
    sg[c] = b_scale[line0 + col];
    su[c] = MODE == kModeGlu ? b_scale[line0 + ocols + col] : 0.0f;
  }
  const CastRows X{x, lcast, lmax};
  for (int first = 0; first < cnt; first += P.rows) {
    i32x4 acc[MT][NL];
    if (first) __syncthreads();  // the last pass is done with the staged rows and the joined sums
    const int rows = min(cnt - first, P.rows);
    auto row_of = [&](int i) { return (int64_t)(pair_at(first + i) / per); };
    token_multiply<MT, NL>(W, P, X, k, rows, wave, lane, xlds, row_of, acc);
    if (P.ks > 1) join_waves<MT, NL>(acc, red, wave, lane);
    // each wave finishes its share: with split waves the tiles whose number
    // is its part's
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      if (mt * 16 >= rows) continue;
#pragma unroll
      for (int c = 0; c < kCols / 16; ++c) {
        if ((mt * (kCols / 16) + c) % P.ks != part || col0 + 16 * c >= ocols) continue;
        const int64_t col = col0 + 16 * c + (lane & 15);
        i32x4 a, b;
        if (MODE == kModeGlu) {
          a = P.ks > 1 ? joined<MT, NL>(red, group, P.ks, mt, 2 * c, lane) : acc[mt][2 * c];
          b = P.ks > 1 ? joined<MT, NL>(red, group, P.ks, mt, 2 * c + 1, lane) : acc[mt][2 * c + 1];
        } else {
          a = P.ks > 1 ? joined<MT, NL>(red, group, P.ks, mt, c, lane) : acc[mt][c];
        }
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int i = mt * 16 + 4 * (lane >> 4) + v;
          if (i >= rows) continue;
          const int64_t p = pair_at(first + i);
          const float sx = lcast[i].scale, g = ((float)a[v] * sx) * sg[c];
          if (MODE == kModeGlu) {
            float dv;
            const float u = ((float)b[v] * sx) * su[c];
            reinterpret_cast<uint16_t*>(out)[p * ocols + col] = to_bf16(g * act_logistic<ACT>(g, &dv) * u);
          } else {
            reinterpret_cast<float*>(out)[p * ocols + col] = g;
          }
        }
      }
    }
  }
}

// A few rows of codes times the lines of one projection: no experts to find,
// and the rows are copied as they are.
template <int MT, int NL, bool F32OUT>
__global__ __launch_bounds__(kTokenThreads, token_waves(MT)) void few_rows_kernel(
    const int8_t* __restrict__ a_q, const float* __restrict__ a_scale, int rows, int64_t k,
    const int8_t* __restrict__ b_q, const float* __restrict__ b_scale, int64_t n, TokenPlan P, void* __restrict__ out) {
  extern __shared__ __attribute__((aligned(16))) uint8_t xlds[];
  constexpr int kCols = NL * 16;
  const int lane = threadIdx.x & 63, wave = uni((int32_t)(threadIdx.x >> 6));
  const int groups = kTokenWaves / P.ks, group = wave / P.ks, part = wave % P.ks;
  const int64_t col0 = ((int64_t)blockIdx.x * groups + group) * kCols;
  TileLines<kModeLinear, NL> W;
  W.init(b_q, 0, col0, n, k, lane);
  float sb[NL];
#pragma unroll
  for (int t = 0; t < NL; ++t) sb[t] = b_scale[min<int64_t>(col0 + 16 * t, n - 16) + (lane & 15)];
  i32x4* red = reinterpret_cast<i32x4*>(xlds);
  const CodeRows X{a_q};
  for (int first = 0; first < rows; first += P.rows) {
    i32x4 acc[MT][NL];
    if (first) __syncthreads();  // the last pass is done with the staged rows and the joined sums
    const int cnt = min(rows - first, P.rows);
    token_multiply<MT, NL>(W, P, X, k, cnt, wave, lane, xlds, [&](int i) { return (int64_t)(first + i); }, acc);
    if (P.ks > 1) join_waves<MT, NL>(acc, red, wave, lane);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      if (mt * 16 >= cnt) continue;
#pragma unroll
      for (int t = 0; t < NL; ++t) {
        if ((mt * NL + t) % P.ks != part || col0 + 16 * t >= n) continue;
        const i32x4 s = P.ks > 1 ? joined<MT, NL>(red, group, P.ks, mt, t, lane) : acc[mt][t];
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int i = mt * 16 + 4 * (lane >> 4) + v;
          if (i >= cnt) continue;
          const float y = ((float)s[v] * a_scale[first + i]) * sb[t];
          const int64_t at = (first + i) * n + col0 + 16 * t + (lane & 15);
          if (F32OUT) reinterpret_cast<float*>(out)[at] = y;
          else reinterpret_cast<uint16_t*>(out)[at] = to_bf16(y);
        }
      }
    }
  }
}

// ------------------------------------------------------------- host side

// Waves that split the contraction: the fewest rounds of work-groups (two a CU
// where LDS and registers hold them; `experts` times the column tiles) times
// steps of a wave and a start that takes about three of them.
template <class Tiles>
TokenPlan best_plan(int64_t k, int rows, int mt, int nl, int64_t experts, Tiles tiles) {
  TokenPlan P{};
  int64_t best = INT64_MAX;
  for (int ks = 1; ks <= kTokenWaves; ks *= 2) {
    const TokenPlan q = token_plan(k, rows, ks, mt * nl, experts * tiles(ks));
    if (q.ks != ks) break;
    const int64_t slots = (token_waves(mt) == 4 && q.lds <= kTokenLds ? 2 : 1) * kCus;
    const int64_t cost = (experts * tiles(ks) + slots - 1) / slots * ((int64_t)q.per * q.chunks + 3);
    if (cost < best) best = cost, P = q;
  }
  return P;
}

// NL: one tile of lines a wave in place of two while a work-group has a CU to itself
// (the gated block needs a gate and an up tile): the lines' way into one CU takes half as
// long (1 token, 2048 x 7168: 6.6 us and 8.7; 8 of 64 experts, 2048 x 2048: 9.4 and 9.9;
// 32 tokens of 2 experts: 10.7 and 13.1).
template <int MODE, int ACT, int MT, int NL = 2>
void launch(const uint16_t* x, int64_t k, int per, const int32_t* ids, int pairs, const int8_t* bq, const float* bs,
            int64_t n, int E, void* out, hipStream_t st) {
  constexpr int kCols = MODE == kModeGlu ? 8 * NL : 16 * NL;
  const int64_t ocols = MODE == kModeGlu ? n / 2 : n, experts = std::min(pairs, E);
  auto tiles = [&](int ks) { return (ocols + kCols * (kTokenWaves / ks) - 1) / (kCols * (kTokenWaves / ks)); };
  // an expert has at most one pair of a token, or takes more passes
  const int rows = std::min((pairs + per - 1) / per, 16 * MT);
  const TokenPlan P = best_plan(k, rows, MT, NL, experts, tiles);
  if constexpr (MODE == kModeLinear && NL > 1)
    if (experts * tiles(P.ks) <= kCus) return launch<MODE, ACT, MT, 1>(x, k, per, ids, pairs, bq, bs, n, E, out, st);
  hipLaunchKernelGGL((token_kernel<MODE, ACT, MT, NL>), dim3((uint32_t)tiles(P.ks), (uint32_t)pairs),
                     dim3(kTokenThreads), P.lds, st, x, k, per, ids, pairs, bq, bs, n, E, P, out);
}

template <int MODE, int ACT>
void dispatch(const uint16_t* x, int64_t k, int per, const int32_t* ids, int pairs, const int8_t* bq, const float* bs,
              int64_t n, int E, void* out, hipStream_t st) {
  // Token tiles of a pass: the pairs an expert gets on average, with room for
  // an uneven choice, never more than the tokens there are.
  const int64_t experts = std::min(pairs, E), mean = (pairs + experts - 1) / experts, most = (pairs + per - 1) / per;
  const int64_t rows = std::min(mean * 3 / 2, most);
  if (rows <= 16) launch<MODE, ACT, 1>(x, k, per, ids, pairs, bq, bs, n, E, out, st);
  else if (rows <= 32) launch<MODE, ACT, 2>(x, k, per, ids, pairs, bq, bs, n, E, out, st);
  else launch<MODE, ACT, 4>(x, k, per, ids, pairs, bq, bs, n, E, out, st);
}

int check_token(const uint16_t* x, int64_t pairs, int64_t k, const int32_t* ids, const int8_t* bq, const float* bs,
                int64_t n, int32_t E, const void* out) {
  if (!valid_k(k) || !valid_n(n)) return NVFP4G_EINVAL;
  if (pairs < 0 || pairs > MOE_MAX_TOKEN_PAIRS || E < 1 || E > MOE_MAX_EXPERTS) return NVFP4G_EINVAL;
  if (pairs && (!x || !ids || !out || !bq || !bs)) return NVFP4G_EINVAL;
  if (!aligned(x, 16) || !aligned(bq, 16) || !aligned(bs, 4) || !aligned(ids, 4) || !aligned(out, 16))
    return NVFP4G_EALIGN;
  return NVFP4G_OK;
}

// NL as above (8 rows of 2048 x 7168: 6.8 us and 8.7, of 7168 x 2048: 9.2 and 12.8, of
// 8192 x 8192: 17.0 and 18.4; 16 rows of 7168 x 7168: 16.7 and 16.1).
template <int MT, int NL>
int launch_few(const int8_t* a_q, const float* a_scale, int64_t rows, int64_t k, const int8_t* b_q,
               const float* b_scale, int64_t n, void* out, int32_t out_type, hipStream_t st) {
  constexpr int kCols = 16 * NL;
  auto tiles = [&](int ks) { return (n + kCols * (kTokenWaves / ks) - 1) / (kCols * (kTokenWaves / ks)); };
  const TokenPlan P = best_plan(k, (int)std::min<int64_t>(rows, 16 * MT), MT, NL, 1, tiles);
  if (NL > 1 && tiles(P.ks) <= kCus)
    return launch_few<MT, 1>(a_q, a_scale, rows, k, b_q, b_scale, n, out, out_type, st);
  auto go = [&](auto* kernel) {
    hipLaunchKernelGGL(kernel, dim3((uint32_t)tiles(P.ks)), dim3(kTokenThreads), P.lds, st, a_q, a_scale, (int)rows, k,
                       b_q, b_scale, n, P, out);
  };
  if (out_type == MOE_F32) go(few_rows_kernel<MT, NL, true>);
  else go(few_rows_kernel<MT, NL, false>);
  return hip_status();
}

}  // namespace

namespace i8 {

int few_rows(const int8_t* a_q, const float* a_scale, int64_t rows, int64_t k, const int8_t* b_q, const float* b_scale,
             int64_t n, void* out, int32_t out_type, hipStream_t st) {
  if (rows <= 16) return launch_few<1, 2>(a_q, a_scale, rows, k, b_q, b_scale, n, out, out_type, st);
  if (rows <= 32) return launch_few<2, 2>(a_q, a_scale, rows, k, b_q, b_scale, n, out, out_type, st);
  return launch_few<4, 2>(a_q, a_scale, rows, k, b_q, b_scale, n, out, out_type, st);
}

}  // namespace i8

extern "C" {

int i8_token_glu(const uint16_t* x, int64_t tokens, int64_t k, int32_t topk, const int32_t* ids, const int8_t* b_q,
                 const float* b_scale, int64_t f, int32_t num_experts, int32_t act, uint16_t* h, void* stream) {
  if (topk < 1 || topk > MOE_MAX_TOPK || tokens < 0 || tokens > MOE_MAX_TOKEN_PAIRS) return NVFP4G_EINVAL;
  if (f <= 0 || f % 16 != 0 || f > (1 << 19) || (act != MOE_ACT_SILU && act != MOE_ACT_GELU)) return NVFP4G_EINVAL;
  const int rc = check_token(x, tokens * topk, k, ids, b_q, b_scale, 2 * f, num_experts, h);
  if (rc) return rc;
  if (tokens == 0) return NVFP4G_OK;
  const int pairs = (int)tokens * topk;
  if (act == MOE_ACT_SILU)
    dispatch<kModeGlu, MOE_ACT_SILU>(x, k, topk, ids, pairs, b_q, b_scale, 2 * f, num_experts, h, (hipStream_t)stream);
  else
    dispatch<kModeGlu, MOE_ACT_GELU>(x, k, topk, ids, pairs, b_q, b_scale, 2 * f, num_experts, h, (hipStream_t)stream);
  return hip_status();
}

int i8_token_linear(const uint16_t* x, int64_t pairs, int64_t k, const int32_t* ids, const int8_t* b_q,
                    const float* b_scale, int64_t n, int32_t num_experts, float* out, void* stream) {
  const int rc = check_token(x, pairs, k, ids, b_q, b_scale, n, num_experts, out);
  if (rc) return rc;
  if (pairs == 0) return NVFP4G_OK;
  dispatch<kModeLinear, 0>(x, k, 1, ids, (int)pairs, b_q, b_scale, n, num_experts, out, (hipStream_t)stream);
  return hip_status();
}

}  // extern "C"
