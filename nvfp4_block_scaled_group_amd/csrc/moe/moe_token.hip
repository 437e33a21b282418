// moe_token.hip -- the experts' projections for single tokens: bf16 tokens
// times NVFP4 weights, no packed groups, behind the C ABI of
// include/moe_ops.h.
//
// A work-group takes one expert (the first pair that chose it is its leader;
// the work-groups of later pairs with the same expert end at once) and a run
// of weight lines, and multiplies them by all pairs of that expert, 16 * MT at
// a time, so each chosen expert's weights are read once.  That read bounds it:
// 24 tokens, 6 of 64 experts, 2048 x 7168 in 97 us, 4.9 TB/s; a lone token, 8
// experts, 7168 x 2 x 2048 in 32 us, 4.1 TB/s (with the launch's start and end).
#include <algorithm>

#include "moe_token.hpp"

namespace {

using namespace moe;

// Whether no pair before `lead` has its expert (each wave finds out by
// itself).  mine: ids[lane], loaded beside e.
__device__ __forceinline__ bool leads(const int32_t* ids, int lead, int e, int lane, int mine) {
  bool earlier = lane < lead && mine == e;
  for (int p = lane + 64; p < lead; p += 64) earlier |= ids[p] == e;
  return !__any(earlier);
}

// Pairs of expert e, in pair order, into list[]; returns their number.  All
// threads of the work-group; the list is there after the last barrier inside.
// own: ids[thread], loaded beside e.  Done before the weights' first loads:
// behind them it took 1 to 3% longer.
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
    const uint8_t* __restrict__ b_data, const uint8_t* __restrict__ b_scale, const float* __restrict__ b_amax,
    int64_t n, int E, TokenPlan P, void* __restrict__ out) {
  __shared__ int32_t list[MOE_MAX_TOKEN_PAIRS];
  __shared__ int32_t wcnt[kTokenWaves];
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
  W.init(b_data, b_scale, line0, col0, ocols, k, lane);
  f32x4* red = reinterpret_cast<f32x4*>(xlds);
  // 2688 times the line factors of this lane's columns, loaded before anything waits
  float sg[kCols / 16], su[kCols / 16];
#pragma unroll
  for (int c = 0; c < kCols / 16; ++c) {
    const int64_t col = min<int64_t>(col0 + 16 * c, ocols - 16) + (lane & 15);
    sg[c] = b_amax[line0 + col];
    su[c] = MODE == kModeGlu ? b_amax[line0 + ocols + col] : 0.0f;
  }
  for (int first = 0; first < cnt; first += P.rows) {
    f32x4 acc[MT][NL];
    if (first) __syncthreads();  // the last pass is done with the staged rows and the joined sums
    const int rows = min(cnt - first, P.rows);
    token_multiply<MT, NL>(W, P, x, k, rows, wave, lane, xlds,
                           [&](int i) { return (int64_t)(pair_at(first + i) / per); }, acc, [] {});
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
        f32x4 a, b;
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
          if (MODE == kModeGlu) {
            float dv;
            const float g = a[v] * (sg[c] / 2688.0f), u = b[v] * (su[c] / 2688.0f);
            reinterpret_cast<uint16_t*>(out)[p * ocols + col] = to_bf16(g * act_logistic<ACT>(g, &dv) * u);
          } else {
            reinterpret_cast<float*>(out)[p * ocols + col] = a[v] * (sg[c] / 2688.0f);
          }
        }
      }
    }
  }
}

// ------------------------------------------------------------- host side

template <int MODE, int ACT, int MT>
void launch(const uint16_t* x, int64_t k, int per, const int32_t* ids, int pairs, const uint8_t* bd,
            const uint8_t* bs, const float* ba, int64_t n, int E, void* out, hipStream_t st) {
  constexpr int NL = 2, kCols = MODE == kModeGlu ? 16 : 32;
  const int64_t ocols = MODE == kModeGlu ? n / 2 : n, experts = std::min(pairs, E);
  auto tiles = [&](int ks) { return (ocols + kCols * (kTokenWaves / ks) - 1) / (kCols * (kTokenWaves / ks)); };
  // an expert has at most one pair of a token, or takes more passes
  const int rows = std::min((pairs + per - 1) / per, 16 * MT);
  // Waves that split the contraction: the fewest rounds of work-groups (two a
  // CU where LDS and registers hold them, with the experts that the pairs can
  // reach) times steps of a wave and a start that takes about three of them.
  // 5 tokens, 5600 x 1824, 8 of 8 experts: 32 us 4 ways, 52 not split, 45 with
  // 8; 24 pairs of 64 experts, 2048 x 7168: 97 us not split, 131 with 8.
  TokenPlan P{};
  int64_t best = INT64_MAX;
  for (int ks = 1; ks <= kTokenWaves; ks *= 2) {
    const TokenPlan q = token_plan(k, rows, ks, MT * NL, 0, experts * tiles(ks));
    if (q.ks != ks) break;
    const int64_t slots = (token_waves(MT) == 4 && q.lds <= kTokenLds ? 2 : 1) * kCus;
    const int64_t cost = (experts * tiles(ks) + slots - 1) / slots * ((int64_t)q.per * q.chunks + 3);
    if (cost < best) best = cost, P = q;
  }
  hipLaunchKernelGGL((token_kernel<MODE, ACT, MT, NL>), dim3((uint32_t)tiles(P.ks), (uint32_t)pairs),
                     dim3(kTokenThreads), P.lds, st, x, k, per, ids, pairs, bd, bs, ba, n, E, P, out);
}

template <int MODE, int ACT>
void dispatch(const uint16_t* x, int64_t k, int per, const int32_t* ids, int pairs, const uint8_t* bd,
              const uint8_t* bs, const float* ba, int64_t n, int E, void* out, hipStream_t st) {
  // Token tiles of a pass: the pairs an expert gets on average, with room for
  // an uneven choice, never more than the tokens there are.  64 tokens all to 8
  // experts (7168 x 2 x 2048): 105 us with 4 tiles, 134 with 2, 185 with 1 (the
  // weights are read again); 24 tokens, 6 of 64 experts: 96 with 1, 126 with 4.
  const int64_t experts = std::min(pairs, E), mean = (pairs + experts - 1) / experts, most = (pairs + per - 1) / per;
  const int64_t rows = std::min(mean * 3 / 2, most);
  if (rows <= 16) launch<MODE, ACT, 1>(x, k, per, ids, pairs, bd, bs, ba, n, E, out, st);
  else if (rows <= 32) launch<MODE, ACT, 2>(x, k, per, ids, pairs, bd, bs, ba, n, E, out, st);
  else launch<MODE, ACT, 4>(x, k, per, ids, pairs, bd, bs, ba, n, E, out, st);
}

int check_token(const uint16_t* x, int64_t pairs, int64_t k, const int32_t* ids, const uint8_t* bd, const uint8_t* bs,
                const float* ba, int64_t n, int32_t E, const void* out) {
  if (k <= 0 || k % 32 != 0 || k > kMaxK || n <= 0 || n % 16 != 0 || n > (1 << 20)) return NVFP4G_EINVAL;
  if (pairs < 0 || pairs > MOE_MAX_TOKEN_PAIRS || E < 1 || E > MOE_MAX_EXPERTS) return NVFP4G_EINVAL;
  if (pairs && (!x || !ids || !out || !bd || !bs || !ba)) return NVFP4G_EINVAL;
  if (!aligned(x, 16) || !aligned(bd, 16) || !aligned(bs, 4) || !aligned(ba, 4) || !aligned(ids, 4) ||
      !aligned(out, 16))
    return NVFP4G_EALIGN;
  return NVFP4G_OK;
}

}  // namespace

extern "C" {

int moe_token_glu(const uint16_t* x, int64_t tokens, int64_t k, int32_t topk, const int32_t* ids,
                  const uint8_t* b_data, const uint8_t* b_scale, const float* b_amax, int64_t f, int32_t num_experts,
                  int32_t act, uint16_t* h, void* stream) {
  if (topk < 1 || topk > MOE_MAX_TOPK || tokens < 0 || tokens > MOE_MAX_TOKEN_PAIRS) return NVFP4G_EINVAL;
  if (f <= 0 || f % 16 != 0 || f > (1 << 19) || (act != MOE_ACT_SILU && act != MOE_ACT_GELU)) return NVFP4G_EINVAL;
  const int rc = check_token(x, tokens * topk, k, ids, b_data, b_scale, b_amax, 2 * f, num_experts, h);
  if (rc) return rc;
  if (tokens == 0) return NVFP4G_OK;
  const int pairs = (int)tokens * topk;
  if (act == MOE_ACT_SILU)
    dispatch<kModeGlu, MOE_ACT_SILU>(x, k, topk, ids, pairs, b_data, b_scale, b_amax, 2 * f, num_experts, h,
                                     (hipStream_t)stream);
  else
    dispatch<kModeGlu, MOE_ACT_GELU>(x, k, topk, ids, pairs, b_data, b_scale, b_amax, 2 * f, num_experts, h,
                                     (hipStream_t)stream);
  return hip_status();
}

int moe_token_linear(const uint16_t* x, int64_t pairs, int64_t k, const int32_t* ids, const uint8_t* b_data,
                     const uint8_t* b_scale, const float* b_amax, int64_t n, int32_t num_experts, float* out,
                     void* stream) {
  const int rc = check_token(x, pairs, k, ids, b_data, b_scale, b_amax, n, num_experts, out);
  if (rc) return rc;
  if (pairs == 0) return NVFP4G_OK;
  dispatch<kModeLinear, 0>(x, k, 1, ids, (int)pairs, b_data, b_scale, b_amax, n, num_experts, out,
                           (hipStream_t)stream);
  return hip_status();
}

}  // extern "C"
