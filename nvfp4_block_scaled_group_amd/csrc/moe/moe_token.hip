// moe_token.hip -- the experts' projections for single tokens: bf16 tokens
// times NVFP4 weights, no packed groups, behind the C ABI of
// include/moe_ops.h.  Also the adapter projection of a few tokens.
//
// What bounds it is reading the chosen experts' weights once (0.5625 byte an
// element).  A work-group takes one expert (the first pair that chose it is
// its leader; the work-groups of later pairs with the same expert end at once)
// and a run of weight lines, and multiplies them by all pairs of that expert,
// 16 * MT at a time.  MFMA 16x16x32: rows are tokens, columns are lines, so a
// tile costs the same for 1 token as for 16, and the matrix units are far from
// the limit.  Lane (n = lane % 16, g = lane / 16) loads 16 bytes of line n's
// 64-byte step (32 codes, two blocks) and its two scale bytes, decodes them in
// registers, and the same lane mapping picks the matching 32 values of x.
// With few work-groups the contraction is split over the KS waves of a
// work-group and joined in LDS in a fixed order.
#include "moe_token.hpp"

namespace {

using namespace moe;

// Pairs of the leader's expert, in pair order, into list[]; returns their
// number, or 0 if an earlier pair leads.  All threads of the work-group.
__device__ int gather_pairs(const int32_t* ids, int pairs, int lead, int e, int32_t* list, int32_t* wcnt) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int at = 0;
  bool earlier = false;
  for (int p0 = 0; p0 < pairs; p0 += kThreads) {
    const int p = p0 + tid;
    const bool mine = p < pairs && ids[p] == e;
    earlier |= mine && p < lead;
    const uint64_t b = __ballot(mine);
    if (lane == 0) wcnt[wave] = __popcll(b);
    if (__syncthreads_or(earlier)) return 0;
    int before = at;
    for (int w = 0; w < kThreads / 64; ++w) {
      if (w < wave) before += wcnt[w];
      at += wcnt[w];
    }
    if (mine) list[before + __popcll(b & ((1ull << lane) - 1))] = p;
    __syncthreads();
  }
  return at;
}

// x rows: pair / per (per = topk: the token's row is shared by its choices).
template <int MODE, int ACT, int MT, int NL, int KS>
__global__ __launch_bounds__(kThreads, MT * NL >= 8 ? 2 : MT * NL >= 4 ? 3 : 4) void token_kernel(
    const uint16_t* __restrict__ x, int64_t k, int per, const int32_t* __restrict__ ids, int pairs,
    const uint8_t* __restrict__ b_data, const uint8_t* __restrict__ b_scale, const float* __restrict__ b_amax,
    int64_t n, int E, void* __restrict__ out) {
  __shared__ int32_t list[MOE_MAX_TOKEN_PAIRS];
  __shared__ int32_t wcnt[kThreads / 64];
  __shared__ f32x4 red[KS > 1 ? KS * MT * NL * 64 : 1];
  constexpr int kCols = MODE == kModeGlu ? NL / 2 * 16 : NL * 16;   // output columns of a wave
  const int lane = threadIdx.x & 63, wave = uni((int32_t)(threadIdx.x >> 6));
  const int lead = uni((int32_t)blockIdx.y);
  const int e = uni(ids[lead]);
  const int64_t ocols = MODE == kModeGlu ? n / 2 : n;
  const int64_t col0 = ((int64_t)blockIdx.x * (4 / KS) + wave / KS) * kCols;
  if ((uint32_t)e >= (uint32_t)E) {  // no expert: a row of zeros
    const int64_t c0 = (int64_t)blockIdx.x * (4 / KS) * kCols, c1 = min<int64_t>(c0 + 4 / KS * kCols, ocols);
    for (int64_t c = c0 + threadIdx.x; c < c1; c += kThreads) {
      if (MODE == kModeGlu) reinterpret_cast<uint16_t*>(out)[lead * ocols + c] = 0;
      else reinterpret_cast<float*>(out)[lead * ocols + c] = 0.0f;
    }
    return;
  }
  const int cnt = gather_pairs(ids, pairs, lead, e, list, wcnt);
  if (cnt == 0) return;
  const int64_t line0 = (int64_t)e * n;
  TileLines<MODE, NL> W;
  W.init(b_data, b_scale, line0, col0, ocols, k, lane);
  for (int first = 0; first < cnt; first += 16 * MT) {
    const uint16_t* xr[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const int i = first + mt * 16 + (lane & 15);
      xr[mt] = x + (int64_t)(list[i < cnt ? i : first] / per) * k;
    }
    f32x4 acc[MT][NL];
    token_multiply<MT, NL, KS>(W, xr, k, wave % KS, lane, acc);
    if (KS > 1) join_waves<MT, NL, KS>(acc, red, wave, lane);
    // each wave finishes its share: all of its tiles, or with split waves the
    // tiles whose number is the wave's own
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      if (first + mt * 16 >= cnt) continue;
#pragma unroll
      for (int c = 0; c < kCols / 16; ++c) {
        if (KS > 1 && (mt * (kCols / 16) + c) % KS != wave) continue;
        const int64_t col = col0 + 16 * c + (lane & 15);
        if (col0 + 16 * c >= ocols) continue;
        f32x4 a, b;
        if (MODE == kModeGlu) {
          a = KS > 1 ? joined<MT, NL, KS>(red, mt, 2 * c, lane) : acc[mt][2 * c];
          b = KS > 1 ? joined<MT, NL, KS>(red, mt, 2 * c + 1, lane) : acc[mt][2 * c + 1];
        } else {
          a = KS > 1 ? joined<MT, NL, KS>(red, mt, c, lane) : acc[mt][c];
        }
        const float s = b_amax[line0 + col] / 2688.0f;
        const float su = MODE == kModeGlu ? b_amax[line0 + ocols + col] / 2688.0f : 0.0f;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int i = first + mt * 16 + 4 * (lane >> 4) + v;
          if (i >= cnt) continue;
          const int64_t p = list[i];
          if (MODE == kModeGlu) {
            float dv;
            const float g = a[v] * s, u = b[v] * su;
            reinterpret_cast<uint16_t*>(out)[p * ocols + col] = to_bf16(g * act_logistic<ACT>(g, &dv) * u);
          } else {
            reinterpret_cast<float*>(out)[p * ocols + col] = a[v] * s;
          }
        }
      }
    }
    if (KS > 1) __syncthreads();  // red is written again by the next pass
  }
}

// ------------------------------------------------------------- host side

template <int MODE, int ACT, int MT, int NL, int KS>
void launch(const uint16_t* x, int64_t k, int per, const int32_t* ids, int pairs, const uint8_t* bd,
            const uint8_t* bs, const float* ba, int64_t n, int E, void* out, hipStream_t st) {
  constexpr int kCols = (MODE == kModeGlu ? NL / 2 * 16 : NL * 16) * (4 / KS);
  const int64_t ocols = MODE == kModeGlu ? n / 2 : n;
  const dim3 grid((uint32_t)((ocols + kCols - 1) / kCols), (uint32_t)pairs);
  hipLaunchKernelGGL((token_kernel<MODE, ACT, MT, NL, KS>), grid, dim3(kThreads), 0, st, x, k, per, ids, pairs, bd, bs,
                     ba, n, E, out);
}

template <int MODE, int ACT>
void dispatch(const uint16_t* x, int64_t k, int per, const int32_t* ids, int pairs, const uint8_t* bd,
              const uint8_t* bs, const float* ba, int64_t n, int E, void* out, hipStream_t st) {
  // Work-groups there will be at least: the experts that pairs can reach.
  const int64_t experts = pairs < E ? pairs : E;
  // Token tiles of a pass: the pairs an expert gets on average, with room for
  // an uneven choice, never more than the tokens there are.
  const int64_t mean = (pairs + experts - 1) / experts, most = (pairs + per - 1) / per;
  const int64_t tiles = ((mean * 3 / 2 < most ? mean * 3 / 2 : most) + 15) / 16;
  const int64_t wide_waves = experts * ((n + 63) / 64);
  if (tiles <= 1) {
    if (wide_waves >= 4096) launch<MODE, ACT, 1, 4, 1>(x, k, per, ids, pairs, bd, bs, ba, n, E, out, st);
    else launch<MODE, ACT, 1, 2, 4>(x, k, per, ids, pairs, bd, bs, ba, n, E, out, st);
  } else if (tiles == 2) {
    launch<MODE, ACT, 2, 2, 4>(x, k, per, ids, pairs, bd, bs, ba, n, E, out, st);
  } else {
    launch<MODE, ACT, 4, 2, 4>(x, k, per, ids, pairs, bd, bs, ba, n, E, out, st);
  }
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
