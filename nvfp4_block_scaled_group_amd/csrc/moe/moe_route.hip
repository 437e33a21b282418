// moe_route.hip -- selection of experts with weights, its gradient, and the
// plan of the packed 128-row groups, behind the C ABI of include/moe_ops.h.
//
// Selection.  A token's choice is the topk largest keys  l + bias, ties to the
// lower index; its weights are softmax or sigmoid scores of the logits.  It is
// bound by instructions, not by the read of the logits, so the lanes of a wave
// share several tokens: LANES lanes hold VPL consecutive experts each.  A key
// and its index become one 64-bit pattern, unique and ordered, that is also an
// ordered finite double, so that one maximum or minimum instruction compares
// both.  Each lane sorts its patterns once; then topk rounds take the maximum
// of the lanes' heads (log2 LANES exchanges) and the lane that had it drops its
// head.  32768 x 256, 8 chosen, sigmoid: 16 us (2.3 TB/s); 28 us with one token a
// wave and the keys searched every round.
//
// Plan.  A stable counting sort of the pairs by expert without atomics that
// decide an order: a wave ranks 64 pairs at a time by matching expert
// numbers with one ballot a bit, on top of its running counts in LDS.
#include "moe_common.hpp"

namespace {

using namespace moe;

constexpr float kNegInf = -__builtin_huge_valf();

// Order-preserving integer of a key; 0 for a masked one (-inf), -0 as +0.
__device__ __forceinline__ uint32_t key_bits(float k) {
  if (!(k > kNegInf)) return 0;
  const uint32_t b = __float_as_uint(k + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// A logit as the operator reads it: NaN and -inf masked, +inf as FLT_MAX.
__device__ __forceinline__ float clean(float l) { return l > kNegInf ? fminf(l, FLT_MAX) : kNegInf; }

template <class T>
__device__ __forceinline__ float logit_at(const T* p, int64_t i);
template <>
__device__ __forceinline__ float logit_at<float>(const float* p, int64_t i) { return p[i]; }
template <>
__device__ __forceinline__ float logit_at<uint16_t>(const uint16_t* p, int64_t i) {
  return __uint_as_float((uint32_t)p[i] << 16);
}

// VPL consecutive values of a row of E (experts lane*VPL ..) as fp32, whatever
// is there past E.  With `wide` (E a multiple of VPL and the row aligned to the
// lane's piece) as vector loads.  A lane or an element past E reads one inside
// the row: no branch holds the other loads up.
template <class T, int VPL>
__device__ __forceinline__ void load_row(const T* row, int E, int lane, bool wide, float (&v)[VPL]) {
  const int e0 = lane * VPL;
  constexpr int kPer = 16 / (int)sizeof(T) < VPL ? 16 / (int)sizeof(T) : VPL;  // elements of one load
  if (wide) {
    const T* p = row + (e0 < E ? e0 : 0);
#pragma unroll
    for (int i = 0; i < VPL; i += kPer) {
      typedef T vec_t __attribute__((ext_vector_type(kPer)));
      const vec_t q = *reinterpret_cast<const vec_t*>(p + i);
#pragma unroll
      for (int c = 0; c < kPer; ++c) {
        const T x = q[c];
        v[i + c] = logit_at<T>(&x, 0);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) v[i] = logit_at<T>(row, min(e0 + i, E - 1));
  }
}
template <class T, int VPL>
__device__ __forceinline__ void load_logits(const T* row, int E, int lane, bool wide, float (&l)[VPL]) {
  load_row<T, VPL>(row, E, lane, wide, l);
#pragma unroll
  for (int i = 0; i < VPL; ++i) l[i] = lane * VPL + i < E ? clean(l[i]) : kNegInf;
}

// Value of lane ^ (the step's distance) inside a group of lanes: 1, 2, then
// the mirror of 8 and the rotation of 16, which serve reductions as well.
template <int STEP>
__device__ __forceinline__ uint32_t exchange(uint32_t v) {
  if constexpr (STEP == 0) return dpp_x1(v);
  else if constexpr (STEP == 1) return dpp_x2(v);
  else if constexpr (STEP == 2) return dpp_hmirror(v);
  else if constexpr (STEP == 3) return swap8(v);
  else {
    // the swap gives own and other half; which is which depends on the lane
    const auto r = STEP == 4 ? __builtin_amdgcn_permlane16_swap(v, v, false, false)
                             : __builtin_amdgcn_permlane32_swap(v, v, false, false);
    const bool upper = (threadIdx.x >> STEP) & 1;
    return upper ? r[0] : r[1];
  }
}
template <int LANES, int STEP = 0>
__device__ __forceinline__ double group_max(double v) {
  if constexpr ((1 << STEP) >= LANES) {
    return v;
  } else {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint64_t o = (uint64_t)exchange<STEP>((uint32_t)(b >> 32)) << 32 | exchange<STEP>((uint32_t)b);
    return group_max<LANES, STEP + 1>(__builtin_fmax(v, __builtin_bit_cast(double, o)));
  }
}
template <int LANES, int STEP = 0>
__device__ __forceinline__ float group_fmax(float v) {
  if constexpr ((1 << STEP) >= LANES) return v;
  else return group_fmax<LANES, STEP + 1>(fmaxf(v, __uint_as_float(exchange<STEP>(__float_as_uint(v)))));
}
template <int LANES, int STEP = 0>
__device__ __forceinline__ float group_sum(float v) {
  if constexpr ((1 << STEP) >= LANES) return v;
  else return group_sum<LANES, STEP + 1>(v + __uint_as_float(exchange<STEP>(__float_as_uint(v))));
}

// By value: a conditional on two array elements selects an address, and the
// array leaves its registers.
__device__ __forceinline__ double pick(bool c, double a, double b) { return c ? a : b; }

// Key bits above the complemented index: the two top bits are 0, so the
// pattern is a finite double and its order is that of the pair.
__device__ __forceinline__ double key_pattern(uint32_t key, uint32_t index) {
  return __builtin_bit_cast(double, (uint64_t)key << 30 | (uint64_t)(MOE_MAX_EXPERTS - 1 - index));
}

// Odd-even merge sort, descending.
template <int N>
__device__ __forceinline__ void sort_desc(double (&v)[N]) {
#pragma unroll
  for (int p = 1; p < N; p *= 2)
#pragma unroll
    for (int q = p; q >= 1; q /= 2)
#pragma unroll
      for (int j = q % p; j + q < N; j += 2 * q)
#pragma unroll
        for (int i = 0; i < q; ++i)
          if (i + j + q < N && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
            const double a = v[i + j], b = v[i + j + q];
            v[i + j] = __builtin_fmax(a, b);
            v[i + j + q] = __builtin_fmin(a, b);
          }
}

// Scores of the chosen logits, slot j of a token in lane j of its group (z =
// -inf elsewhere and for no choice): the unscaled weight.  top and sum are the
// softmax's maximum and sum over all unmasked experts (used without normalize).
template <int LANES>
__device__ __forceinline__ float group_score(float z, int score, int normalize, float top, float sum) {
  const bool on = z > kNegInf;
  float s;
  if (score == MOE_SCORE_SIGMOID) {
    s = on ? 1.0f / (1.0f + expf(-z)) : 0.0f;
  } else if (normalize) {
    const float m = group_fmax<LANES>(z);
    s = on ? expf(z - m) : 0.0f;
  } else {
    s = on ? expf(z - top) / sum : 0.0f;
  }
  if (normalize) {
    const float tot = group_sum<LANES>(s);
    s = tot > 0.0f ? s / tot : 0.0f;
  }
  return s;
}

// KMAX: the sorted patterns a lane keeps, topk at least.
template <class T, int LANES, int VPL, int KMAX>
__global__ __launch_bounds__(kThreads) void route_kernel(const T* __restrict__ logits, int64_t tokens, int E, int topk,
                                                         const float* __restrict__ bias, int score, int normalize,
                                                         float scale, bool wide, bool wide_bias,
                                                         int32_t* __restrict__ ids, float* __restrict__ weights) {
  const int li = threadIdx.x & (LANES - 1);
  const int64_t t = (int64_t)blockIdx.x * (kThreads / LANES) + threadIdx.x / LANES;
  const bool live = t < tokens;  // the others work on the last token and write nothing: exchanges need all lanes
  const T* row = logits + (live ? t : tokens - 1) * E;
  float l[VPL];
  load_logits<T, VPL>(row, E, li, wide, l);
  float top = 0.0f, sum = 1.0f;
  if (score == MOE_SCORE_SOFTMAX && !normalize) {
    float m = l[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) m = fmaxf(m, l[i]);
    top = fmaxf(group_fmax<LANES>(m), -FLT_MAX);
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) s += expf(l[i] - top);
    sum = group_sum<LANES>(s);
  }
  if (bias) {  // a masked logit stays -inf, whatever its bias; a sum of -inf or NaN is not chosen either
    float b[VPL];
    load_row<float, VPL>(bias, E, li, wide_bias, b);
#pragma unroll
    for (int i = 0; i < VPL; ++i) l[i] = l[i] > kNegInf ? l[i] + b[i] : kNegInf;
  }
  double key[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) key[i] = key_pattern(key_bits(l[i]), li * VPL + i);
  sort_desc(key);
  constexpr int kKeep = KMAX < VPL ? KMAX : VPL;
  int my_id = -1;
  for (int j = 0; j < topk; ++j) {
    const double w = group_max<LANES>(key[0]);
    const uint64_t b = __builtin_bit_cast(uint64_t, w);
    const int id = (uint32_t)(b >> 30) ? MOE_MAX_EXPERTS - 1 - (int)(b & (MOE_MAX_EXPERTS - 1)) : -1;  // key 0: masked
    if (li == j) my_id = id;
    const bool mine = key[0] == w;
#pragma unroll
    for (int i = 0; i + 1 < kKeep; ++i) key[i] = pick(mine, key[i + 1], key[i]);
    if (mine) key[kKeep - 1] = 0.0;
  }
  const float z = my_id >= 0 ? clean(logit_at<T>(row, my_id)) : kNegInf;
  const float s = group_score<LANES>(z, score, normalize, top, sum);
  if (live && li < topk) {
    ids[t * topk + li] = my_id;
    weights[t * topk + li] = my_id >= 0 ? s * scale : 0.0f;
  }
}

// Gradient: with q the (normalised) score of a choice and g = scale * dw,
//   softmax            dl_i = p_i (g_i - sum_j p_j g_j) over all unmasked i
//   softmax normalised the same over the chosen logits alone
//   sigmoid            dl_j = g_j s_j (1 - s_j)
//   sigmoid normalised dl_j = (g_j - sum_i q_i g_i) q_j (1 - s_j)
// The choices' values are scattered into the token's row in LDS and the row
// is written once, densely: 8191 x 64 of bf16 in 4.5 us, a launch.
template <class T, int VPL>
__global__ __launch_bounds__(kThreads) void route_bwd_kernel(const T* __restrict__ logits, int64_t tokens, int E,
                                                             int topk, const int32_t* __restrict__ ids,
                                                             const float* __restrict__ dweights, int score,
                                                             int normalize, float scale, bool wide,
                                                             T* __restrict__ dlogits) {
  extern __shared__ float lrows[];
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
  if (t >= tokens) return;  // whole waves; no barrier below
  float* row = lrows + (threadIdx.x >> 6) * (64 * VPL);
  const bool dense = score == MOE_SCORE_SOFTMAX && !normalize;
  float z = kNegInf, g = 0.0f;
  int id = -1;
  if (lane < topk) {
    id = ids[t * topk + lane];
    if ((uint32_t)id >= (uint32_t)E) id = -1;
    if (id >= 0) {
      z = clean(logit_at<T>(logits, t * E + id));
      g = scale * dweights[t * topk + lane];
    }
  }
  float l[VPL], top = 0.0f, sum = 1.0f;
  if (dense) {
    load_logits<T, VPL>(logits + t * E, E, lane, wide, l);
    float m = l[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) m = fmaxf(m, l[i]);
    top = fmaxf(group_fmax<64>(m), -FLT_MAX);
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      l[i] = expf(l[i] - top);
      s += l[i];
    }
    sum = wave_sum(s);
  }
  const bool on = z > kNegInf;  // a masked logit that was named as a choice has no gradient
  const float q = group_score<64>(z, score, normalize, top, sum);
  if (!on) g = 0.0f;
  const float inner = wave_sum(q * g);
  float d;
  if (score == MOE_SCORE_SIGMOID) {
    const float s1 = on ? 1.0f / (1.0f + expf(z)) : 0.0f;  // 1 - sigmoid(z)
    d = normalize ? (g - inner) * q * s1 : g * q * s1;
  } else {
    d = normalize ? q * (g - inner) : q * g;
  }
  float v[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) row[lane * VPL + i] = dense && sum > 0.0f ? -inner * (l[i] / sum) : 0.0f;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  if (on) atomicAdd(&row[id], d);
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
  for (int i = 0; i < VPL; ++i) v[i] = row[lane * VPL + i];
  T* out = dlogits + t * E;
  const int e0 = lane * VPL;
  if (wide) {
    constexpr int kPer = 16 / (int)sizeof(T) < VPL ? 16 / (int)sizeof(T) : VPL;
    if (e0 < E) {
#pragma unroll
      for (int i = 0; i < VPL; i += kPer) {
        typedef T vec_t __attribute__((ext_vector_type(kPer)));
        vec_t o;
#pragma unroll
        for (int q2 = 0; q2 < kPer; ++q2) {
          if constexpr (sizeof(T) == 4) o[q2] = v[i + q2];
          else o[q2] = to_bf16(v[i + q2]);
        }
        *reinterpret_cast<vec_t*>(out + e0 + i) = o;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (e0 + i < E) {
        if constexpr (sizeof(T) == 4) out[e0 + i] = v[i];
        else out[e0 + i] = to_bf16(v[i]);
      }
  }
}

// ------------------------------------------------------------------- plan

constexpr int kPlanSteps = 4;         // steps of 64 pairs a wave ranks in the split form
// The one-launch form: steps of 64 pairs a wave keeps in registers, experts.
// With more steps the three launches are faster (at 11: 20 us and 15).
constexpr int kSmallSteps = 4;
constexpr int kSmallExperts = 512;
constexpr int kSmallThreads = 1024;
constexpr int kSmallWaves = kSmallThreads / 64;
constexpr int kSmallPairs = kSmallThreads * kSmallSteps;

__device__ __forceinline__ int expert_of(const int32_t* ids, int64_t p, int64_t end, int E) {
  const int e = p < end ? ids[p] : -1;
  return (uint32_t)e < (uint32_t)E ? e : -1;
}

// Ranks the 64 pairs of a wave step: a pair's rank is base[e] plus the pairs
// of the same expert in lower lanes; base[e] then moves on by their number.
__device__ __forceinline__ int wave_rank(int e, int ebits, int32_t* base) {
  uint64_t same = __ballot(e >= 0);
  for (int b = 0; b < ebits; ++b) {
    const uint64_t bal = __ballot((e >> b) & 1);
    same &= (e >> b) & 1 ? bal : ~bal;
  }
  const uint64_t below = same & ((1ull << (threadIdx.x & 63)) - 1);
  int r = 0;
  if (e >= 0) r = base[e] + __popcll(below);
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  if (e >= 0 && below == 0) base[e] += __popcll(same);
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  return r;
}

// Exclusive prefix over the experts of their padded group sizes, from counts
// in cnt[E]; leaves begin[e] in `begin`, returns the total.  All threads of
// the work-group take part; blockDim.x is a multiple of 64.
__device__ int group_begins(const int32_t* cnt, int E, int32_t* begin, int32_t* wtot) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, nw = blockDim.x >> 6;
  const int per = (E + blockDim.x - 1) / blockDim.x;
  int mine = 0;
  for (int i = 0; i < per; ++i) {
    const int e = tid * per + i;
    if (e < E) mine += (cnt[e] + kTileRows - 1) / kTileRows * kTileRows;
  }
  int inc = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(inc, d);
    if (lane >= d) inc += o;
  }
  if (lane == 63) wtot[wave] = inc;
  __syncthreads();
  int before = 0, total = 0;
  for (int w = 0; w < nw; ++w) {
    if (w < wave) before += wtot[w];
    total += wtot[w];
  }
  int at = before + inc - mine;
  for (int i = 0; i < per; ++i) {
    const int e = tid * per + i;
    if (e < E) {
      begin[e] = at;
      at += (cnt[e] + kTileRows - 1) / kTileRows * kTileRows;
    }
  }
  __syncthreads();
  return total;
}

// src of the rows no pair has: the padding of the groups of experts `part`,
// `part` + `parts`, .., a wave each, and a share of the rows past the last
// group.
__device__ __forceinline__ void fill_padding(int part, int parts, int64_t cap, int E, int total, const int32_t* begin,
                                             const int32_t* cnt, int32_t* src) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  for (int e = part * waves + wave; e < E; e += parts * waves) {
    const int64_t end = min<int64_t>(begin[e] + (cnt[e] + kTileRows - 1) / kTileRows * kTileRows, cap);
    for (int64_t r = begin[e] + cnt[e] + lane; r < end; r += 64) src[r] = -1;
  }
  for (int64_t r = total + (int64_t)part * blockDim.x + threadIdx.x; r < cap; r += (int64_t)parts * blockDim.x) src[r] = -1;
}

__device__ __forceinline__ void write_ends(int E, const int32_t* begin, const int32_t* cnt, int64_t cap, int total,
                                           int32_t* offs, int32_t* counts, int32_t* status) {
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    offs[e] = begin[e] + (cnt[e] + kTileRows - 1) / kTileRows * kTileRows;
    counts[e] = cnt[e];
  }
  if (threadIdx.x == 0 && total > cap) atomicOr(status, NVFP4G_DEV_OVERFLOW);
}

__device__ __forceinline__ void write_pair(int64_t p, int row, int64_t cap, int32_t* rows, int32_t* src) {
  const bool fits = row >= 0 && row < cap;
  rows[p] = fits ? row : -1;
  if (fits) src[row] = (int32_t)p;
}

// Few pairs: one work-group does it all (a launch costs more than the work):
// 5.6 us for 8 pairs.
__global__ __launch_bounds__(kSmallThreads) void plan_small_kernel(const int32_t* __restrict__ ids, int pairs, int E,
                                                                   int ebits, int64_t cap, int32_t* offs,
                                                                   int32_t* counts, int32_t* rows, int32_t* src,
                                                                   int32_t* status) {
  extern __shared__ int32_t lds[];
  int32_t* hist = lds;                        // [kSmallWaves][E]: a wave's counts, then its first ranks
  int32_t* cnt = hist + kSmallWaves * E;      // [E]
  int32_t* begin = cnt + E;                   // [E]
  int32_t* wtot = begin + E;                  // [kSmallWaves]
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int share = (pairs + kSmallThreads - 1) / kSmallThreads * 64;  // pairs of a wave, whole steps
  const int p0 = wave * share, p1 = min(p0 + share, pairs);
  int id[kSmallSteps];
#pragma unroll
  for (int i = 0; i < kSmallSteps; ++i)
    if (p0 + 64 * i < p1) id[i] = expert_of(ids, p0 + 64 * i + lane, p1, E);
  for (int i = tid; i < kSmallWaves * E; i += kSmallThreads) hist[i] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kSmallSteps; ++i)
    if (p0 + 64 * i < p1 && id[i] >= 0) atomicAdd(&hist[wave * E + id[i]], 1);
  __syncthreads();
  for (int e = tid; e < E; e += kSmallThreads) {
    int acc = 0;
    for (int w = 0; w < kSmallWaves; ++w) {
      const int v = hist[w * E + e];
      hist[w * E + e] = acc;
      acc += v;
    }
    cnt[e] = acc;
  }
  __syncthreads();
  const int total = group_begins(cnt, E, begin, wtot);
#pragma unroll
  for (int i = 0; i < kSmallSteps; ++i) {
    const int p = p0 + 64 * i;
    if (p >= p1) break;
    const int r = wave_rank(id[i], ebits, hist + wave * E);
    if (p + lane < p1) write_pair(p + lane, id[i] >= 0 ? begin[id[i]] + r : -1, cap, rows, src);
  }
  fill_padding(0, 1, cap, E, total, begin, cnt, src);
  write_ends(E, begin, cnt, cap, total, offs, counts, status);
}

// Many pairs, step 1: counts of each work-group's pairs (a chunk, kPlanSteps
// steps a wave), ws[chunk][E].  A chunk a wave gave the next step four times as
// much to add up: 7.4 us instead of 5.9 for 262144 pairs of 256 experts (three
// launches: 20 us and 16).
__global__ __launch_bounds__(kThreads) void plan_count_kernel(const int32_t* __restrict__ ids, int64_t pairs, int E,
                                                              int32_t* __restrict__ ws) {
  extern __shared__ int32_t lds[];
  const int64_t p0 = (int64_t)blockIdx.x * blockDim.x * kPlanSteps + threadIdx.x;
  int id[kPlanSteps];
#pragma unroll
  for (int i = 0; i < kPlanSteps; ++i) id[i] = expert_of(ids, p0 + i * (int64_t)blockDim.x, pairs, E);
  for (int i = threadIdx.x; i < E; i += blockDim.x) lds[i] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPlanSteps; ++i)
    if (id[i] >= 0) atomicAdd(&lds[id[i]], 1);
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x) ws[(int64_t)blockIdx.x * E + e] = lds[e];
}

// Step 2: per expert the exclusive prefix over the chunks (in place) and the
// count, which goes to the row after the last chunk.  A work-group takes 16
// experts; 64 groups of 16 lanes take a run of chunks each.
constexpr int kScanExperts = 16;
__global__ __launch_bounds__(kSmallThreads) void plan_scan_kernel(int32_t* __restrict__ ws, int64_t chunks, int E) {
  constexpr int kRuns = kSmallThreads / kScanExperts;
  __shared__ int32_t part[kRuns][kScanExperts];
  const int le = threadIdx.x % kScanExperts, run = threadIdx.x / kScanExperts;
  const int e = blockIdx.x * kScanExperts + le;
  const int64_t per = (chunks + kRuns - 1) / kRuns;
  const int64_t c0 = min(run * per, chunks), c1 = min(c0 + per, chunks);
  int acc = 0;
  if (e < E) {
#pragma unroll 8
    for (int64_t c = c0; c < c1; ++c) acc += ws[c * E + e];
  }
  part[run][le] = acc;
  __syncthreads();
  int at = 0, total = 0;
#pragma unroll 16
  for (int r = 0; r < kRuns; ++r) {
    const int v = part[r][le];
    at += r < run ? v : 0;
    total += v;
  }
  if (e < E) {
#pragma unroll 8
    for (int64_t c = c0; c < c1; ++c) {
      const int v = ws[c * E + e];
      ws[c * E + e] = at;
      at += v;
    }
    if (run == 0) ws[chunks * E + e] = total;
  }
}

// Step 3: every work-group finds the groups' begins from the counts (they
// are few), counts its waves' pairs again and ranks them, and fills its share
// of the padding.
__global__ __launch_bounds__(kThreads) void plan_write_kernel(const int32_t* __restrict__ ids, int64_t pairs, int E,
                                                              int ebits, int64_t cap, const int32_t* __restrict__ ws,
                                                              int64_t chunks, int32_t* offs, int32_t* counts,
                                                              int32_t* rows, int32_t* src, int32_t* status) {
  extern __shared__ int32_t lds[];
  const int waves = blockDim.x >> 6;
  int32_t* base = lds;              // [waves][E]: a wave's counts, then its first ranks
  int32_t* cnt = base + waves * E;  // [E]
  int32_t* begin = cnt + E;         // [E]
  int32_t* wtot = begin + E;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t p0 = ((int64_t)blockIdx.x * waves + wave) * 64 * kPlanSteps;
  int id[kPlanSteps];
#pragma unroll
  for (int i = 0; i < kPlanSteps; ++i) id[i] = expert_of(ids, p0 + 64 * i + lane, pairs, E);
  for (int e = threadIdx.x; e < waves * E; e += blockDim.x) base[e] = 0;
  for (int e = threadIdx.x; e < E; e += blockDim.x) cnt[e] = ws[chunks * E + e];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPlanSteps; ++i)
    if (id[i] >= 0) atomicAdd(&base[wave * E + id[i]], 1);
  const int total = group_begins(cnt, E, begin, wtot);  // with barriers: the counts are there after it
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    int acc = ws[(int64_t)blockIdx.x * E + e];
    for (int w = 0; w < waves; ++w) {
      const int v = base[w * E + e];
      base[w * E + e] = acc;
      acc += v;
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPlanSteps; ++i) {
    const int64_t p = p0 + 64 * i;
    if (p >= pairs) break;
    const int r = wave_rank(id[i], ebits, base + wave * E);
    if (p + lane < pairs) write_pair(p + lane, id[i] >= 0 ? begin[id[i]] + r : -1, cap, rows, src);
  }
  fill_padding(blockIdx.x, gridDim.x, cap, E, total, begin, cnt, src);
  if (blockIdx.x == 0) write_ends(E, begin, cnt, cap, total, offs, counts, status);
}

// ------------------------------------------------------------- host side

bool plan_is_small(int64_t pairs, int32_t E) { return pairs <= kSmallPairs && E <= kSmallExperts; }
// Threads of the counting and writing steps: four waves, each with its
// counts of all experts in LDS; one wave where four would pass 64 KB.
int plan_threads(int32_t E) { return E <= 2048 ? kThreads : 64; }
int64_t plan_chunks(int64_t pairs, int32_t E) {
  const int64_t chunk = (int64_t)plan_threads(E) * kPlanSteps;
  return pairs > 0 ? (pairs + chunk - 1) / chunk : 1;
}

int check_route(int32_t type, int64_t tokens, int32_t E, int32_t topk, int32_t score) {
  if (!valid_type(type) || (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID)) return NVFP4G_EINVAL;
  if (E < 1 || E > MOE_MAX_EXPERTS || topk < 1 || topk > MOE_MAX_TOPK || topk > E) return NVFP4G_EINVAL;
  if (tokens < 0 || tokens > MOE_MAX_PAIRS / topk) return NVFP4G_EINVAL;
  return NVFP4G_OK;
}

// Calls f(VPL) with the experts a lane holds as a compile-time constant.
template <class F>
void with_vpl(int E, F f) {
  const int v = (E + 63) / 64;
  if (v <= 1) f(std::integral_constant<int, 1>());
  else if (v <= 2) f(std::integral_constant<int, 2>());
  else if (v <= 4) f(std::integral_constant<int, 4>());
  else if (v <= 8) f(std::integral_constant<int, 8>());
  else if (v <= 16) f(std::integral_constant<int, 16>());
  else f(std::integral_constant<int, 64>());
}

// Vector loads of a lane's experts: a row starts on their alignment and no
// lane's piece is cut by the row's end.
bool wide_rows(const void* p, int E, int vpl, int size) {
  const int piece = vpl * size < 16 ? vpl * size : 16;
  return E % vpl == 0 && (int64_t)E * size % piece == 0 && aligned(p, piece);
}

struct RouteCall {
  const void* logits;
  int64_t tokens;
  int32_t E, topk;
  const float* bias;
  int32_t score, normalize;
  float scale;
  int32_t* ids;
  float* weights;
  hipStream_t stream;
};

template <class T, int LANES, int VPL, int KMAX>
int launch_route(const RouteCall& c) {
  const dim3 grid((uint32_t)((c.tokens + kThreads / LANES - 1) / (kThreads / LANES)));
  hipLaunchKernelGGL((route_kernel<T, LANES, VPL, KMAX>), grid, dim3(kThreads), 0, c.stream, (const T*)c.logits,
                     c.tokens, c.E, c.topk, c.bias, c.score, c.normalize, c.scale,
                     wide_rows(c.logits, c.E, VPL, sizeof(T)), wide_rows(c.bias, c.E, VPL, 4), c.ids, c.weights);
  return hip_status();
}

// As few lanes as hold the experts, 8 or 16 each, and the choices, one each.
template <class T>
int route(const RouteCall& c) {
  if (c.topk <= 8) {
    if (c.E <= 64) return launch_route<T, 8, 8, 8>(c);
    if (c.E <= 128) return launch_route<T, 8, 16, 8>(c);
    if (c.E <= 256) return launch_route<T, 16, 16, 8>(c);
    if (c.E <= 512) return launch_route<T, 32, 16, 8>(c);
    if (c.E <= 1024) return launch_route<T, 64, 16, 8>(c);
  }
  if (c.E <= 256) return launch_route<T, 16, 16, 16>(c);
  if (c.E <= 1024) return launch_route<T, 64, 16, 16>(c);
  return launch_route<T, 64, 64, 16>(c);
}

}  // namespace

extern "C" {

int moe_route(const void* logits, int32_t logits_type, int64_t tokens, int32_t num_experts, int32_t topk,
              const float* select_bias, int32_t score, int32_t normalize, float scale, int32_t* ids, float* weights,
              void* stream) {
  const int rc = check_route(logits_type, tokens, num_experts, topk, score);
  if (rc) return rc;
  if (tokens == 0) return NVFP4G_OK;
  if (!logits || !ids || !weights) return NVFP4G_EINVAL;
  if (!aligned(logits, logits_type == MOE_F32 ? 4 : 2) || !aligned(select_bias, 4) || !aligned(ids, 4) ||
      !aligned(weights, 4))
    return NVFP4G_EALIGN;
  const RouteCall c{logits, tokens, num_experts, topk, select_bias, score, normalize, scale, ids, weights, (hipStream_t)stream};
  return logits_type == MOE_F32 ? route<float>(c) : route<uint16_t>(c);
}

int moe_route_bwd(const void* logits, int32_t logits_type, int64_t tokens, int32_t num_experts, int32_t topk,
                  const int32_t* ids, const float* dweights, int32_t score, int32_t normalize, float scale,
                  void* dlogits, void* stream) {
  const int rc = check_route(logits_type, tokens, num_experts, topk, score);
  if (rc) return rc;
  if (tokens == 0) return NVFP4G_OK;
  if (!logits || !ids || !dweights || !dlogits) return NVFP4G_EINVAL;
  const int size = logits_type == MOE_F32 ? 4 : 2;
  if (!aligned(logits, size) || !aligned(dlogits, size) || !aligned(ids, 4) || !aligned(dweights, 4))
    return NVFP4G_EALIGN;
  const dim3 grid((uint32_t)((tokens + 3) / 4));
  with_vpl(num_experts, [&](auto v) {
    constexpr int VPL = decltype(v)::value;
    const bool wide = wide_rows(logits, num_experts, VPL, size) && wide_rows(dlogits, num_experts, VPL, size);
    const uint32_t lds = 4 * 64 * VPL * 4;
    if (logits_type == MOE_F32)
      hipLaunchKernelGGL((route_bwd_kernel<float, VPL>), grid, dim3(kThreads), lds, (hipStream_t)stream,
                         (const float*)logits, tokens, num_experts, topk, ids, dweights, score, normalize, scale, wide,
                         (float*)dlogits);
    else
      hipLaunchKernelGGL((route_bwd_kernel<uint16_t, VPL>), grid, dim3(kThreads), lds, (hipStream_t)stream,
                         (const uint16_t*)logits, tokens, num_experts, topk, ids, dweights, score, normalize, scale,
                         wide, (uint16_t*)dlogits);
  });
  return hip_status();
}

int64_t moe_plan_workspace(int64_t pairs, int32_t num_experts) {
  if (pairs < 0 || num_experts < 1 || plan_is_small(pairs, num_experts)) return 0;
  return (plan_chunks(pairs, num_experts) + 1) * num_experts * 4;
}

int moe_plan(const int32_t* ids, int64_t pairs, int32_t num_experts, int64_t m_capacity, int32_t* offs,
             int32_t* counts, int32_t* rows, int32_t* src, int32_t* d_status, void* workspace,
             int64_t workspace_bytes, void* stream) {
  const int E = num_experts;
  if (pairs < 0 || pairs > MOE_MAX_PAIRS || E < 1 || E > MOE_MAX_EXPERTS) return NVFP4G_EINVAL;
  if (m_capacity < 0 || m_capacity > kMaxRows || m_capacity % kTileRows != 0) return NVFP4G_EINVAL;
  if ((pairs && (!ids || !rows)) || (m_capacity && !src) || !offs || !counts || !d_status) return NVFP4G_EINVAL;
  if (!aligned(ids, 4) || !aligned(rows, 4) || !aligned(src, 4) || !aligned(offs, 4) || !aligned(counts, 4) ||
      !aligned(d_status, 4) || !aligned(workspace, 4))
    return NVFP4G_EALIGN;
  int ebits = 1;
  while ((1 << ebits) < E) ++ebits;
  const hipStream_t st = (hipStream_t)stream;
  if (plan_is_small(pairs, E)) {
    const uint32_t lds = ((kSmallWaves + 2) * E + kSmallWaves) * 4;
    hipLaunchKernelGGL(plan_small_kernel, dim3(1), dim3(kSmallThreads), lds, st, ids, (int)pairs, E, ebits, m_capacity,
                       offs, counts, rows, src, d_status);
    return hip_status();
  }
  if (!workspace || workspace_bytes < moe_plan_workspace(pairs, E)) return NVFP4G_EINVAL;
  int32_t* ws = (int32_t*)workspace;
  const int64_t chunks = plan_chunks(pairs, E);
  const int threads = plan_threads(E), waves = threads / 64;
  const dim3 grid((uint32_t)chunks);
  hipLaunchKernelGGL(plan_count_kernel, grid, dim3(threads), E * 4, st, ids, pairs, E, ws);
  hipLaunchKernelGGL(plan_scan_kernel, dim3((E + kScanExperts - 1) / kScanExperts), dim3(kSmallThreads), 0, st, ws,
                     chunks, E);
  hipLaunchKernelGGL(plan_write_kernel, grid, dim3(threads), ((waves + 2) * E + waves) * 4, st, ids, pairs, E, ebits,
                     m_capacity, ws, chunks, offs, counts, rows, src, d_status);
  return hip_status();
}

}  // extern "C"
