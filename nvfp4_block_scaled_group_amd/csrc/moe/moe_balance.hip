// moe_balance.hip -- balance loss of a router over the sequences of a batch,
// with the counts it is made of, and its gradient, behind the C ABI of
// include/moe_ops.h.
//
//   p[t, e]  softmax of the unmasked logits, or s_e / sum_i s_i of sigmoids
//   loss     coef / S * sum_s E / (k n_s^2) * sum_e counts[s, e] probs[s, e]
//   a[s, e]  its derivative in p[t, e]: coef / S * E / (k n_s^2) * counts[s, e]
//   dl[t, e] p_e (a_e - sum_i p_i a_i), with sigmoids times 1 - s_e
//
// Forward: a work-group takes a chunk of rows, LANES lanes a token with VPL
// experts each, and keeps the sums of its experts in registers from token to
// token; a sequence that ends (or the chunk's end) joins the groups in LDS in a
// fixed order and writes one slot.  The pair (chunk, sequence) goes up in one
// of the two or in both from slot to slot, so slot chunk + sequence is its own
// without any list.  A second launch adds the slots of each sequence in order,
// and the work-group of it that ends last adds the sequences.  No float is added
// by an atomic.  With many sequences a third launch adds them.
//
// What bounds it: reading the logits and, in the gradient, writing as much
// (32768 x 256 fp32: 10.4 to 11.0 us forward, 3.1 to 3.3 TB/s of logits and choices, of
// which two to three dependent rounds of loads; 5.3 for the join, three quarters of it a
// launch and two more such rounds; 14.7 to 15.1 for the gradient, 4.5 TB/s).  Small batches cost a launch (33 x 8: one work-group,
// 4.0 us, and 2.9 for the gradient).
#include <algorithm>

#include "moe_logits.hpp"

namespace {

using namespace moe;

constexpr int kFwdThreads = 1024;
// Threads of a forward work-group: many experts a lane need the registers of
// many waves, and small chunks give 1024 threads nothing to do.
constexpr int fwd_threads(int vpl, bool small) { return vpl <= 16 && !small ? kFwdThreads : kFwdThreads / 4; }
constexpr int kChunks = 256;    // chunks of a large batch: one for each CU
constexpr int kOneRows = 128;   // rows of one sequence that one work-group takes by itself
constexpr int kJoinCols = 32;   // columns of a joining work-group

// The first sequence from lo on whose end is above row t (num_seqs if none): the
// row's sequence.  Whatever the ends hold, the result is in lo .. num_seqs.
__device__ __forceinline__ int sequence_of(const int32_t* ends, int num_seqs, int64_t t, int lo = 0) {
  if (!ends) return 0;
  int hi = num_seqs;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (ends[mid] > t) hi = mid; else lo = mid + 1;
  }
  return lo;
}

// Probabilities of a token's experts from its logits (masked ones -inf, which
// get 0), l replaced; with sigmoids slope gets 1 - s.  Returns whether any
// expert is unmasked.
template <int LANES, int VPL, bool SIGMOID>
__device__ __forceinline__ bool probabilities(float (&l)[VPL], float (&slope)[SIGMOID ? VPL : 1]) {
  float m = l[0];
#pragma unroll
  for (int i = 1; i < VPL; ++i) m = fmaxf(m, l[i]);
  m = group_fmax<LANES>(m);
  const bool any = m > kNegInf;
  float sum = 0.0f;
  if constexpr (SIGMOID) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      // s = 1 / (1 + e^-l) and 1 - s = s e^-l, which keeps its digits near s = 1
      const float e = __expf(-l[i]), s = __builtin_amdgcn_rcpf(1.0f + e);  // e^inf = inf: s = 0 where masked
      slope[i] = s > 0.0f ? s * e : 1.0f;
      l[i] = s;
      sum += s;
    }
  } else {
    const float top = fmaxf(m, -FLT_MAX);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      l[i] = __expf(l[i] - top);
      sum += l[i];
    }
  }
  sum = group_sum<LANES>(sum);
  const float inv = sum >= FLT_MIN ? 1.0f / sum : 0.0f;
#pragma unroll
  for (int i = 0; i < VPL; ++i) l[i] *= inv;
  return any;
}

struct Slots {
  float* probs;     // [slots, E]
  int32_t* counts;  // [slots, E]
  int32_t* tokens;  // [slots]
  float* loss;      // [num_seqs, blocks of kJoinCols columns]
  uint32_t* done;   // work-groups of the second launch that have ended: 0 after the first
};
struct Results {
  float* loss;
  int32_t* counts;
  float* probs;
  int32_t* tokens;
};

// coef / S * E / (k n^2): the weight of a sequence with n tokens.
__device__ __forceinline__ float sequence_weight(float coef, int num_seqs, int E, int topk, int n) {
  return n > 0 ? coef / (float)num_seqs * (float)E / (float)topk / ((float)n * (float)n) : 0.0f;
}

// Sum over the work-group's threads, in a fixed order, in thread 0.  lred: one
// float a wave.
__device__ __forceinline__ float block_sum(float v, float* lred, int waves) {
  v = wave_sum(v);
  if ((threadIdx.x & 63) == 0) lred[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.0f;
  if (threadIdx.x == 0)
    for (int w = 0; w < waves; ++w) s += lred[w];
  return s;
}

// whole: the launch is one work-group and one sequence, and writes the results
// themselves.
template <class T, int LANES, int VPL, bool SIGMOID, bool SMALL>
__global__ __launch_bounds__(fwd_threads(VPL, SMALL)) void balance_kernel(
    const T* __restrict__ logits, int64_t tokens, int E, int topk, const int32_t* __restrict__ ids,
    const int32_t* __restrict__ ends, int num_seqs, int64_t rows, bool wide, bool whole, float coef, Slots P,
    Results out) {
  constexpr int kFwd = fwd_threads(VPL, SMALL), kWaves = kFwd / 64;
  extern __shared__ float lds[];  // E sums of each wave, E counts
  __shared__ int32_t lany;
  __shared__ float lred[kWaves];
  int32_t* lcount = reinterpret_cast<int32_t*>(lds + kWaves * E);
  constexpr int kPass = kFwd / LANES;  // tokens at a time
  const int tid = threadIdx.x, li = tid & (LANES - 1), wave = tid >> 6;
  const int64_t c0 = (int64_t)blockIdx.x * rows, c1 = min(c0 + rows, tokens);
  if (!whole && blockIdx.x == 0 && tid == 0) *P.done = 0;
  int64_t at = c0;
  for (int s = sequence_of(ends, num_seqs, c0); s < num_seqs && at < c1;) {
    const int64_t to = ends ? min<int64_t>(ends[s], c1) : c1;
    // Empty sequences, however many, by one search: ends padded to a fixed number
    // end with a long run of them (8191 rows of 64 experts in 11 sequences padded to
    // 65535: 0.49 ms, the same as without a row; one after another 9 ms more).
    if (to <= at) {
      s = sequence_of(ends, num_seqs, at, s + 1);
      continue;
    }
    const int64_t t0 = at + tid / LANES, p0 = at * topk + tid, p1 = to * topk;
    float l[VPL];
    load_logits<T, VPL>(logits + min(t0, tokens - 1) * E, E, li, wide, l);
    const int first = p0 < p1 ? ids[p0] : -1;  // on its way beside the logits
    for (int e = tid; e < E; e += kFwd) lcount[e] = 0;
    if (tid == 0) lany = 0;
    __syncthreads();
    if ((uint32_t)first < (uint32_t)E) atomicAdd(&lcount[first], 1);
    for (int64_t p = p0 + kFwd; p < p1; p += kFwd) {
      const int e = ids[p];
      if ((uint32_t)e < (uint32_t)E) atomicAdd(&lcount[e], 1);
    }
    float acc[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) acc[i] = 0.0f;
    int n = 0;
    for (int64_t t = t0; t - tid / LANES < to; t += kPass) {
      float next[VPL], slope[SIGMOID ? VPL : 1];
      load_logits<T, VPL>(logits + min(t + kPass, tokens - 1) * E, E, li, wide, next);
      const bool any = probabilities<LANES, VPL, SIGMOID>(l, slope);
      if (t < to) {
        n += any;
#pragma unroll
        for (int i = 0; i < VPL; ++i) acc[i] += l[i];
      }
#pragma unroll
      for (int i = 0; i < VPL; ++i) l[i] = next[i];
    }
    if (li == 0 && n) atomicAdd(&lany, n);
    // the groups of a wave, then the waves in order
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      float v = acc[i];
      if constexpr (LANES <= 8) v += __uint_as_float(exchange<3>(__float_as_uint(v)));
      if constexpr (LANES <= 16) v += __uint_as_float(exchange<4>(__float_as_uint(v)));
      if constexpr (LANES <= 32) v += __uint_as_float(exchange<5>(__float_as_uint(v)));
      if ((tid & 63) < LANES && li * VPL + i < E) lds[wave * E + li * VPL + i] = v;
    }
    __syncthreads();
    const int64_t slot = (int64_t)blockIdx.x + s;
    float* probs = whole ? out.probs : P.probs + slot * E;
    int32_t* counts = whole ? out.counts : P.counts + slot * E;
    float v = 0.0f;
    for (int e = tid; e < E; e += kFwd) {
      float sum = lds[e];
      for (int w = 1; w < kWaves; ++w) sum += lds[w * E + e];
      const int c = lcount[e];
      probs[e] = sum;
      counts[e] = c;
      v += (float)c * sum;
    }
    if (whole) {
      v = block_sum(v, lred, kWaves);
      if (tid == 0) {
        *out.tokens = lany;
        const bool good = !ends || (ends[0] >= 0 && ends[0] <= tokens);
        *out.loss = good ? v * sequence_weight(coef, 1, E, topk, lany) : __uint_as_float(0x7FC00000u);
      }
      return;
    }
    if (tid == 0) P.tokens[slot] = lany;
    __syncthreads();
    at = to;
    ++s;
  }
  // one work-group and an empty sequence
  if (whole) {
    for (int e = tid; e < E; e += kFwd) {
      out.probs[e] = 0.0f;
      out.counts[e] = 0;
    }
    if (tid == 0) {
      *out.tokens = 0;
      *out.loss = !ends || ends[0] == 0 ? 0.0f : __uint_as_float(0x7FC00000u);
    }
  }
}

// The shares of the loss, in order, by a work-group.
__device__ __forceinline__ float add_shares(const float* loss, int64_t n, float* lred) {
  float v = 0.0f;
  for (int64_t i = threadIdx.x; i < n; i += kFwdThreads)
    v += __hip_atomic_load(loss + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return block_sum(v, lred, kFwdThreads / 64);
}

// The slots of a sequence, in order: work-group (b, s) has kJoinCols columns and
// a share of the loss; the last one to end adds the shares in order, or with
// `apart` a launch of its own.
__global__ __launch_bounds__(kFwdThreads) void balance_join_kernel(Slots P, int64_t tokens, int E, int topk,
                                                                   const int32_t* __restrict__ ends, int num_seqs,
                                                                   int64_t rows, float coef, bool apart, Results out) {
  constexpr int kParts = kFwdThreads / kJoinCols, kWaves = kFwdThreads / 64, kAhead = 8;
  __shared__ float lsum[kWaves][kJoinCols + 1];
  __shared__ int32_t lcount[kWaves][kJoinCols + 1];
  __shared__ int32_t ltok[kWaves];
  __shared__ float lred[kWaves];
  __shared__ bool llast;
  const int s = blockIdx.y, tid = threadIdx.x, part = tid / kJoinCols, c = tid % kJoinCols;
  const int64_t from = ends && s ? ends[s - 1] : 0, to = ends ? ends[s] : tokens;
  const bool good = from >= 0 && to >= from && to <= tokens;
  const int64_t b = min(max(from, (int64_t)0), tokens), e = min(max(to, b), tokens);
  const int64_t first = b / rows, last = e > b ? (e - 1) / rows : first - 1;
  const int col = blockIdx.x * kJoinCols + c;
  float sum = 0.0f;
  int cnt = 0, tok = 0;
  for (int64_t j0 = first + part; j0 <= last; j0 += kParts * kAhead) {
    float p[kAhead];
    int n[kAhead], t[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {  // every load on its way before one is used; past the last slot they count nothing
      const int64_t slot = min(j0 + i * kParts, last) + s;
      p[i] = P.probs[slot * E + min(col, E - 1)];
      n[i] = P.counts[slot * E + min(col, E - 1)];
      t[i] = P.tokens[slot];
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (j0 + i * kParts <= last) {
        sum += p[i];
        cnt += n[i];
        tok += t[i];
      }
  }
  // the two parts of a wave, then the waves in order
  static_assert(kJoinCols == 32, "a wave holds two parts");
  sum += __uint_as_float(exchange<5>(__float_as_uint(sum)));
  cnt += (int)exchange<5>((uint32_t)cnt);
  tok += (int)exchange<5>((uint32_t)tok);
  if ((tid & 63) < kJoinCols) {
    lsum[tid >> 6][c] = sum;
    lcount[tid >> 6][c] = cnt;
    if (c == 0) ltok[tid >> 6] = tok;
  }
  __syncthreads();
  if (tid < 64) {
    float v = 0.0f;
    tok = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) tok += ltok[w];
    if (tid < kJoinCols && col < E) {
      sum = 0.0f;
      cnt = 0;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        sum += lsum[w][c];
        cnt += lcount[w][c];
      }
      out.probs[(int64_t)s * E + col] = sum;
      out.counts[(int64_t)s * E + col] = cnt;
      v = (float)cnt * sum;
    }
    v = wave_sum(v);
    if (tid == 0) {
      if (blockIdx.x == 0) out.tokens[s] = tok;
      const float share = good ? v * sequence_weight(coef, num_seqs, E, topk, tok) : __uint_as_float(0x7FC00000u);
      // shares go past the caches of an XCD, and before the count that tells of them
      __hip_atomic_store(P.loss + (int64_t)s * gridDim.x + blockIdx.x, share, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      const uint32_t all = gridDim.x * gridDim.y;
      llast = !apart && __hip_atomic_fetch_add(P.done, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) + 1 == all;
    }
  }
  if (apart) return;
  __syncthreads();
  if (!llast) return;
  const float v = add_shares(P.loss, (int64_t)gridDim.x * gridDim.y, lred);
  if (tid == 0) *out.loss = v;
}

__global__ __launch_bounds__(kFwdThreads) void balance_loss_kernel(const float* __restrict__ shares, int64_t n,
                                                                   float* __restrict__ loss) {
  __shared__ float lred[kFwdThreads / 64];
  const float v = add_shares(shares, n, lred);
  if (threadIdx.x == 0) *loss = v;
}

template <class T, int LANES, int VPL, bool SIGMOID>
__global__ __launch_bounds__(kThreads) void balance_bwd_kernel(const T* __restrict__ logits, int64_t tokens, int E,
                                                               int topk, const int32_t* __restrict__ ends,
                                                               int num_seqs, float coef,
                                                               const int32_t* __restrict__ counts,
                                                               const int32_t* __restrict__ seq_tokens,
                                                               const float* __restrict__ dloss, const T* add,
                                                               bool wide, bool wide_counts, T* dlogits) {
  const int li = threadIdx.x & (LANES - 1);
  const int64_t t = (int64_t)line_index() * (kThreads / LANES) + threadIdx.x / LANES;
  const bool live = t < tokens;  // the others work on the last token and write nothing: exchanges need all lanes
  const int64_t tt = live ? t : tokens - 1;
  float l[VPL], slope[SIGMOID ? VPL : 1], extra[VPL], a[VPL];
  load_logits<T, VPL>(logits + tt * E, E, li, wide, l);
  if (add) load_row<T, VPL>(add + tt * E, E, li, wide, extra);
  const int s = sequence_of(ends, num_seqs, tt);
  const bool in = s < num_seqs;
  const int row = in ? s : 0;
  load_row<int32_t, VPL>(counts + (int64_t)row * E, E, li, wide_counts, a);
  const float w = in ? sequence_weight(coef, num_seqs, E, topk, seq_tokens[row]) * (dloss ? *dloss : 1.0f) : 0.0f;
  probabilities<LANES, VPL, SIGMOID>(l, slope);
  float inner = 0.0f;
#pragma unroll
  for (int i = 0; i < VPL; ++i) inner += l[i] * a[i];
  inner = group_sum<LANES>(inner);
  float d[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    d[i] = l[i] * (a[i] - inner) * w;
    if constexpr (SIGMOID) d[i] *= slope[i];
    d[i] = in && l[i] > 0.0f ? d[i] : 0.0f;
    if (add) d[i] += extra[i];
  }
  const int e0 = li * VPL;
  if (!live) return;
  T* o = dlogits + t * E;
  if (wide) {
    constexpr int kPer = 16 / (int)sizeof(T) < VPL ? 16 / (int)sizeof(T) : VPL;
    if (e0 < E) {
#pragma unroll
      for (int i = 0; i < VPL; i += kPer) {
        typedef T vec_t __attribute__((ext_vector_type(kPer)));
        vec_t v;
#pragma unroll
        for (int q = 0; q < kPer; ++q) {
          if constexpr (sizeof(T) == 4) v[q] = d[i + q];
          else v[q] = to_bf16(d[i + q]);
        }
        *reinterpret_cast<vec_t*>(o + e0 + i) = v;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (e0 + i < E) {
        if constexpr (sizeof(T) == 4) o[e0 + i] = d[i];
        else o[e0 + i] = to_bf16(d[i]);
      }
  }
}

// ------------------------------------------------------------- host side

bool one_group(int64_t tokens, int num_seqs) { return num_seqs == 1 && tokens <= kOneRows; }
// Rows of a chunk: 32 at least, fewer where several sequences would share them,
// since a chunk takes its sequences one after another.
int64_t least_rows(int64_t tokens, int num_seqs) {
  return num_seqs == 1 ? 32 : std::clamp<int64_t>(tokens / num_seqs / 4, 4, 32);
}
int64_t chunk_rows(int64_t tokens, int num_seqs) {
  if (one_group(tokens, num_seqs)) return kOneRows;
  return std::max(least_rows(tokens, num_seqs), (tokens + kChunks - 1) / kChunks);
}
// Joining work-groups that count themselves, so that the last one adds the
// sequences' shares; more of them wait for each other at the counter, 18 ns apiece,
// and a launch of its own adds (8191 rows; 64 work-groups 12 us both ways, 128:
// 13.2 counted and 12.5 apart, 256: 16 and 13, 2048: 56 and 27, 131070: 2377 and 643).
constexpr int64_t kCountedJoin = 128;
int64_t join_blocks(int E) { return (E + kJoinCols - 1) / kJoinCols; }

int check_balance(const void* logits, int32_t type, int64_t tokens, int32_t E, int32_t topk, int32_t score,
                  const int32_t* ends, int32_t num_seqs) {
  if (!valid_type(type) || (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID)) return NVFP4G_EINVAL;
  if (E < 1 || E > MOE_MAX_EXPERTS || topk < 1 || topk > MOE_MAX_TOPK || topk > E) return NVFP4G_EINVAL;
  if (tokens < 0 || tokens > MOE_MAX_PAIRS / topk || num_seqs < 1 || num_seqs > MOE_MAX_SEQS) return NVFP4G_EINVAL;
  if (tokens && !logits) return NVFP4G_EINVAL;
  if (num_seqs > 1 && !ends) return NVFP4G_EINVAL;
  if (!aligned(logits, type == MOE_F32 ? 4 : 2) || !aligned(ends, 4)) return NVFP4G_EALIGN;
  return NVFP4G_OK;
}

// Calls f with the lanes of a token and the experts of a lane.
template <class F>
void by_experts(int E, F f) {
  if (E <= 32) f(std::integral_constant<int, 8>{}, std::integral_constant<int, 4>{});
  else if (E <= 64) f(std::integral_constant<int, 8>{}, std::integral_constant<int, 8>{});
  else if (E <= 128) f(std::integral_constant<int, 16>{}, std::integral_constant<int, 8>{});
  else if (E <= 256) f(std::integral_constant<int, 32>{}, std::integral_constant<int, 8>{});
  else if (E <= 512) f(std::integral_constant<int, 64>{}, std::integral_constant<int, 8>{});
  else if (E <= 1024) f(std::integral_constant<int, 64>{}, std::integral_constant<int, 16>{});
  else if (E <= 2048) f(std::integral_constant<int, 64>{}, std::integral_constant<int, 32>{});
  else f(std::integral_constant<int, 64>{}, std::integral_constant<int, 64>{});
}

}  // namespace

extern "C" {

int64_t moe_balance_workspace(int64_t tokens, int32_t num_experts, int32_t num_seqs) {
  if (tokens < 0 || tokens > MOE_MAX_PAIRS || num_experts < 1 || num_experts > MOE_MAX_EXPERTS || num_seqs < 1 ||
      num_seqs > MOE_MAX_SEQS)
    return NVFP4G_EINVAL;
  if (one_group(tokens, num_seqs)) return 0;
  // more rows never need fewer bytes, though they may make fewer chunks
  const int64_t least = num_seqs == 1 ? 32 : 4, chunks = std::min<int64_t>(kChunks, (tokens + least - 1) / least);
  return (chunks + num_seqs) * (8 * (int64_t)num_experts + 4) + 4 * num_seqs * join_blocks(num_experts) + 4;
}

int moe_balance(const void* logits, int32_t logits_type, int64_t tokens, int32_t num_experts, int32_t topk,
                const int32_t* ids, int32_t score, const int32_t* seq_ends, int32_t num_seqs, float coef, float* loss,
                int32_t* counts, float* probs, int32_t* seq_tokens, void* workspace, int64_t workspace_bytes,
                void* stream) {
  const int rc = check_balance(logits, logits_type, tokens, num_experts, topk, score, seq_ends, num_seqs);
  if (rc) return rc;
  if ((tokens && !ids) || !loss || !counts || !probs || !seq_tokens) return NVFP4G_EINVAL;
  const int64_t need = moe_balance_workspace(tokens, num_experts, num_seqs);
  if (need && (!workspace || workspace_bytes < need)) return NVFP4G_EINVAL;
  if (!aligned(ids, 4) || !aligned(loss, 4) || !aligned(counts, 4) || !aligned(probs, 4) || !aligned(seq_tokens, 4) ||
      !aligned(workspace, 4))
    return NVFP4G_EALIGN;
  const hipStream_t st = (hipStream_t)stream;
  const int E = num_experts;
  const int64_t rows = chunk_rows(tokens, num_seqs), chunks = (tokens + rows - 1) / rows, slots = chunks + num_seqs;
  const bool whole = one_group(tokens, num_seqs);
  const Results R{loss, counts, probs, seq_tokens};
  const int64_t blocks = join_blocks(E);
  int32_t* w = (int32_t*)workspace;
  const Slots P = whole ? Slots{}
                        : Slots{(float*)w, w + slots * E, w + 2 * slots * E, (float*)(w + 2 * slots * E + slots),
                                (uint32_t*)(w + 2 * slots * E + slots + num_seqs * blocks)};
  const int size = logits_type == MOE_F32 ? 4 : 2;
  by_experts(E, [&](auto lanes, auto vpl) {
    constexpr int L = decltype(lanes)::value, V = decltype(vpl)::value;
    const bool wide = wide_rows(logits, E, V, size);
    auto go = [&](auto* kernel, auto* p, int threads) {
      hipLaunchKernelGGL(kernel, dim3((uint32_t)std::max<int64_t>(chunks, 1)), dim3(threads),
                         4 * E * (threads / 64 + 1), st, p, tokens, E, topk, ids, seq_ends, num_seqs, rows, wide,
                         whole, coef, P, R);
    };
    auto pick = [&](auto sigmoid, auto* p) {
      using T = std::remove_const_t<std::remove_pointer_t<decltype(p)>>;
      constexpr bool G = decltype(sigmoid)::value;
      // the rows of a chunk in two passes of 256 threads
      if (rows * L <= 2 * fwd_threads(V, true)) go(balance_kernel<T, L, V, G, true>, p, fwd_threads(V, true));
      else go(balance_kernel<T, L, V, G, false>, p, fwd_threads(V, false));
    };
    auto typed = [&](auto* p) {
      if (score == MOE_SCORE_SIGMOID) pick(std::true_type{}, p);
      else pick(std::false_type{}, p);
    };
    if (logits_type == MOE_F32) typed((const float*)logits);
    else typed((const uint16_t*)logits);
  });
  if (whole) return hip_status();
  const bool apart = blocks * num_seqs > kCountedJoin;
  hipLaunchKernelGGL(balance_join_kernel, dim3((uint32_t)blocks, (uint32_t)num_seqs), dim3(kFwdThreads), 0, st, P,
                     tokens, E, topk, seq_ends, num_seqs, rows, coef, apart, R);
  if (apart)
    hipLaunchKernelGGL(balance_loss_kernel, dim3(1), dim3(kFwdThreads), 0, st, P.loss, blocks * num_seqs, loss);
  return hip_status();
}

int moe_balance_bwd(const void* logits, int32_t logits_type, int64_t tokens, int32_t num_experts, int32_t topk,
                    int32_t score, const int32_t* seq_ends, int32_t num_seqs, float coef, const int32_t* counts,
                    const int32_t* seq_tokens, const float* dloss, const void* add, void* dlogits, void* stream) {
  const int rc = check_balance(logits, logits_type, tokens, num_experts, topk, score, seq_ends, num_seqs);
  if (rc) return rc;
  if (tokens && (!counts || !seq_tokens || !dlogits)) return NVFP4G_EINVAL;
  const int size = logits_type == MOE_F32 ? 4 : 2;
  if (!aligned(counts, 4) || !aligned(seq_tokens, 4) || !aligned(dloss, 4) || !aligned(add, size) ||
      !aligned(dlogits, size))
    return NVFP4G_EALIGN;
  if (tokens == 0) return NVFP4G_OK;
  const int E = num_experts;
  by_experts(E, [&](auto lanes, auto vpl) {
    constexpr int L = decltype(lanes)::value, V = decltype(vpl)::value;
    const bool wide = wide_rows(logits, E, V, size) && wide_rows(dlogits, E, V, size) && wide_rows(add, E, V, size);
    const int64_t groups = (tokens + kThreads / L - 1) / (kThreads / L);
    auto go = [&](auto* kernel, auto* p) {
      using P = decltype(p);
      hipLaunchKernelGGL(kernel, line_grid((uint32_t)groups), dim3(kThreads), 0, (hipStream_t)stream, p, tokens, E,
                         topk, seq_ends, num_seqs, coef, counts, seq_tokens, dloss, (P)add, wide,
                         wide_rows(counts, E, V, 4), const_cast<std::remove_const_t<std::remove_pointer_t<P>>*>((P)dlogits));
    };
    if (logits_type == MOE_F32) {
      if (score == MOE_SCORE_SIGMOID) go(balance_bwd_kernel<float, L, V, true>, (const float*)logits);
      else go(balance_bwd_kernel<float, L, V, false>, (const float*)logits);
    } else {
      if (score == MOE_SCORE_SIGMOID) go(balance_bwd_kernel<uint16_t, L, V, true>, (const uint16_t*)logits);
      else go(balance_bwd_kernel<uint16_t, L, V, false>, (const uint16_t*)logits);
    }
  });
  return hip_status();
}

}  // extern "C"
