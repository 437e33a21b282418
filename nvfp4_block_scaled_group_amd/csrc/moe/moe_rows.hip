// moe_rows.hip -- tokens into the packed 128-row expert groups and back, with
// the gradients, behind the C ABI of include/moe_ops.h.
//
// All of it moves memory: dispatch reads a token's row once and writes it to
// its topk packed rows; combine reads topk packed rows and writes one.  A unit
// of work is one token times a run of columns; a lane moves 16 bytes of bf16
// (8 columns) at a time.  HBM bounds all of it once there are tokens enough:
// dispatch of 8192 x 7168 to 8 experts each in 210 us, 5.0 TB/s (a large copy
// reaches 5.85, a large fill 5.4); the gradient of combine, 4095 x 2048, 6 each, fp32 results, in
// 63 us, 5.0 TB/s; combine of 33 x 2064 in 4 us, a launch.
#include "moe_common.hpp"

namespace {

using namespace moe;

typedef uint32_t u32v4 __attribute__((ext_vector_type(4)));

constexpr int kLaneCols = 8;            // columns of a lane: 16 bytes of bf16
constexpr int64_t kRowCols = 64 * kLaneCols;  // columns of a wave at a time

__device__ __forceinline__ void unpack8(const u32v4& q, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16lo(q[i]);
    v[2 * i + 1] = bf16hi(q[i]);
  }
}
__device__ __forceinline__ u32v4 pack8(const float (&v)[8]) {
  return u32v4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
}

// Eight consecutive values of a packed row, as fp32.
template <bool F32>
struct Piece {
  u32v4 q[F32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* base, int64_t at) {
    const u32v4* p = reinterpret_cast<const u32v4*>(reinterpret_cast<const char*>(base) + at * (F32 ? 4 : 2));
#pragma unroll
    for (int i = 0; i < (F32 ? 2 : 1); ++i) q[i] = __builtin_nontemporal_load(p + i);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < (F32 ? 2 : 1); ++i) q[i] = u32v4{0, 0, 0, 0};
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    if constexpr (F32) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(q[i >> 2][i & 3]);
    } else {
      unpack8(q[0], v);
    }
  }
};

// Zeros for the padding rows among kPadRows rows (src -1 below the last
// group's end).  Only the last tile of a group has any, so most work-groups
// end after a look at src; a whole tile each left the padding to one
// work-group in 128 rows (17 us for 8 groups of 3232 columns).
constexpr int kPadRows = 16;
__device__ __forceinline__ void zero_padding(int64_t piece, int64_t width, const int32_t* src, int32_t total,
                                             int64_t cap, uint16_t* out) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t end = min<int64_t>(total, cap);
  for (int r = wave; r < kPadRows; r += kThreads / 64) {
    const int64_t row = piece * kPadRows + r;
    if (row >= end) break;
    if (uni(src[row]) >= 0) continue;
    u32v4* o = reinterpret_cast<u32v4*>(out + row * width);
    for (int64_t c = lane; c < width / kLaneCols; c += 64) __builtin_nontemporal_store(u32v4{0, 0, 0, 0}, o + c);
  }
}

// Dispatch.  Work-groups 0 .. units/4-1: a wave takes a token and `span`
// columns of it; the others zero the padding among kPadRows rows (those past
// the last row find none).
__global__ __launch_bounds__(kThreads) void dispatch_kernel(const uint16_t* __restrict__ x, int64_t tokens,
                                                            int64_t width, int topk, int32_t span, int32_t spans,
                                                            const int32_t* __restrict__ rows,
                                                            const int32_t* __restrict__ src,
                                                            const int32_t* __restrict__ offs, int E, int64_t cap,
                                                            const float* __restrict__ weights, uint32_t token_groups,
                                                            uint16_t* __restrict__ out) {
  const uint32_t group = line_index();
  if (group >= token_groups) {
    zero_padding(group - token_groups, width, src, offs[E - 1], cap, out);
    return;
  }
  const int lane = threadIdx.x & 63;
  const int64_t unit = (int64_t)group * (kThreads / 64) + uni((uint32_t)(threadIdx.x >> 6));
  const int64_t t = unit / spans;
  if (t >= tokens) return;
  const int64_t c0 = (unit - t * spans) * span, c1 = min<int64_t>(c0 + span, width);
  const int32_t* trow = rows + t * topk;
  for (int64_t c = c0 + lane * kLaneCols; c < c1; c += 64 * kLaneCols) {
    const u32v4 q = __builtin_nontemporal_load(reinterpret_cast<const u32v4*>(x + t * width + c));
    for (int j = 0; j < topk; ++j) {
      const int64_t r = uni(trow[j]);
      if ((uint64_t)r >= (uint64_t)cap) continue;
      u32v4 o = q;
      if (weights) {
        const float w = __uint_as_float(uni(__float_as_uint(weights[t * topk + j])));
        float v[8];
        unpack8(q, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= w;
        o = pack8(v);
      }
      __builtin_nontemporal_store(o, reinterpret_cast<u32v4*>(out + r * width + c));
    }
  }
}

// Gradient of combine: a work-group takes a token; every packed row of it is
// read once for its dot product with the token's row and written once.  KMAX:
// choices whose sums a lane keeps in registers.
template <bool F32, int KMAX>
__global__ __launch_bounds__(kThreads) void dispatch_dot_kernel(const uint16_t* __restrict__ x, int64_t tokens,
                                                                int64_t width, int topk,
                                                                const int32_t* __restrict__ rows,
                                                                const int32_t* __restrict__ src,
                                                                const int32_t* __restrict__ offs, int E, int64_t cap,
                                                                const float* __restrict__ weights,
                                                                const void* __restrict__ y, uint32_t token_groups,
                                                                uint16_t* __restrict__ out,
                                                                float* __restrict__ dweights) {
  __shared__ float part[kThreads / 64][KMAX];
  const uint32_t group = line_index();
  if (group >= token_groups) {
    zero_padding(group - token_groups, width, src, offs[E - 1], cap, out);
    return;
  }
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = group;
  float acc[KMAX], w[KMAX];
  int64_t r[KMAX];
#pragma unroll
  for (int j = 0; j < KMAX; ++j) {
    acc[j] = 0.0f;
    r[j] = j < topk ? (int64_t)uni(rows[t * topk + j]) : -1;
    if (r[j] >= cap) r[j] = -1;
    w[j] = weights && j < topk ? __uint_as_float(uni(__float_as_uint(weights[t * topk + j]))) : 1.0f;
  }
  for (int64_t c = (int64_t)threadIdx.x * kLaneCols; c < width; c += kThreads * kLaneCols) {
    float v[8];
    unpack8(*reinterpret_cast<const u32v4*>(x + t * width + c), v);
    Piece<F32> p[KMAX];
#pragma unroll
    for (int j = 0; j < KMAX; ++j)
      if (r[j] >= 0) p[j].load(y, r[j] * width + c);
#pragma unroll
    for (int j = 0; j < KMAX; ++j) {
      if (r[j] < 0) continue;
      float yv[8], o[8];
      p[j].get(yv);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        acc[j] = __builtin_fmaf(v[i], yv[i], acc[j]);
        o[i] = v[i] * w[j];
      }
      __builtin_nontemporal_store(pack8(o), reinterpret_cast<u32v4*>(out + r[j] * width + c));
    }
  }
#pragma unroll
  for (int j = 0; j < KMAX; ++j) {
    const float s = wave_sum(acc[j]);
    if (lane == 0) part[wave][j] = s;
  }
  __syncthreads();
  if ((int)threadIdx.x < topk) {
    const int j = threadIdx.x;
    float s = 0.0f;
    for (int i = 0; i < kThreads / 64; ++i) s += part[i][j];
    const int64_t row = rows[t * topk + j];
    dweights[t * topk + j] = row >= 0 && row < cap ? s : 0.0f;
  }
}

// Combine.  A wave takes a token and 512 columns; the loads of KMAX choices are
// in flight together, the sum runs in the order of the choices.  One piece of a
// row a wave: 8192 x 7168, 8 choices of fp32 in 360 to 374 us, 5.4 TB/s (four
// pieces one after another 411).
template <bool F32, int KMAX>
__global__ __launch_bounds__(kThreads) void combine_kernel(const void* __restrict__ y, int64_t cap, int64_t tokens,
                                                           int64_t width, int topk, int32_t pieces,
                                                           const int32_t* __restrict__ rows,
                                                           const float* __restrict__ weights,
                                                           uint16_t* __restrict__ out) {
  const int lane = threadIdx.x & 63;
  const int64_t unit = (int64_t)line_index() * (kThreads / 64) + uni((uint32_t)(threadIdx.x >> 6));
  const int64_t t = unit / pieces, c = (unit - t * pieces) * kRowCols + lane * kLaneCols;
  if (t >= tokens) return;
  int64_t r[KMAX];
  float w[KMAX];
#pragma unroll
  for (int j = 0; j < KMAX; ++j) {
    r[j] = j < topk ? (int64_t)uni(rows[t * topk + j]) : -1;
    if (r[j] >= cap) r[j] = -1;
    w[j] = weights && j < topk ? __uint_as_float(uni(__float_as_uint(weights[t * topk + j]))) : 1.0f;
  }
  if (c >= width) return;
  Piece<F32> p[KMAX];
#pragma unroll
  for (int j = 0; j < KMAX; ++j)
    if (r[j] >= 0) p[j].load(y, r[j] * width + c);
  float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < KMAX; ++j) {
    if (r[j] < 0) continue;
    float v[8];
    p[j].get(v);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = __builtin_fmaf(w[j], v[i], acc[i]);
  }
  __builtin_nontemporal_store(pack8(acc), reinterpret_cast<u32v4*>(out + t * width + c));
}

// ------------------------------------------------------------- host side

int check_rows(int64_t tokens, int64_t width, int32_t topk, int64_t cap) {
  if (width <= 0 || width % 16 != 0 || width > kMaxK || topk < 1 || topk > MOE_MAX_TOPK) return NVFP4G_EINVAL;
  if (tokens < 0 || tokens > MOE_MAX_PAIRS / topk) return NVFP4G_EINVAL;
  if (cap < 0 || cap > kMaxRows || cap % kTileRows != 0) return NVFP4G_EINVAL;
  return NVFP4G_OK;
}

// Columns of a wave of dispatch: whole lane rows of 512 columns, up to four
// where that leaves 4096 waves.  64 tokens of 7168: 11.5 us with one, 13.9 with
// four; 8192 tokens: 218 and 211.
int32_t pick_span(int64_t tokens, int64_t width) {
  constexpr int64_t kWant = 4096;
  const int64_t pieces = (width + kRowCols - 1) / kRowCols;
  int64_t per = tokens * pieces / kWant;
  per = per < 1 ? 1 : per > 4 ? 4 : per;
  return (int32_t)(per * kRowCols);
}

template <class F>
void with_choices(int topk, F f) {
  if (topk <= 2) f(std::integral_constant<int, 2>());
  else if (topk <= 4) f(std::integral_constant<int, 4>());
  else if (topk <= 8) f(std::integral_constant<int, 8>());
  else f(std::integral_constant<int, 16>());
}

}  // namespace

extern "C" {

int moe_dispatch(const uint16_t* x, int64_t tokens, int64_t width, int32_t topk, const int32_t* rows,
                 const int32_t* src, const int32_t* offs, int32_t num_experts, int64_t m_capacity,
                 const float* weights, const void* y, int32_t y_type, uint16_t* out, float* dweights, void* stream) {
  const int rc = check_rows(tokens, width, topk, m_capacity);
  if (rc) return rc;
  if (num_experts < 1 || num_experts > MOE_MAX_EXPERTS || !valid_type(y_type)) return NVFP4G_EINVAL;
  if (tokens && (y != nullptr) != (dweights != nullptr)) return NVFP4G_EINVAL;
  if ((tokens && (!x || !rows)) || (m_capacity && (!src || !out)) || !offs) return NVFP4G_EINVAL;
  if (!aligned(x, 16) || !aligned(out, 16) || !aligned(y, 16) || !aligned(rows, 4) || !aligned(src, 4) ||
      !aligned(offs, 4) || !aligned(weights, 4) || !aligned(dweights, 4))
    return NVFP4G_EALIGN;
  const uint32_t tiles = (uint32_t)(m_capacity / kPadRows);
  const hipStream_t st = (hipStream_t)stream;
  if (y && dweights) {
    const uint32_t groups = (uint32_t)tokens;
    if (groups + tiles == 0) return NVFP4G_OK;
    const dim3 grid = line_grid(groups + tiles);
    with_choices(topk, [&](auto v) {
      constexpr int KMAX = decltype(v)::value;
      if (y_type == MOE_F32)
        hipLaunchKernelGGL((dispatch_dot_kernel<true, KMAX>), grid, dim3(kThreads), 0, st, x, tokens, width,
                           topk, rows, src, offs, num_experts, m_capacity, weights, y, groups, out, dweights);
      else
        hipLaunchKernelGGL((dispatch_dot_kernel<false, KMAX>), grid, dim3(kThreads), 0, st, x, tokens, width,
                           topk, rows, src, offs, num_experts, m_capacity, weights, y, groups, out, dweights);
    });
    return hip_status();
  }
  const int32_t span = pick_span(tokens, width), spans = (int32_t)((width + span - 1) / span);
  const int64_t want = (tokens * spans + kThreads / 64 - 1) / (kThreads / 64);
  if (want + tiles > (int64_t)INT32_MAX) return NVFP4G_EINVAL;
  const uint32_t groups = (uint32_t)want;
  if (groups + tiles == 0) return NVFP4G_OK;
  hipLaunchKernelGGL(dispatch_kernel, line_grid(groups + tiles), dim3(kThreads), 0, st, x, tokens, width, topk, span,
                     spans, rows, src, offs, num_experts, m_capacity, weights, groups, out);
  return hip_status();
}

int moe_combine(const void* y, int32_t y_type, int64_t m_capacity, int64_t tokens, int64_t width, int32_t topk,
                const int32_t* rows, const float* weights, uint16_t* out, void* stream) {
  const int rc = check_rows(tokens, width, topk, 0);
  if (rc) return rc;
  if (m_capacity < 0 || m_capacity > kMaxRows || !valid_type(y_type)) return NVFP4G_EINVAL;
  if (tokens == 0) return NVFP4G_OK;
  if ((m_capacity && !y) || !rows || !out) return NVFP4G_EINVAL;
  if (!aligned(y, 16) || !aligned(out, 16) || !aligned(rows, 4) || !aligned(weights, 4)) return NVFP4G_EALIGN;
  const int32_t pieces = (int32_t)((width + kRowCols - 1) / kRowCols);
  if ((tokens * pieces + 3) / 4 > (int64_t)INT32_MAX) return NVFP4G_EINVAL;
  const dim3 grid = line_grid((uint32_t)((tokens * pieces + 3) / 4));
  with_choices(topk, [&](auto v) {
    constexpr int KMAX = decltype(v)::value;
    if (y_type == MOE_F32)
      hipLaunchKernelGGL((combine_kernel<true, KMAX>), grid, dim3(kThreads), 0, (hipStream_t)stream, y, m_capacity,
                         tokens, width, topk, pieces, rows, weights, out);
    else
      hipLaunchKernelGGL((combine_kernel<false, KMAX>), grid, dim3(kThreads), 0, (hipStream_t)stream, y, m_capacity,
                         tokens, width, topk, pieces, rows, weights, out);
  });
  return hip_status();
}

}  // extern "C"
