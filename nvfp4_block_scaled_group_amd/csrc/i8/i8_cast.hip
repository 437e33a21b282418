// i8_cast.hip -- cast of bf16 rows to 8-bit integers with a scale for each
// row, behind the C ABI of include/i8_group.h.
//
// It reads 2 bytes an element and writes 1: memory bounds it (65536 x 7168 in 223 us,
// 6.3 TB/s, the rate of a copy and more).  A wave or a work-group takes a row, whose
// values stay in registers between the maximum and the codes; rows past 8192
// columns are read twice.
#include "i8_common.hpp"

namespace {

using namespace i8;

constexpr int kSegCols = 512;  // a wave's 16-byte loads: 8 columns a lane
constexpr int kRegSegs = 8;     // of a wave's row at most

// Rows that exist: all of them, or the routed ones.  Every wave checks all ends:
// up to 256 experts that costs nothing (65536 x 7168 in 250 us), 1024 of them 404.
__device__ __forceinline__ bool routed_rows(const Routing& R, int64_t* rows) {
  if (R.d_offs) {
    if (!routing_ok(R)) return false;
    *rows = route_end(R, R.num_experts - 1);
  }
  return true;
}

// Codes past the caches where they would not stay there (`stream`).
__device__ __forceinline__ void put(int8_t* to, u32x2 codes, bool stream) {
  if (stream) __builtin_nontemporal_store(codes, reinterpret_cast<u32x2*>(to));
  else *reinterpret_cast<u32x2*>(to) = codes;
}
// From 16 MB of codes on: 65536 x 7168 in 223 us (248 through the caches), 4095 x 7168
// 15.1 (16.1); 1024 x 7168 with its reader 10.9 (10.6), 193 x 5920 alone 4.0 (3.5).
bool streams(int64_t rows, int64_t k) { return rows * k >= 1 << 24; }

template <int SEGS>
__global__ __launch_bounds__(kThreads) void cast_rows_kernel(const uint16_t* __restrict__ x, int64_t rows, int64_t k,
                                                             Routing R, int8_t* __restrict__ q,
                                                             float* __restrict__ scale, bool stream) {
  if (!routed_rows(R, &rows)) return;
  const int lane = threadIdx.x & 63;
  const int64_t r = (int64_t)line_index() * (kThreads / 64) + uni((int32_t)(threadIdx.x >> 6));
  if (r >= rows) return;
  const rsrc_t xr = range_rsrc(x + r * k, 2 * k);
  u32x4 v[SEGS];
#pragma unroll
  for (int s = 0; s < SEGS; ++s)
    v[s] = __builtin_amdgcn_raw_buffer_load_b128(xr, 16 * lane, s * 2 * kSegCols, kLoadStream);
  uint32_t m = 0;
#pragma unroll
  for (int s = 0; s < SEGS; ++s) m = max(m, abs_max8(v[s]));
  m = wave_reduce(m, [](uint32_t a, uint32_t b) { return max(a, b); });
  const RowCast c = row_cast(m);
  if (lane == 0) scale[r] = c.scale;
#pragma unroll
  for (int s = 0; s < SEGS; ++s) {
    const int64_t col = s * kSegCols + 8 * lane;
    if (col < k) put(q + r * k + col, cast8(v[s], c), stream);
  }
}

// A row of up to 2048 SEGS columns on the four waves of a work-group.
template <int SEGS>
__global__ __launch_bounds__(kThreads) void cast_wide_kernel(const uint16_t* __restrict__ x, int64_t rows, int64_t k,
                                                             Routing R, int8_t* __restrict__ q,
                                                             float* __restrict__ scale, bool stream) {
  __shared__ uint32_t lmax[kThreads / 64];
  if (!routed_rows(R, &rows)) return;
  const int64_t r = line_index();
  if (r >= rows) return;
  const rsrc_t xr = range_rsrc(x + r * k, 2 * k);
  u32x4 v[SEGS];
#pragma unroll
  for (int s = 0; s < SEGS; ++s)
    v[s] = __builtin_amdgcn_raw_buffer_load_b128(xr, 16 * threadIdx.x, s * 16 * kThreads, kLoadStream);
  uint32_t m = 0;
#pragma unroll
  for (int s = 0; s < SEGS; ++s) m = max(m, abs_max8(v[s]));
  m = wave_reduce(m, [](uint32_t a, uint32_t b) { return max(a, b); });
  if ((threadIdx.x & 63) == 0) lmax[threadIdx.x >> 6] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) m = max(m, lmax[w]);
  const RowCast c = row_cast(m);
  if (threadIdx.x == 0) scale[r] = c.scale;
#pragma unroll
  for (int s = 0; s < SEGS; ++s) {
    const int64_t col = 8 * ((int64_t)s * kThreads + threadIdx.x);
    if (col < k) put(q + r * k + col, cast8(v[s], c), stream);
  }
}

__global__ __launch_bounds__(kThreads) void cast_long_kernel(const uint16_t* __restrict__ x, int64_t rows, int64_t k,
                                                             Routing R, int8_t* __restrict__ q,
                                                             float* __restrict__ scale, bool stream) {
  __shared__ uint32_t lmax[kThreads / 64];
  if (!routed_rows(R, &rows)) return;
  const int64_t r = line_index();
  if (r >= rows) return;
  const u32x4* row = reinterpret_cast<const u32x4*>(x + r * k);
  uint32_t m = 0;
  for (int64_t i = threadIdx.x; i < k / 8; i += kThreads) m = max(m, abs_max8(row[i]));
  m = wave_reduce(m, [](uint32_t a, uint32_t b) { return max(a, b); });
  if ((threadIdx.x & 63) == 0) lmax[threadIdx.x >> 6] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) m = max(m, lmax[w]);
  const RowCast c = row_cast(m);
  if (threadIdx.x == 0) scale[r] = c.scale;
  for (int64_t i = threadIdx.x; i < k / 8; i += kThreads) put(q + r * k + 8 * i, cast8(row[i], c), stream);
}

template <int SEGS>
void launch(const uint16_t* x, int64_t rows, int64_t k, const Routing& R, int8_t* q, float* scale, hipStream_t st) {
  const uint32_t per = kThreads / 64;
  hipLaunchKernelGGL((cast_rows_kernel<SEGS>), line_grid((uint32_t)((rows + per - 1) / per)), dim3(kThreads), 0, st, x,
                     rows, k, R, q, scale, streams(rows, k));
}

template <int SEGS>
int launch_wide(const uint16_t* x, int64_t rows, int64_t k, const Routing& R, int8_t* q, float* scale, hipStream_t st) {
  hipLaunchKernelGGL((cast_wide_kernel<SEGS>), line_grid((uint32_t)rows), dim3(kThreads), 0, st, x, rows, k, R, q, scale,
                     streams(rows, k));
  return hip_status();
}

int cast(const uint16_t* x, int64_t rows, int64_t k, const Routing& R, int8_t* q, float* scale, hipStream_t st) {
  const int64_t segs = (k + kSegCols - 1) / kSegCols;
  // A work-group to a row where a wave would hold many pieces or the rows do not
  // fill the CUs: 7168 columns, 193 rows 3.4 us (a wave to a row 4.4), 65536 rows
  // 248 (255); 4096 columns, 193 rows 3.1 (3.5), 16384 rows 33.6 (34.0); 1536
  // columns, 16384 rows 18.3 (13.4).
  if (segs > kRegSegs) {
    if (segs <= 12) return launch_wide<3>(x, rows, k, R, q, scale, st);
    if (segs <= 16) return launch_wide<4>(x, rows, k, R, q, scale, st);
    hipLaunchKernelGGL(cast_long_kernel, line_grid((uint32_t)rows), dim3(kThreads), 0, st, x, rows, k, R, q, scale,
                       streams(rows, k));
  } else if (segs > 2 && rows <= 512) {
    return segs <= 4 ? launch_wide<1>(x, rows, k, R, q, scale, st) : launch_wide<2>(x, rows, k, R, q, scale, st);
  } else if (segs <= 1) {
    launch<1>(x, rows, k, R, q, scale, st);
  } else if (segs <= 2) {
    launch<2>(x, rows, k, R, q, scale, st);
  } else if (segs <= 4) {
    launch<4>(x, rows, k, R, q, scale, st);
  } else {
    launch<kRegSegs>(x, rows, k, R, q, scale, st);
  }
  return hip_status();
}

int check_cast(const uint16_t* x, int64_t rows, int64_t k, const int8_t* q, const float* scale) {
  if (!valid_k(k) || rows < 0 || rows > kMaxRows) return NVFP4G_EINVAL;
  if (rows && (!x || !q || !scale)) return NVFP4G_EINVAL;
  if (!aligned(x, 16) || !aligned(q, 16) || !aligned(scale, 4)) return NVFP4G_EALIGN;
  return NVFP4G_OK;
}

}  // namespace

extern "C" {

int i8_group_cast(const uint16_t* x, int64_t rows, int64_t k, int8_t* q, float* scale, void* stream) {
  const int rc = check_cast(x, rows, k, q, scale);
  if (rc || rows == 0) return rc;
  Routing R;
  R.num_experts = 0;
  R.m_capacity = (int32_t)rows;
  R.d_offs = nullptr;
  R.d_status = nullptr;
  return cast(x, rows, k, R, q, scale, (hipStream_t)stream);
}

int i8_group_cast_graphsafe(const uint16_t* x, int64_t m_capacity, int64_t k, int32_t num_experts,
                            const int32_t* d_offs, int8_t* q, float* scale, int32_t* d_status, void* stream) {
  int rc = check_cast(x, m_capacity, k, q, scale);
  if (rc) return rc;
  Routing R;
  R.num_experts = num_experts;
  R.m_capacity = (int32_t)m_capacity;
  if ((rc = graph_routing(d_offs, d_status, num_experts, m_capacity, &R))) return rc;
  if (m_capacity == 0) return NVFP4G_OK;
  return cast(x, m_capacity, k, R, q, scale, (hipStream_t)stream);
}

}  // extern "C"
