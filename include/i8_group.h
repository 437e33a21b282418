/*
 * i8_group.h -- C ABI of the products in 8-bit integers in libnvfp4g.so: rows
 * with a scale for each token times weights with a scale for each channel, as
 * one projection, grouped by expert, as the experts' gated block, and for
 * single tokens.
 *
 * Conventions are those of nvfp4_group.h and moe_ops.h: every pointer except
 * h_splits is a device pointer owned by the caller, calls only enqueue work on
 * `stream`, are checked on the host first (a call that fails enqueues nothing
 * and returns a negative NVFP4G_* status), keep no state and can be captured
 * in a hipGraph; a workspace belongs to one call at a time.
 *
 * A line of k codes q (int8) with scale s (fp32) stands for q * s.  A product
 * of two lines is (sum_c qa[c] qb[c]) * sa * sb: the sum is exact in int32 for
 * every k up to I8_MAX_K and all codes, -128 among them, then becomes fp32 and
 * is multiplied in this order, each step rounded to fp32.
 *
 * k: a positive multiple of 16 up to I8_MAX_K; n a multiple of 16 up to 2^20;
 * codes, x and outputs are 16-byte aligned, scales 4-byte.
 */
#ifndef I8_GROUP_H_
#define I8_GROUP_H_

#include <stdint.h>

#include "moe_ops.h"
#include "nvfp4_group.h"

#ifdef __cplusplus
extern "C" {
#endif

#define I8_MAX_K 131056

/* Cast of rows: x bf16 [rows, k] -> q [rows, k], scale [rows],
 *     A = max |x|,   scale = A / 127,   q = the whole number nearest to
 *     x * (127 / A), ties to even, quotient and product rounded to fp32
 * (for A below 2^-100 on x and A times 2^64).  A row of zeros gives scale 0
 * and codes 0; a row with an infinity or NaN gives scale NaN and codes 0.
 * Weights have the same form, a channel to a row.  The graph-safe form (routing
 * and status as in nvfp4_group_cast_graphsafe) neither reads nor writes rows
 * at or beyond offs[E-1]. */
int i8_group_cast(const uint16_t* x, int64_t rows, int64_t k, int8_t* q,
                  float* scale, void* stream);
int i8_group_cast_graphsafe(const uint16_t* x, int64_t m_capacity, int64_t k,
                            int32_t num_experts, const int32_t* d_offs,
                            int8_t* q, float* scale, int32_t* d_status,
                            void* stream);

/* One projection of any number of rows: out[r, j] of a [rows, k] and b [n, k],
 * out [rows, n] fp32 or rounded once to bf16 (out_type MOE_F32, MOE_BF16).
 * workspace: i8_linear_workspace(rows, k, n) bytes, 16-byte aligned (NULL if
 * that is 0); at most 32 MiB. */
int64_t i8_linear_workspace(int64_t rows, int64_t k, int64_t n);
int i8_linear(const int8_t* a_q, const float* a_scale, int64_t rows, int64_t k,
              const int8_t* b_q, const float* b_scale, int64_t n, void* out,
              int32_t out_type, void* workspace, int64_t workspace_bytes,
              void* stream);

/* The experts' products: packed rows a [sum_m, k] in 128-row groups times the
 * weights b [E, n, k] (scales [E, n]) of the row's expert; routing as in
 * nvfp4_group_gemm, out as in i8_linear. */
int i8_group_gemm(const int8_t* a_q, const float* a_scale, const int8_t* b_q,
                  const float* b_scale, int64_t sum_m, int64_t n, int64_t k,
                  int32_t num_experts, const int64_t* h_splits, void* out,
                  int32_t out_type, void* stream);
int i8_group_gemm_graphsafe(const int8_t* a_q, const float* a_scale,
                            const int8_t* b_q, const float* b_scale,
                            int64_t m_capacity, int64_t n, int64_t k,
                            int32_t num_experts, const int32_t* d_offs,
                            void* out, int32_t out_type, int32_t* d_status,
                            void* stream);

/* The experts' gated block: b [E, 2f, k] with the f gate channels first,
 * h = act(g) * u (moe_glu's act), g and u kept in fp32 up to h, which is
 * rounded once to bf16 [sum_m, f].  f: a multiple of 16 up to 2^19. */
int i8_group_glu(const int8_t* a_q, const float* a_scale, const int8_t* b_q,
                 const float* b_scale, int64_t sum_m, int64_t f, int64_t k,
                 int32_t num_experts, const int64_t* h_splits, int32_t act,
                 uint16_t* h, void* stream);
int i8_group_glu_graphsafe(const int8_t* a_q, const float* a_scale,
                           const int8_t* b_q, const float* b_scale,
                           int64_t m_capacity, int64_t f, int64_t k,
                           int32_t num_experts, const int32_t* d_offs,
                           int32_t act, uint16_t* h, int32_t* d_status,
                           void* stream);

/* Forms for single tokens, as moe_token_glu and moe_token_linear: bf16 rows,
 * cast as by i8_group_cast inside the call, times the weights of each pair's
 * expert; an id outside 0 .. E-1 gives a row of zeros.  pairs <=
 * MOE_MAX_TOKEN_PAIRS.
 *   i8_token_glu     x [tokens, k], ids [tokens, topk], b [E, 2f, k],
 *                    h bf16 [tokens * topk, f]
 *   i8_token_linear  x [pairs, k], ids [pairs], b [E, n, k], out fp32 [pairs, n] */
int i8_token_glu(const uint16_t* x, int64_t tokens, int64_t k, int32_t topk,
                 const int32_t* ids, const int8_t* b_q, const float* b_scale,
                 int64_t f, int32_t num_experts, int32_t act, uint16_t* h,
                 void* stream);
int i8_token_linear(const uint16_t* x, int64_t pairs, int64_t k,
                    const int32_t* ids, const int8_t* b_q, const float* b_scale,
                    int64_t n, int32_t num_experts, float* out, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* I8_GROUP_H_ */
