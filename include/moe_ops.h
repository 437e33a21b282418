/*
 * moe_ops.h -- C ABI of the operators around the grouped NVFP4 path in
 * libnvfp4g.so: routing of tokens to experts, movement of rows into and out
 * of the packed 128-row expert groups, the experts' gated feed-forward block
 * with its backward pass and its single-token form, the router's balance loss
 * with its gradient, and low-rank adapters of many requests beside a shared
 * projection.
 *
 * Conventions are those of nvfp4_group.h: every pointer except h_splits is a
 * device pointer owned by the caller, `stream` is a hipStream_t, calls only
 * enqueue work and never synchronise or allocate, arguments are checked on
 * the host first and a call that fails a check enqueues nothing and returns a
 * negative NVFP4G_* status (nvfp4_group_strerror describes it).  The library
 * keeps no state between calls.  All of them can be captured in a hipGraph
 * (kernel launches only); a workspace belongs to one call at a time.
 *
 * An NVFP4 line (codes, E4M3 scales, line amax A) stands for
 * value(code) * value(S) * (A / 2688), in the rowwise layout of
 * nvfp4_group.h.  A "pair" is one choice of one token: p = t * topk + j.
 */
#ifndef MOE_OPS_H_
#define MOE_OPS_H_

#include <stdint.h>

#include "nvfp4_group.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Limits: experts of a router, choices a token, tokens times choices. */
#define MOE_MAX_EXPERTS 4096
#define MOE_MAX_TOPK 16
#define MOE_MAX_PAIRS (1 << 24)

/* Element types of logits and of expert results. */
#define MOE_F32 0
#define MOE_BF16 1

/* Scores: the weight of a chosen expert is its softmax probability over the
 * token's unmasked experts, or the sigmoid of its own logit. */
#define MOE_SCORE_SOFTMAX 0
#define MOE_SCORE_SIGMOID 1

/* Activation of the gate: g / (1 + exp(-g)), or the tanh form of GELU. */
#define MOE_ACT_SILU 0
#define MOE_ACT_GELU 1

/* Selection of experts.  logits [tokens, E] (MOE_F32 or MOE_BF16, row-major).
 * A logit of -inf or NaN masks that expert for that token; +inf counts as
 * the largest finite value.  Per token the topk experts with the largest
 * logit + select_bias[e] (fp32 sum; select_bias may be NULL) are chosen, in
 * descending order, equal keys by the lower index; a sum of -inf or NaN is not
 * chosen (its logit still counts in the softmax over the unmasked).  ids
 * [tokens, topk] gets them, -1 where fewer than topk are left; weights
 * [tokens, topk] (fp32) gets scale * s_j, or with normalize scale * s_j / sum_i
 * s_i over the chosen, where s is the fp32 score of the logit without the bias;
 * 0 for -1 (and for every choice when the chosen scores sum to 0).
 * 1 <= topk <= E. */
int moe_route(const void* logits, int32_t logits_type, int64_t tokens,
              int32_t num_experts, int32_t topk, const float* select_bias,
              int32_t score, int32_t normalize, float scale, int32_t* ids,
              float* weights, void* stream);

/* Gradient of moe_route's weights: dlogits [tokens, E] in the type of the
 * logits, fully written (0 where the gradient is 0, and at masked experts),
 * from dweights [tokens, topk].  The choice itself has no gradient.  ids as
 * moe_route wrote them: an id outside 0 .. E-1 is no choice. */
int moe_route_bwd(const void* logits, int32_t logits_type, int64_t tokens,
                  int32_t num_experts, int32_t topk, const int32_t* ids,
                  const float* dweights, int32_t score, int32_t normalize,
                  float scale, void* dlogits, void* stream);

/* Balance loss of a router, sequence by sequence, with the counts it is made
 * of.  The rows of logits [tokens, E] are cut into num_seqs sequences by
 * seq_ends [num_seqs], device row ends in non-decreasing order (NULL: one
 * sequence of all rows); rows at or past the last end count nowhere.  With
 *     p[t, e]      softmax over the token's unmasked experts, or with
 *                  MOE_SCORE_SIGMOID s_e / sum_i s_i of the sigmoids (0 where
 *                  that sum underflows); masked logits as in moe_route
 *     counts[s, e] pairs of sequence s whose id is e (an id outside 0 .. E-1
 *                  is no choice)
 *     seq_tokens[s] tokens n_s of s with at least one unmasked expert
 *     probs[s, e]  sum of p[t, e] over the tokens of s
 * the loss is
 *     coef / num_seqs * sum_s E / (topk n_s^2) * sum_e counts[s, e] probs[s, e]
 * (0 for a sequence with n_s = 0): coef where all experts get the same.  All
 * four are written; sums are fp32 or wider in a fixed order.  Ends that
 * decrease or leave 0 .. tokens make the loss NaN (nothing outside the buffers
 * is touched; counts, probs and gradients are then of no use).
 * num_seqs <= MOE_MAX_SEQS, tokens times topk <= MOE_MAX_PAIRS.  workspace:
 * moe_balance_workspace(tokens, E, num_seqs) bytes, 4-byte aligned. */
#define MOE_MAX_SEQS 65535
int64_t moe_balance_workspace(int64_t tokens, int32_t num_experts,
                              int32_t num_seqs);
int moe_balance(const void* logits, int32_t logits_type, int64_t tokens,
                int32_t num_experts, int32_t topk, const int32_t* ids,
                int32_t score, const int32_t* seq_ends, int32_t num_seqs,
                float coef, float* loss, int32_t* counts, float* probs,
                int32_t* seq_tokens, void* workspace, int64_t workspace_bytes,
                void* stream);

/* Gradient of moe_balance's loss in the logits, with the counts held constant:
 * dlogits [tokens, E] in the type of the logits, fully written (0 at masked
 * experts and past the last end), times *dloss (device fp32; NULL: 1), plus
 * add [tokens, E] (the type of the logits, may be dlogits itself; NULL: none),
 * rounded once.  counts and seq_tokens as moe_balance wrote them; those of
 * several ranks may be summed first, and the gradient is then that of the loss
 * of all their tokens. */
int moe_balance_bwd(const void* logits, int32_t logits_type, int64_t tokens,
                    int32_t num_experts, int32_t topk, int32_t score,
                    const int32_t* seq_ends, int32_t num_seqs, float coef,
                    const int32_t* counts, const int32_t* seq_tokens,
                    const float* dloss, const void* add, void* dlogits,
                    void* stream);

/* Plan of the packed rows.  ids: [pairs] expert of each pair; an id outside
 * 0 .. E-1 is no choice.  Expert e's group holds its pairs in pair order,
 * padded to a multiple of 128 rows (none if it has no pair).  Writes
 *   offs   [E]          inclusive row ends, the routing the graph-safe calls
 *                       of nvfp4_group.h take as d_offs
 *   counts [E]          pairs of each expert
 *   rows   [pairs]      packed row of each pair, -1 for no choice
 *   src    [m_capacity] pair in each packed row, -1 for padding and for rows
 *                       past the last group
 * If the groups need more than m_capacity rows, NVFP4G_DEV_OVERFLOW is ORed
 * into *d_status, offs and counts still tell the need (the graph-safe calls
 * then refuse offs), and pairs beyond the capacity get row -1.  m_capacity: a
 * multiple of 128, at most NVFP4G_MAX_ROWS.  workspace: at least
 * moe_plan_workspace(pairs, E) bytes, 4-byte aligned (NULL if that is 0). */
int64_t moe_plan_workspace(int64_t pairs, int32_t num_experts);
int moe_plan(const int32_t* ids, int64_t pairs, int32_t num_experts,
             int64_t m_capacity, int32_t* offs, int32_t* counts, int32_t* rows,
             int32_t* src, int32_t* d_status, void* workspace,
             int64_t workspace_bytes, void* stream);

/* Tokens into packed rows: out[rows[p]] = x[t] for every pair p = t*topk + j
 * with 0 <= rows[p] < m_capacity, or weights[p] * x[t] when weights is set
 * (fp32 product, rounded once); the padding rows of the experts' groups (src
 * -1 below offs[E-1]) become 0; other rows are not written.  x [tokens,
 * width] and out [m_capacity, width] are bf16.  rows and src have to be
 * moe_plan's for the same pairs.
 * With y [m_capacity, width] (MOE_F32 or MOE_BF16) and dweights [tokens,
 * topk], also dweights[p] = sum_c x[t, c] * y[rows[p], c] (fp32; 0 where the
 * pair has no row): with x the gradient of moe_combine's output this is the
 * gradient of moe_combine in y (out) and in its weights (dweights).
 * width: a positive multiple of 16, at most NVFP4G_MAX_K; x, y and out are
 * 16-byte aligned (in moe_combine too). */
int moe_dispatch(const uint16_t* x, int64_t tokens, int64_t width,
                 int32_t topk, const int32_t* rows, const int32_t* src,
                 const int32_t* offs, int32_t num_experts, int64_t m_capacity,
                 const float* weights, const void* y, int32_t y_type,
                 uint16_t* out, float* dweights, void* stream);

/* Packed rows back to tokens: out[t] = sum_j weights[p] * y[rows[p]] over the
 * token's pairs that have a row (fp32 sum in the order of j, rounded once to
 * bf16; 0 if there is none); weights NULL: plain sum, which is the gradient
 * of moe_dispatch without weights.  y [m_capacity, width] MOE_F32 or
 * MOE_BF16, out [tokens, width] bf16. */
int moe_combine(const void* y, int32_t y_type, int64_t m_capacity,
                int64_t tokens, int64_t width, int32_t topk,
                const int32_t* rows, const float* weights, uint16_t* out,
                void* stream);

/* Gated feed-forward block of the experts on row-scaled NVFP4 operands: with
 * a the rowwise cast of the packed rows (a_data [sum_m, k/2], a_scale, a_amax
 * [sum_m]) and b the experts' weights, 2f lines of length k each, the f gate
 * lines first (b_data [E, 2f, k/2], b_scale [E, 2f, k/16], b_amax [E*2f]),
 *     g[r, j] = sum_t xa[r, t] * xb_e[j, t],   u[r, j] = ... xb_e[f + j, t],
 *     h[r, j] = act(g) * u,
 * computed as in nvfp4_group_gemm (exact products, fp32 sums), g and u kept
 * in fp32 up to h, which is rounded once to bf16 [sum_m, f].  gu, if not
 * NULL, gets (g, u) rounded to bf16, [sum_m, 2f] with g first, for the
 * backward call.  k: a positive multiple of 128; f: of 16; limits and
 * alignment as in nvfp4_group_gemm, h and gu 16-byte aligned. */
int moe_glu(const uint8_t* a_data, const uint8_t* a_scale, const float* a_amax,
            const uint8_t* b_data, const uint8_t* b_scale, const float* b_amax,
            int64_t sum_m, int64_t f, int64_t k, int32_t num_experts,
            const int64_t* h_splits, int32_t act, uint16_t* h, uint16_t* gu,
            void* stream);

/* Graph-safe form of moe_glu (routing, buffers and status as in
 * nvfp4_group_gemm_graphsafe; rows at or beyond offs[E-1] are neither read
 * nor written). */
int moe_glu_graphsafe(const uint8_t* a_data, const uint8_t* a_scale,
                      const float* a_amax, const uint8_t* b_data,
                      const uint8_t* b_scale, const float* b_amax,
                      int64_t m_capacity, int64_t f, int64_t k,
                      int32_t num_experts, const int32_t* d_offs, int32_t act,
                      uint16_t* h, uint16_t* gu, int32_t* d_status,
                      void* stream);

/* Backward pass of the gated block through the down projection: with a the
 * rowwise cast of the gradient of the block's output (lines of length k, the
 * hidden size) and b the down projection's weights as f lines of length k per
 * expert (the columnwise cast of each [k, f] weight; b_data [E, f, k/2]),
 *     dh[r, j] = sum_t xa[r, t] * xb_e[j, t],
 *     dgu[r, j] = dh * u * act'(g),   dgu[r, f + j] = dh * act(g),
 * with (g, u) read from gu [sum_m, 2f] (bf16) and dh kept in fp32; dgu is
 * bf16 [sum_m, 2f].  The gradients of the inputs and weights of the gate and
 * up projections are then nvfp4_group_gemm and nvfp4_group_gemm_wgrad on the
 * casts of dgu.  Sizes, limits and alignment as in moe_glu. */
int moe_glu_bwd(const uint8_t* a_data, const uint8_t* a_scale,
                const float* a_amax, const uint8_t* b_data,
                const uint8_t* b_scale, const float* b_amax, int64_t sum_m,
                int64_t f, int64_t k, int32_t num_experts,
                const int64_t* h_splits, const uint16_t* gu, int32_t act,
                uint16_t* dgu, void* stream);

/* Graph-safe form of moe_glu_bwd. */
int moe_glu_bwd_graphsafe(const uint8_t* a_data, const uint8_t* a_scale,
                          const float* a_amax, const uint8_t* b_data,
                          const uint8_t* b_scale, const float* b_amax,
                          int64_t m_capacity, int64_t f, int64_t k,
                          int32_t num_experts, const int32_t* d_offs,
                          const uint16_t* gu, int32_t act, uint16_t* dgu,
                          int32_t* d_status, void* stream);

/* The gated block with its checkpoint in 8 bits: moe_glu, with g and u kept
 * for the backward call as whole numbers of a scale that 32 columns of a row
 * share (16 where f ends inside a group):
 *     S = bf16(max |v| / 127),   code = the whole number nearest to v / S
 * (both quotients rounded to fp32; ties to even), value code * S, off by at
 * most S / 2 (and the quotient's rounding).  A group whose
 * largest magnitude is below 2^-112 is kept as zeros, one with a value that is
 * not finite as S = NaN and codes 0.  gu8 [sum_m, 2f] with g first; gu_scale
 * [2 * ceil(f / 32), sum_m], the groups of g first (m_capacity in place of
 * sum_m in the graph-safe form): 1.06 bytes a value in place of 2.  h is
 * moe_glu's, from the values before they are kept.  gu8 16-byte, gu_scale 4-byte
 * aligned. */
#define MOE_KEEP8_GROUP 32
int moe_glu_keep8(const uint8_t* a_data, const uint8_t* a_scale,
                  const float* a_amax, const uint8_t* b_data,
                  const uint8_t* b_scale, const float* b_amax, int64_t sum_m,
                  int64_t f, int64_t k, int32_t num_experts,
                  const int64_t* h_splits, int32_t act, uint16_t* h,
                  int8_t* gu8, uint16_t* gu_scale, void* stream);
int moe_glu_keep8_graphsafe(const uint8_t* a_data, const uint8_t* a_scale,
                            const float* a_amax, const uint8_t* b_data,
                            const uint8_t* b_scale, const float* b_amax,
                            int64_t m_capacity, int64_t f, int64_t k,
                            int32_t num_experts, const int32_t* d_offs,
                            int32_t act, uint16_t* h, int8_t* gu8,
                            uint16_t* gu_scale, int32_t* d_status,
                            void* stream);

/* moe_glu_bwd on the values that moe_glu_keep8 kept.  h [sum_m, f] bf16, if
 * not NULL, gets act(g) * u of the kept values, for the weight gradient of the
 * down projection: the forward pass's h need not be kept then. */
int moe_glu_bwd_keep8(const uint8_t* a_data, const uint8_t* a_scale,
                      const float* a_amax, const uint8_t* b_data,
                      const uint8_t* b_scale, const float* b_amax,
                      int64_t sum_m, int64_t f, int64_t k, int32_t num_experts,
                      const int64_t* h_splits, const int8_t* gu8,
                      const uint16_t* gu_scale, int32_t act, uint16_t* dgu,
                      uint16_t* h, void* stream);
int moe_glu_bwd_keep8_graphsafe(const uint8_t* a_data, const uint8_t* a_scale,
                                const float* a_amax, const uint8_t* b_data,
                                const uint8_t* b_scale, const float* b_amax,
                                int64_t m_capacity, int64_t f, int64_t k,
                                int32_t num_experts, const int32_t* d_offs,
                                const int8_t* gu8, const uint16_t* gu_scale,
                                int32_t act, uint16_t* dgu, uint16_t* h,
                                int32_t* d_status, void* stream);

/* Single-token form of the gated block: bf16 tokens, NVFP4 weights, no
 * packed groups.  For every pair p of token t with expert e = ids[p],
 *     h[p, j] = act(sum_c x[t, c] xb_e[j, c]) * (sum_c x[t, c] xb_e[f+j, c])
 * with x [tokens, k] bf16 unquantised, b as in moe_glu, h [pairs, f] bf16;
 * an id outside 0 .. E-1 gives a row of zeros.  Each chosen expert's weights
 * are read once for up to 16 pairs that share it (32 or 64 where the pairs are
 * that many an expert; for each pair of a lone token).  Meant for decoding: pairs
 * <= MOE_MAX_TOKEN_PAIRS.  k: a positive multiple of 32, f of 16; alignment
 * of b as in nvfp4_group_gemm, x and h 16-byte aligned. */
#define MOE_MAX_TOKEN_PAIRS 1024
int moe_token_glu(const uint16_t* x, int64_t tokens, int64_t k, int32_t topk,
                  const int32_t* ids, const uint8_t* b_data,
                  const uint8_t* b_scale, const float* b_amax, int64_t f,
                  int32_t num_experts, int32_t act, uint16_t* h, void* stream);

/* Single-token down projection: out[p, j] = sum_c x[p, c] xb_e[j, c] for
 * every pair p with expert e = ids[p]; x [pairs, k] bf16, b_data [E, n, k/2]
 * as in nvfp4_group_gemm, out fp32 [pairs, n]; rows of zeros for pairs
 * without an expert.  moe_combine with rows[p] = p joins the pairs of a
 * token.  k: a positive multiple of 32, n of 16; alignment as in
 * moe_token_glu, out 16-byte aligned. */
int moe_token_linear(const uint16_t* x, int64_t pairs, int64_t k,
                     const int32_t* ids, const uint8_t* b_data,
                     const uint8_t* b_scale, const float* b_amax, int64_t n,
                     int32_t num_experts, float* out, void* stream);

/* Low-rank adapters of many requests beside one shared projection:
 *     y[t, j] = sum_c x[t, c] xw[j, c]
 *               + alpha[a] * sum_r B_a[j, r] * (sum_c A_a[r, c] x[t, c]),
 * a = adapter_ids[t]; an id outside 0 .. num_adapters-1 is no adapter (the
 * projection alone).  x [tokens, k] bf16; the projection in NVFP4, n lines
 * (w_data [n, k/2], w_scale [n, k/16], w_amax [n]); lora_a [num_adapters,
 * rank, k] and lora_b [num_adapters, n, rank] bf16, alpha [num_adapters]
 * fp32; y [tokens, n] bf16, rounded once from fp32.  The inner product A_a x
 * is kept in fp32 between the two steps.  adapter_ids may be in any order.  k: a
 * positive multiple of 32 up to NVFP4G_MAX_K, n of 16 up to 2^20, rank of 8 up
 * to LORA_MAX_RANK; tokens up to NVFP4G_MAX_ROWS; num_adapters 0 (with NULL
 * lora_a, lora_b, alpha, adapter_ids) is the projection alone.
 * x, w_data, lora_a, lora_b and y are 16-byte aligned, the others 4-byte.
 * workspace: lora_workspace(tokens, k, n, rank) bytes, 16-byte aligned, which
 * also serve every call with the same k and n, up to as many tokens and up to
 * that rank (or no adapters: rank 0).  It is at most 32 MiB or, if that is
 * more, 6 bytes a token and rank (rounded up to 16) and 4 a token, in multiples
 * of 256 bytes. */
#define LORA_MAX_RANK 128
int64_t lora_workspace(int64_t tokens, int64_t k, int64_t n, int32_t rank);
int lora_linear(const uint16_t* x, int64_t tokens, int64_t k,
                const uint8_t* w_data, const uint8_t* w_scale,
                const float* w_amax, int64_t n, const uint16_t* lora_a,
                const uint16_t* lora_b, const float* alpha,
                int32_t num_adapters, int32_t rank, const int32_t* adapter_ids,
                uint16_t* y, void* workspace, int64_t workspace_bytes,
                void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_OPS_H_ */
