/*
 * w4a16_routed.h -- C ABI of the operators of libw4a16.so in which every row
 * of a batch meets weights of its own: routing to experts, the experts'
 * products over int4 weights, and low-rank adapters beside a shared int4
 * projection.  Conventions, status codes and flags are those of w4a16.h
 * (the caller owns every buffer, arguments checked on the host before any
 * launch, work enqueued on `stream`; X, weights in the device layout, A, B, Y
 * and workspaces 16-byte aligned, while logits, bias, ids, routing weights
 * and adapter scales only need their element's alignment, so that they can be
 * rows of a larger tensor).
 *
 * Whole numbers that live on the device (expert ids, adapter ids) cannot be
 * checked on the host: an id outside its range selects nothing.
 */
#ifndef W4A16_ROUTED_H
#define W4A16_ROUTED_H

#include "w4a16.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- routing to experts ------------------------------------------------- */
/* Element type of the logits. */
#define W4A16_LOGITS_F16  0
#define W4A16_LOGITS_BF16 1
#define W4A16_LOGITS_F32  2

/* flags of w4a16_route */
#define W4A16_ROUTE_SIGMOID     0x1u /* scores sigmoid(logit); else softmax over the row */
#define W4A16_ROUTE_RENORMALIZE 0x2u /* divide the chosen scores by their sum */

/* Chooses k of E experts for each of T rows of logits [T][E].
 *   score  s = softmax over the row, or sigmoid;
 *   key    s + bias[e] (bias fp32 [E], or NULL): decides, but does not weigh;
 *   groups n_groups groups of E / n_groups consecutive experts; a group's
 *          value is the sum of its group_top (1 or 2) best keys, and only the
 *          topk_groups groups of the largest values stay;
 *   ids    int32 [T][k]: the experts of the k largest keys left, largest
 *          first; of equal keys (and equal groups) the lowest index;
 *   weights fp32 [T][k]: their scores, divided by their sum with
 *          W4A16_ROUTE_RENORMALIZE (a sum of 0 gives 0), times scale.  They are
 *          formed in 64 bits: a sigmoid of a logit of -700 still weighs, one
 *          below -745 is 0.
 * A NaN logit counts as -infinity, +infinity as the largest float.  An expert
 * with a logit of -infinity, or a bias of -infinity or NaN, is never chosen
 * (and adds nothing to its group's value): a slot that no expert is left for
 * gets id -1 and weight 0.
 * Limits: 1 <= E <= 1024, 1 <= n_groups <= 64, E % n_groups == 0,
 * 1 <= k <= 32, k <= topk_groups * (E / n_groups), T <= 2^24.
 * Errors: W4A16_ERR_NULL, W4A16_ERR_SHAPE (limits, dtype, group_top, a scale
 * that is not finite), W4A16_ERR_FLAGS, W4A16_ERR_ALIGN. */
int32_t w4a16_route(const void *logits, int32_t logits_dtype, int64_t T, int64_t E,
                    const float *bias, int32_t k, int32_t n_groups, int32_t topk_groups,
                    int32_t group_top, float scale, uint32_t flags, int32_t *ids, float *weights,
                    void *stream);
int32_t w4a16_check_route_args(const void *logits, int32_t logits_dtype, int64_t T, int64_t E,
                               const float *bias, int32_t k, int32_t n_groups,
                               int32_t topk_groups, int32_t group_top, float scale,
                               uint32_t flags, const int32_t *ids, const float *weights);

/* ---- the experts' products ---------------------------------------------- */
/* The weights of E experts in the device layout: every expert's weight is a
 * w4a16_repack result of its own, one after the other (q, s and z each one
 * buffer of E times w4a16_repack_size's bytes).  A gated weight holds two
 * [I][K] matrices for each expert, gate then up, each a repack result.
 *
 * For every row t of X [T][K] and slot j < k with e = ids[t][j]:
 *   h = silu(X[t] . Wgate_e^T) * (X[t] . Wup_e^T),   silu(v) = v / (1 + exp(-v))
 *   Y[t] = sum over j of weights[t][j] * (h . Wdown_e^T)
 * with W = RNE((q - z) * s) in the 16-bit type, as w4a16_dequant has it.  All
 * sums are fp32; h is rounded to the 16-bit type between the products (it
 * feeds 16-bit matrix instructions), Y once.  An h beyond fp16's range enters
 * the second product in 32 bits instead: a row that has one takes a path of
 * plain fp32 sums, which is slow.  A slot whose id lies outside
 * 0..E-1 adds nothing; a row with no other slot is 0.  A row may name an
 * expert twice.
 *   gate_up  gated, [E][2][I][K];   down [E][D][I];   Y [T][D].
 *   flags    W4A16_SYMMETRIC, W4A16_PARTIAL_LAST_GROUP, W4A16_BF16, for both
 *            weights.
 * workspace: w4a16_experts_workspace_size bytes (no fill needed); calls that
 * may run at the same time need separate ones.
 * Limits: 1 <= E <= 1024, 1 <= k <= 32, T <= 2^20, T * k <= 2^22, X below
 * 2 GiB, each expert's 2 I K and D I below 2^32 elements, I and D below
 * 2^22; W4A16_BF16: scales below 2^124 in magnitude (z s is formed in fp32).
 * Errors: W4A16_ERR_NULL, W4A16_ERR_SHAPE (also where Y overlaps X, ids or
 * weights), W4A16_ERR_GROUP, W4A16_ERR_FLAGS, W4A16_ERR_ALIGN,
 * W4A16_ERR_WORKSPACE, W4A16_ERR_ARCH, W4A16_ERR_HIP. */
int32_t w4a16_experts_workspace_size(int64_t T, int32_t k, int64_t K, int64_t I, int64_t D,
                                     int64_t E, int32_t g, uint32_t flags, size_t *bytes);
int32_t w4a16_experts(const uint16_t *X, int64_t T, int64_t K, const int32_t *ids,
                      const float *weights, int32_t k, int64_t E, const void *gate_up_q,
                      const void *gate_up_s, const void *gate_up_z, int64_t I,
                      const void *down_q, const void *down_s, const void *down_z, int64_t D,
                      int32_t g, uint32_t flags, uint16_t *Y, void *workspace,
                      size_t workspace_bytes, void *stream);
int32_t w4a16_check_experts_args(const uint16_t *X, int64_t T, int64_t K, const int32_t *ids,
                                 const float *weights, int32_t k, int64_t E,
                                 const void *gate_up_q, const void *gate_up_s,
                                 const void *gate_up_z, int64_t I, const void *down_q,
                                 const void *down_s, const void *down_z, int64_t D, int32_t g,
                                 uint32_t flags, const uint16_t *Y, const void *workspace,
                                 size_t workspace_bytes);

/* ---- low-rank adapters beside a shared projection ------------------------ */
#define W4A16_LORA_MAX_PARTS 8

/* w4a16_gemm with one of n adapters added to each row:
 *   Y[m] = X[m] . W^T + scales[a] * (X[m] . A_a^T) . B_a^T,   a = adapter_ids[m]
 * in which a row whose id lies outside 0..n-1 has no adapter.  The columns of
 * Y are cut into n_parts parts of part_sizes[p] columns (fused projections:
 * q, k and v); part p uses rows p r .. (p+1) r - 1 of A_a.
 *   A       16-bit [n][n_parts * r][K];   B 16-bit [n][N][r];
 *   scales  fp32 [n];   adapter_ids int32 [M].
 * All sums are fp32; the low-rank values scales[a] X . A_a^T enter the second
 * product as pairs of 16-bit values (16 bits of each in bf16, 22 of the row's
 * largest in fp16, whatever their range), and Y is rounded once.  part_sizes is read on the host during the call.
 * workspace: w4a16_gemm_lora_workspace_size bytes (no fill needed); calls
 * that may run at the same time need separate ones.
 * Limits: those of w4a16_gemm, n <= 65536, r a multiple of 8 up to 256,
 * n_parts <= W4A16_LORA_MAX_PARTS, part sizes positive with sum N, one
 * adapter's A below 2 GiB.
 * Errors: as w4a16_gemm (Y must not overlap adapter_ids either). */
int32_t w4a16_gemm_lora_workspace_size(int64_t M, int64_t N, int64_t K, int32_t g,
                                       uint32_t flags, int32_t n_parts, int32_t r,
                                       size_t *bytes);
int32_t w4a16_gemm_lora(const uint16_t *X, int64_t M, int64_t K, const void *q_dev,
                        const void *s_dev, const void *z_dev, int64_t N, int32_t g,
                        uint32_t flags, const uint16_t *A, const uint16_t *B,
                        const float *scales, int64_t n, int32_t r, int32_t n_parts,
                        const int64_t *part_sizes, const int32_t *adapter_ids, uint16_t *Y,
                        void *workspace, size_t workspace_bytes, void *stream);
int32_t w4a16_check_gemm_lora_args(const uint16_t *X, int64_t M, int64_t K, const void *q_dev,
                                   const void *s_dev, const void *z_dev, int64_t N, int32_t g,
                                   uint32_t flags, const uint16_t *A, const uint16_t *B,
                                   const float *scales, int64_t n, int32_t r, int32_t n_parts,
                                   const int64_t *part_sizes, const int32_t *adapter_ids,
                                   const uint16_t *Y, const void *workspace,
                                   size_t workspace_bytes);

#ifdef __cplusplus
}
#endif
#endif /* W4A16_ROUTED_H */
