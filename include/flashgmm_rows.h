/*
 * flashgmm_rows.h - C ABI of the row operators for AMD Instinct MI355X
 * (gfx950): rows held in 4 or 8 bits, their products, draws from rows of
 * logits, and losses over such rows with their gradients.
 *
 * They serve what the mixture library (flashgmm.h) leaves a user with: many
 * stored vectors (base rows, component means) that are scored against other
 * rows, and rows of logits from which a component is picked.  gmm_soft_assign
 * picks the likeliest component and further ones above a threshold; gmm_draw
 * picks one at random by its responsibility.  The losses train a model of the
 * components (one that gives a point's logits without the mixture's E-step):
 * gmm_distill on the largest of the mixture's log-densities, gmm_balance on how
 * evenly the components are taken.
 *
 * Conventions: as in flashgmm.h, and
 *   - no context: every call works on the current device, on the given HIP
 *     stream (NULL = the null stream), allocates nothing, synchronises
 *     nothing and keeps nothing; it can be captured into a HIP graph.  Calls
 *     on different streams or from different host threads are independent as
 *     long as they share no output and no workspace;
 *   - every pointer is a device pointer; outputs must not overlap inputs;
 *   - zero rows are allowed and launch nothing;
 *   - gmm_last_error(NULL) returns the message of a failed call.
 */
#ifndef FLASHGMM_ROWS_H
#define FLASHGMM_ROWS_H

#include "flashgmm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of rows. */
typedef enum {
    GMM_TYPE_FLOAT = 0,    /* float32 */
    GMM_TYPE_BFLOAT = 1,   /* bfloat16 */
    GMM_TYPE_HALF = 2,     /* float16 */
    GMM_TYPE_MX = 3,       /* 4-bit codes and block scales (below) */
    GMM_TYPE_BYTE = 4      /* 8-bit codes and block scales (below) */
} gmm_type;

/* Rows in 4 bits: the microscaling format MXFP4 of the OCP Microscaling
 * Formats specification, version 1.0 (elements E2M1, scales E8M0, blocks of
 * 32 consecutive values of a row).
 *   value = (-1)^sign * {0, .5, 1, 1.5, 2, 3, 4, 6}[code & 7] * 2^(scale - 127)
 * Layout: a row of D values is padded to G = ceil(D / 128) groups of 128.
 * codes: 64 G bytes a row, element d in byte d / 2, the even one in the low
 * half; scales: 4 G bytes a row, one for each 32 values; padding has code 0
 * and scale 0.  Row strides are in bytes: ld_codes >= 64 G and a multiple of
 * 16, ld_scales >= 4 G and a multiple of 4, both at most 2^23; codes 16-byte
 * and scales 4-byte aligned.  1 <= D <= 2^20, at most 2^30 rows. */

/* Quantisation: for each block of 32 values, with m their largest magnitude,
 *   e = max(floor(log2 m) - 2, -127), scale = e + 127 (0 for a block of zeros),
 *   code = x / 2^e rounded to the nearest of the grid (ties to the even code),
 *          magnitudes above 6 to 6; the sign is kept, also of zeros.
 * A block that holds a NaN or an infinity gets scale 255 and codes 0: it
 * stands for NaN throughout.  X has row stride ldx (elements, >= D). */
gmm_status gmm_mx_quantize(const void *X, int32_t type, int64_t N, int32_t D, int64_t ldx,
                           uint8_t *codes, int64_t ld_codes, uint8_t *scales, int64_t ld_scales,
                           void *hip_stream);

/* The values that 4-bit rows stand for, rounded once to the type of X (exact
 * in float32 and bfloat16). */
gmm_status gmm_mx_dequantize(const uint8_t *codes, int64_t ld_codes, const uint8_t *scales, int64_t ld_scales,
                             int64_t N, int32_t D, void *X, int32_t type, int64_t ldx, void *hip_stream);

/* Products of rows: C[m, n] = sum_d A[m, d] B[n, d] + bias[n], B in 4 bits.
 * a_type GMM_TYPE_MX: A points to codes with row stride lda bytes, a_scales
 * and ld_a_scales to their scales.  Other a_type: A holds rows of that type
 * with row stride lda elements, which are quantised as by gmm_mx_quantize on
 * the way (a_scales is ignored), so the results are the same.
 * Products are summed in float32.  Each is exact where it lies within
 * float32's range (at most 4 bits of significand): one below 2^-149 counts to
 * within 2^-149; where the magnitudes of a result's products sum past the
 * range, the result may be infinite or NaN.  bias (float32[N]) may be NULL;
 * each result is rounded once to c_type (float, bfloat16 or half).  ldc in
 * elements, >= N.  A block of scale 255 makes its row's results NaN.
 * workspace: gmm_mx_product_workspace bytes, 16-byte aligned, used by this
 * call alone until it completes; NULL where that is 0. */
size_t gmm_mx_product_workspace(int32_t a_type, int64_t M, int64_t N, int32_t D);
gmm_status gmm_mx_product(const void *A, int32_t a_type, int64_t lda, const uint8_t *a_scales, int64_t ld_a_scales,
                          int64_t M, const uint8_t *b_codes, int64_t ldb, const uint8_t *b_scales,
                          int64_t ld_b_scales, int64_t N, int32_t D, const float *bias,
                          void *C, int32_t c_type, int64_t ldc, void *workspace, size_t workspace_bytes,
                          void *hip_stream);

/* Rows in 8 bits: E4M3 elements (OCP 8-bit Floating Point Specification 1.0:
 * 1 sign, 4 exponent and 3 fraction bits, largest value 448, no infinities)
 * and one power of two for each block of 128 consecutive values of a row.
 *   value = e4m3(code) * 2^(scale - 127)
 * Layout: a row of D values is padded to G = ceil(D / 128) groups of 128.
 * codes: 128 G bytes a row; scales: 4 ceil(G / 4) bytes a row, the first G one
 * for each group; padding has code 0 and scale 0.  Row strides are in bytes:
 * ld_codes >= 128 G and a multiple of 16, ld_scales >= 4 ceil(G / 4) and a
 * multiple of 4, both at most 2^23; codes 16-byte and scales 4-byte aligned.
 * 1 <= D <= 2^20, at most 2^30 rows. */

/* Quantisation: for each block, with m its largest magnitude,
 *   e = max(ceil(log2(m / 448)), -127), scale = e + 127 (0 for a block of zeros),
 *   code = x / 2^e rounded to the nearest E4M3 value (ties to the even code);
 * the sign is kept, also of zeros.  No value is above 448 2^e.  A block that
 * holds a NaN or an infinity gets scale 255 and codes 0: it stands for NaN
 * throughout.  X has row stride ldx (elements, >= D). */
gmm_status gmm_byte_quantize(const void *X, int32_t type, int64_t N, int32_t D, int64_t ldx,
                             uint8_t *codes, int64_t ld_codes, uint8_t *scales, int64_t ld_scales,
                             void *hip_stream);

/* The values that 8-bit rows stand for, rounded once to the type of X (exact
 * in float32, and in bfloat16 from 2^-130 on). */
gmm_status gmm_byte_dequantize(const uint8_t *codes, int64_t ld_codes, const uint8_t *scales, int64_t ld_scales,
                               int64_t N, int32_t D, void *X, int32_t type, int64_t ldx, void *hip_stream);

/* Products of rows: C[m, n] = sum_d A[m, d] B[n, d] + bias[n], B in 8 bits, as
 * gmm_mx_product: a_type GMM_TYPE_BYTE takes A's codes and scales, any other
 * rows of that type, quantised as by gmm_byte_quantize on the way (the results
 * are the same).  Products are summed in float32.  With float32 and float16
 * results each is exact where it lies within float32's range; a value of A or B
 * below 2^-130 counts to within 2^-134, one of 2^128 or more (the largest float32
 * numbers are rounded there) as infinite.  With bfloat16 results a product may also
 * lose what lies below 2^-13 of the largest among the 8 products of its place
 * (d / 8): 1.4e-5 of the results of normal operands, more of those that are small
 * against their products, before the rounding to 16 bits.
 * Where the magnitudes of a result's products sum past float32's range, the
 * result may be infinite or NaN.  A block of scale 255 makes its
 * row's results NaN.  workspace: gmm_byte_product_workspace bytes, otherwise as
 * gmm_mx_product. */
size_t gmm_byte_product_workspace(int32_t a_type, int64_t M, int64_t N, int32_t D);
gmm_status gmm_byte_product(const void *A, int32_t a_type, int64_t lda, const uint8_t *a_scales,
                            int64_t ld_a_scales, int64_t M, const uint8_t *b_codes, int64_t ldb,
                            const uint8_t *b_scales, int64_t ld_b_scales, int64_t N, int32_t D, const float *bias,
                            void *C, int32_t c_type, int64_t ldc, void *workspace, size_t workspace_bytes,
                            void *hip_stream);

/* Draws: ids[n] is a component of row n of the logits (N x V, row stride ld
 * elements), drawn with the random number u[n] in [0, 1).  With z_i the row's
 * logits and T its temperature,
 *   w_i = exp((z_i - max z) / T),
 * ranked by z descending, then index ascending, component i stays if
 *   its rank is below top_k                            (top_k >= 1),
 *   the weights ranked before it sum to less than top_p times the sum over
 *   the top_k that stayed; the first always stays      (top_p < 1),
 *   w_i >= min(min_p, 1)                               (min_p > 0),
 * and ids[n] is the first index at which the running sum, in index order, of
 * the weights that stay exceeds u[n] times their sum (u below 0 counts as 0;
 * at or above 1, or NaN, the last index with weight is taken).
 * T that is not above 0 takes the largest logit, lowest index on ties.  top_k
 * below 1, top_p not below 1 and min_p not above 0 are off.
 * A logit of -inf has no weight.  A row that holds a NaN or +inf, or nothing
 * but -inf, has no distribution: ids[n] = -1.
 * Each setting is a device array of N values or, where that is NULL, one
 * value for all rows.  Weights are whole multiples of 2^-42 of the largest,
 * each within 1.2 * 2^-43 (of the largest) of its value, so those below 2^-43
 * are zero, and a sum of n of them is within n times that.  They are summed as
 * integers, so results do not depend on the order of the sums.
 * 1 <= V <= 2^20, N <= 2^30.  workspace as gmm_mx_product. */
size_t gmm_draw_workspace(int64_t N, int32_t V);
gmm_status gmm_draw(const void *logits, int32_t type, int64_t N, int32_t V, int64_t ld, const float *u,
                    const float *temperatures, float temperature, const int32_t *top_ks, int32_t top_k,
                    const float *top_ps, float top_p, const float *min_ps, float min_p,
                    int32_t *ids, void *workspace, size_t workspace_bytes, void *hip_stream);

/* Distillation from a teacher's top logits.  Row n of the logits (N x V, row
 * stride ld elements) is the model's, ids[n, 0 .. k) the components that the
 * teacher lists for it and teacher[n, 0 .. k) their logits (ids of id_bits 32 or
 * 64, row stride ld_ids elements; teacher of any row type, row stride
 * ld_teacher).  With T the temperature,
 *   q = softmax(logits[n] / T) over all V, p = softmax(teacher[n] / T) over the
 *   listed places: those with an id >= 0 and a teacher's logit above -inf,
 *   losses[n] = T^2 sum_j p_j (log p_j - log q_ids[n, j]),
 *   gradient  = w_n T (q_v - sum of the p_j with ids[n, j] = v),
 * w_n the weight of the row's loss.  An id may be listed several times.  A row
 * that lists nothing has loss 0 and gradient 0, whatever its logits.  A row with
 * an id of V or more, a listed logit that is NaN or +inf, a NaN or +inf among
 * its own logits, or nothing above -inf there has loss and gradient NaN; a
 * listed component whose own logit is -inf gives loss +inf (and the gradient
 * above) where its p_j is not 0 in float32.
 * gmm_distill writes losses (float[N]); stats (float[2 N], may be NULL) for
 * gmm_distill_backward; and the gradient in the type of the logits (row stride
 * ld_grad), rounded once, where grad is not NULL, with the row weights given
 * (weights, float[N], or weight for all where that is NULL).
 * gmm_distill_backward writes the gradient from the stats of a call on the same
 * inputs; weights[n * ld_weights] (ld_weights >= 0) is the weight of row n.
 * grad must overlap nothing else.  2^-60 <= temperature <= 2^60, 1 <= V <= 2^20,
 * N <= 2^30, 1 <= k <= 1024.  workspace: gmm_distill_workspace bytes, as
 * gmm_mx_product; the backward needs none. */
size_t gmm_distill_workspace(int64_t N, int32_t V, int32_t k);
gmm_status gmm_distill(const void *logits, int32_t type, int64_t N, int32_t V, int64_t ld, const void *ids,
                       int32_t id_bits, int64_t ld_ids, const void *teacher, int32_t teacher_type,
                       int64_t ld_teacher, int32_t k, float temperature, float *losses, float *stats,
                       const float *weights, float weight, void *grad, int64_t ld_grad,
                       void *workspace, size_t workspace_bytes, void *hip_stream);
gmm_status gmm_distill_backward(const void *logits, int32_t type, int64_t N, int32_t V, int64_t ld, const void *ids,
                                int32_t id_bits, int64_t ld_ids, const void *teacher, int32_t teacher_type,
                                int64_t ld_teacher, int32_t k, float temperature, const float *stats,
                                const float *weights, int64_t ld_weights, void *grad, int64_t ld_grad,
                                void *hip_stream);

/* Balance of components and their counts.  ids[n, 0 .. k) are the components
 * that row n takes (as gmm_draw gives them, or a top-k; negative: none).  With
 * c_e the number of ids that are e, C their sum, R the rows with an id >= 0 and
 * p_n = softmax(logits[n]),
 *   counts[e] = c_e,
 *   loss     = K / (C R) sum over those rows of d_n, d_n = sum_e c_e p_ne
 *            = K sum_e (c_e / C) (mean of p_ne), 1 where all is even,
 *   gradient = w K / (C R) p_ne (c_e - d_n), 0 for the other rows, whatever
 *              their logits and w.
 * The counts are constants of the gradient.  Without any id the loss is 0.  An
 * id of K or more makes the loss and the whole gradient NaN, that of the other
 * rows as well (it is in no count); a row that is counted and holds a NaN or +inf, or nothing above -inf,
 * makes the loss and its own gradient NaN.
 * gmm_balance writes counts (int64[K]), loss (float[1]), stats
 * (gmm_balance_stats floats, for gmm_balance_backward) and, where grad is not
 * NULL, the gradient for weight w, in the type of the logits and rounded once.
 * gmm_balance_backward writes the gradient from those stats, w = *weight (on
 * the device).  Nothing may overlap grad.  1 <= K <= 2^20, N <= 2^30,
 * 1 <= k <= 1024.  With N = 0 counts and loss are written, as zeros. */
size_t gmm_balance_stats(int64_t N, int32_t K);
size_t gmm_balance_workspace(int64_t N, int32_t K, int32_t k);
gmm_status gmm_balance(const void *logits, int32_t type, int64_t N, int32_t K, int64_t ld, const void *ids,
                       int32_t id_bits, int64_t ld_ids, int32_t k, int64_t *counts, float *loss, float *stats,
                       float weight, void *grad, int64_t ld_grad,
                       void *workspace, size_t workspace_bytes, void *hip_stream);
gmm_status gmm_balance_backward(const void *logits, int32_t type, int64_t N, int32_t K, int64_t ld,
                                const float *stats, const float *weight, void *grad, int64_t ld_grad,
                                void *hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* FLASHGMM_ROWS_H */
