/*
 * flashgmm_rows.h - C ABI of the row operators for AMD Instinct MI355X
 * (gfx950): rows held in 4 bits, their products, and draws from rows of
 * logits.
 *
 * They serve what the mixture library (flashgmm.h) leaves a user with: many
 * stored vectors (base rows, component means) that are scored against other
 * rows, and rows of logits from which a component is picked.  gmm_soft_assign
 * picks the likeliest component and further ones above a threshold; gmm_draw
 * picks one at random by its responsibility.
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
    GMM_TYPE_MX = 3        /* 4-bit codes and block scales (below) */
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

#ifdef __cplusplus
}
#endif

#endif /* FLASHGMM_ROWS_H */
