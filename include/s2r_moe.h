/* s2r_moe.h -- a layer of experts, exported by libs2r.so (gfx950): tokens sorted by expert and back
 * with their weights, the gradients of both, and the experts' products and weight gradients in 8
 * bits, beside the linear layer of s2r_q8.h.  The weight gradients of experts that no token chose are
 * zeros, which s2r_topk_ef and s2r_encode leave out.
 *
 *   s2r_moe_route          which row every choice gets, and which rows every expert has
 *   s2r_moe_gather         tokens to their choices' rows, as they are or in 8 bits
 *   s2r_moe_combine        rows back to their tokens, weighted and added; without weights the
 *                          gradient of s2r_moe_gather
 *   s2r_moe_combine_grad   the gradients of s2r_moe_combine's rows (also in 8 bits) and weights
 *   s2r_q8_gemm_experts    every expert's rows times that expert's matrix
 *   s2r_q8_wgrad_experts   every expert's weight gradient from its rows
 *
 * Rows.  Each of T tokens makes K choices among E experts: expert [T][K] int32, dense; anything
 * outside 0 .. E - 1 (such as -1) is no choice.  A token may choose an expert twice.  A sorted matrix
 * has a row for every choice: those of an expert lie together, in the order of (token, choice),
 * from row first[e] on, rows[e] of them.  first[e] is a multiple of 4 and the experts follow each other,
 *   first[0] = 0, first[e + 1] = first[e] + rows[e] rounded up to a multiple of 4,
 * so that s2r_moe_rows(T, K, E) rows are always enough.  place [T][K] is the row of each choice, or
 * -1.  Rows that no choice has are neither read nor written by any of these calls; other calls may
 * run over them, whatever they hold.
 * The calls that take place, or first and rows, take them from device memory, so nothing waits for
 * the host.  They also take those of other programs: place may hold any rows, each at most once, and an
 * expert's rows may begin at any multiple of 4, as long as no two experts share a row.  What lies outside the
 * R (or M) rows of the matrices counts as no row.
 *
 * Conventions are those of s2r.h and s2r_q8.h: descriptors, alignment, sizes, padding, sums in
 * fp32 in an order that the sizes and rows fix, and errors.  Beyond them:
 *   - E is 1 .. 1024 and K 1 .. 64, T * K below 2^27 (S2R_ERR_DIM otherwise).
 *   - first, rows, expert, place, weight and dweight are 4-byte aligned.
 *   - Steps from one expert to the next reach no further than 64 bits of bytes (S2R_ERR_DIM otherwise).
 */
#ifndef S2R_MOE_H
#define S2R_MOE_H

#include "s2r_q8.h"

#ifdef __cplusplus
extern "C" {
#endif

#define S2R_MAX_EXPERTS 1024
#define S2R_MAX_CHOICES 64

/* The rows of E experts (device memory; the struct is copied at call time). */
typedef struct {
  const uint32_t* first; /* [experts] */
  const uint32_t* rows;  /* [experts] */
  uint32_t experts;
} s2r_experts;

/* Rows that always hold the choices of T tokens: T K + 3 min(E, T K), down to a multiple of 4.
 * 0 for sizes that s2r_moe_route refuses. */
uint64_t s2r_moe_rows(uint64_t T, uint32_t K, uint32_t E);

/* Bytes of workspace that s2r_moe_route needs (0: none). */
size_t s2r_moe_route_workspace_bytes(uint64_t T, uint32_t K, uint32_t E);

/* expert [T][K] -> first [E], rows [E], place [T][K].  workspace: 16-byte aligned, contents on entry
 * do not matter. */
s2r_status s2r_moe_route(uint64_t T, uint32_t K, uint32_t E, const int32_t* expert,
                         uint32_t* first, uint32_t* rows, int32_t* place, void* workspace,
                         size_t ws_bytes, void* stream);

/* x [T][D] -> row place[t][k] of out [R][D] (of x's dtype) and of outq [R][D] (row blocks, as
 * s2r_q8_save stores them).  Either may be NULL, not both. */
s2r_status s2r_moe_gather(uint64_t T, uint32_t K, uint64_t D, const s2r_mat* x,
                          const int32_t* place, uint64_t R, const s2r_mat* out,
                          const s2r_q8_mat* outq, void* stream);

/* y[t] = sum over k of weight[t][k] * rows[place[t][k]], in the order of k, in fp32 and rounded
 * once; weight [T][K] fp32, dense, or NULL for ones.  A token without a row gives zeros.  rows [R][D] and y
 * [T][D] may be of different dtypes. */
s2r_status s2r_moe_combine(uint64_t T, uint32_t K, uint64_t D, const s2r_mat* rows, uint64_t R,
                           const int32_t* place, const float* weight, const s2r_mat* y,
                           void* stream);

/* With dy [T][D] the gradient of y:
 *   drows[place[t][k]] = weight[t][k] * dy[t]   (weight NULL: ones) as drows [R][D], of any dtype, and
 *                        drowsq [R][D] in 8 bits (row blocks);
 *   dweight[t][k] = sum over D of dy[t] * rows[place[t][k]], 0 where there is no row; fp32 [T][K].
 * Each output may be NULL, not all; rows [R][D], of dy's dtype, is needed for dweight alone and may be NULL
 * without it. */
s2r_status s2r_moe_combine_grad(uint64_t T, uint32_t K, uint64_t D, const s2r_mat* dy,
                                const int32_t* place, uint64_t R, const float* weight,
                                const s2r_mat* rows, const s2r_mat* drows,
                                const s2r_q8_mat* drowsq, float* dweight, void* stream);

/* c[m][n] = sum over k < K of value(a[m][k]) * value(b_e[n][k]) for the rows m of every expert e,
 * summed and rounded as in s2r_q8_gemm.  a [M][K] row blocks and c [M][N] are sorted matrices.
 * b is expert 0's matrix [N][K] in square blocks; expert e's has its codes b_step * e bytes and its
 * scales b_scale_step * e bytes further on (b_step a multiple of 16).  Weights stacked with NS rows each,
 * NS a multiple of 128, are one matrix for s2r_q8_weight: b_step is NS * ld and b_scale_step NS / 128; the
 * transposed copy has them side by side: NS and NS / 128 * lds. */
s2r_status s2r_q8_gemm_experts(uint64_t M, uint64_t N, uint64_t K, const s2r_experts* experts,
                               const s2r_q8_mat* a, const s2r_q8_mat* b, uint64_t b_step,
                               uint64_t b_scale_step, const s2r_mat* c, void* stream);

/* dw_e[n][k] = (accumulate ? dw_e[n][k] : 0) + sum over the rows m of e of dy[m][n] * value(x[m][k]),
 * dw_e = dw + e * dw_step, each [N][lddw], for every expert; one without rows gets zeros.  dy16, dy8
 * and x are sorted matrices of M rows, the rest as in s2r_q8_wgrad.  dw_step >= (N - 1) * lddw + K. */
s2r_status s2r_q8_wgrad_experts(uint64_t M, uint64_t N, uint64_t K, const s2r_experts* experts,
                                const s2r_mat* dy16, const s2r_q8_mat* dy8, const s2r_q8_mat* x,
                                float* dw, uint64_t lddw, uint64_t dw_step, int accumulate,
                                void* stream);

#ifdef __cplusplus
}
#endif

#endif /* S2R_MOE_H */
