/* s2r_q4.h -- matrices in microscaled 4-bit floating point (OCP MXFP4) and their product, exported by
 * libs2r.so (gfx950), beside the 8-bit ones of s2r_q8.h: a quarter of bf16's bytes and up to four times
 * its matrix rate.
 *
 *   s2r_q4_save   rows of a matrix -> 4 bits, and those of its transpose
 *   s2r_q4_load   4 bits -> bf16 / fp16 / fp32
 *   s2r_q4_gemm   C = A B^T of 4-bit matrices
 *
 * Stored form.  A matrix of R rows and C columns is held as codes q [R][ld bytes], two to a byte, the
 * even column's in the low half, and scale bytes [R][lds]: byte [r][c / 32] covers elements c .. c + 31
 * of row r and stands for 2^(b - 127).  A code is a sign bit over three bits for 0, 0.5, 1, 1.5, 2, 3, 4
 * and 6 (e2m1); an element's value is code * 2^(b - 127), NaN for all 32 where b is 255.
 * Writing: with a the largest magnitude of the 32, the scale is the least power of two with
 * a <= 6 * scale, no less than 2^-110 (b = 17, also for zeros) and no more than 2^125 (b = 252), and a code
 * is value / scale rounded to nearest, ties to the even code, or 6 where that is beyond it (values above
 * 6 * 2^125 alone).  So a value is off by at most a quarter of its scale below 2 scales, half of it below 4
 * and one above.  32 elements with a NaN or an infinity among them are stored as NaN, b = 255 with codes
 * of zero.
 * Matrices written elsewhere may have any b of 17 .. 252 and 255.
 *
 * The product along either side.  A block runs along the summed index, so the product with a
 * transpose takes codes of its own: s2r_q4_save writes those of x and of its transpose in one pass.  With X
 * [M][K], W [N][K] and dY [M][N]: Y = X W^T is s2r_q4_gemm of X and W, dX = dY W of dY and W's
 * transpose, dW = dY^T X of both transposes, its sum running over the tokens.
 *
 * Conventions are those of s2r_q8.h, with ld and lds in bytes: q 16-byte aligned, ld a multiple of 16 and at
 * most 2^22, ld >= C / 2 rounded up; scale 8-byte aligned, lds a multiple of 8 and >= C / 32 rounded up.
 * The bytes after a row's last code up to a multiple of 16, and after its last scale up to a multiple of
 * 8, exist, may hold anything and are left as they are, but for the unused half of an odd row's last code
 * byte, which is written as 0.
 */
#ifndef S2R_Q4_H
#define S2R_Q4_H

#include "s2r_q8.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
  uint8_t* q;      /* [rows][ld] bytes of two codes */
  uint64_t ld;     /* bytes from one row to the next */
  uint8_t* scale;  /* [rows][lds] */
  uint64_t lds;    /* scale bytes from one row to the next */
} s2r_q4_mat;

/* x [R][C] (any s2r_dtype) -> out [R][C] and out_t [C][R], x's transpose with blocks of its own.
 * Either may be NULL, not both. */
s2r_status s2r_q4_save(uint64_t R, uint64_t C, const s2r_mat* x, const s2r_q4_mat* out,
                       const s2r_q4_mat* out_t, void* stream);

/* in [R][C] -> x.  fp32 and bf16 hold the stored values exactly; fp16 rounds once. */
s2r_status s2r_q4_load(uint64_t R, uint64_t C, const s2r_q4_mat* in, const s2r_mat* x,
                       void* stream);

/* Bytes of device workspace that let s2r_q4_gemm cut a long sum among workgroups where the result
 * alone is too small to fill the GPU; 0 where it would not. */
size_t s2r_q4_gemm_workspace_bytes(uint64_t M, uint64_t N, uint64_t K);

/* c[m][n] = sum over k < K of value(a[m][k]) * value(b[n][k]); a [M][K], b [N][K], c [M][N] of any
 * s2r_dtype.  Sums are fp32, c is rounded once.  K == 0 writes zeros.  Any M from one token up.
 * workspace as in s2r_q8_gemm. */
s2r_status s2r_q4_gemm(uint64_t M, uint64_t N, uint64_t K, const s2r_q4_mat* a,
                       const s2r_q4_mat* b, const s2r_mat* c, void* workspace, size_t ws_bytes,
                       void* stream);

#ifdef __cplusplus
}
#endif

#endif /* S2R_Q4_H */
