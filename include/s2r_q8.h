/* s2r_q8.h -- training a linear layer in 8 bits, exported by libs2r.so (gfx950): the step
 * before the aggregation path of s2r.h.  A worker's forward pass keeps what its backward
 * pass needs as 8-bit checkpoints, the products run on 8-bit operands, and the weight
 * gradient is written in fp32 straight into the worker's gradient row, from where
 * s2r_topk_ef and s2r_encode take it.
 *
 *   s2r_q8_save      rows of activations or gradients -> 8 bits, a scale per 128 elements
 *   s2r_q8_load      8 bits -> bf16 / fp16 / fp32
 *   s2r_q8_weight    weights -> 8 bits, a scale per 128 x 128 block, and the transposed copy
 *   s2r_q8_gemm      C = A B^T of 8-bit matrices: layer output and input gradient
 *   s2r_q8_gemm_fast the same at the 8-bit matrix rate, with products cut short
 *   s2r_q8_wgrad     dW (+)= dY^T X from the checkpoint of X: weight gradient
 *   s2r_q8_glu       y = act(g) * u with checkpoints of g and u
 *   s2r_q8_glu_grad  its gradient from those checkpoints
 *
 * Stored form.  A matrix of R rows and C columns is held as codes q [R][ld] (one byte each)
 * and scale bytes.  A scale byte b stands for 2^(b - 127) and the value of an element is
 *   value = code * 2^(b - 127).
 *   row blocks:    scale [ceil(C / 128)][lds], lds >= R: byte [c / 128][r] covers elements
 *                  c .. c + 127 of row r;
 *   square blocks: scale [ceil(C / 128)][lds], lds >= ceil(R / 128): byte [c / 128][r / 128]
 *                  covers a 128 x 128 block (weights).
 * Writing: with a the largest finite magnitude of the block and MAX the format's largest
 * value (448 for e4m3, 57344 for e5m2), the scale is the least power of two with
 * a <= MAX * scale, but no less than 2^-110 (b = 17, also for a block of zeros), and a code is
 * value / scale rounded to nearest, ties to even.  So a value is off by at most 2^-4 (e4m3) or
 * 2^-3 (e5m2) of itself, or by 2^-10 (e4m3) or 2^-17 (e5m2) of its block's scale if it is
 * below the format's normal range.  NaN stays NaN; an infinity becomes NaN in e4m3 and stays
 * in e5m2; neither changes the scale of its block.  Every stored value is exact in bf16 and
 * in fp32, and finite if it was: what would round to 2^128 gets the largest code below it, within
 * the same bounds.  Scale bytes are 17 .. 247 (e4m3) or 17 .. 240 (e5m2), also those of
 * matrices written elsewhere, whose values must be below 2^128.
 *
 * Conventions, beyond those of s2r.h (device memory, streams, host checks before anything is
 * enqueued, no allocation, calls from several threads):
 *   - Matrices are row-major with unit stride along a row.  q, scale and every s2r_mat are
 *     described by the host structs below, copied at call time.
 *   - Alignment: q and data 16 bytes, ld a multiple of 16 bytes (ld % 16 for codes, % 8 for
 *     16-bit and % 4 for fp32 elements); scale 4 bytes and lds % 4 == 0, each scale row whole.
 *     The elements after a row's last column up to a multiple of 16 bytes exist, are never
 *     written, and may hold anything; nothing beyond them is touched.  So a matrix may be a
 *     range of columns of a wider one (of 8-bit ones from a multiple of 128 on, with the scales
 *     of its blocks), and two products that add up, as dX = dG Wg + dU Wu, are one of matrices
 *     side by side.
 *   - Sizes: rows and columns below 2^28; ld of at most 2^22 elements.  A size of 0 is a call
 *     that writes nothing, but an empty sum is a sum: K == 0 in s2r_q8_gemm writes zeros, and
 *     M == 0 in s2r_q8_wgrad without `accumulate` too.
 *   - No output may overlap an input or another output.
 *   - Sums are fp32 in an order fixed by the sizes and by whether there is a workspace: the
 *     same call gives the same bits on every run.
 *   - Errors: S2R_ERR_NULL, S2R_ERR_DIM (sizes, ld or lds too small or too large, an unknown
 *     dtype, format or act), S2R_ERR_ALIGN, S2R_ERR_WORKSPACE, S2R_ERR_HIP.
 */
#ifndef S2R_Q8_H
#define S2R_Q8_H

#include <stddef.h>
#include <stdint.h>

#include "s2r.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { S2R_BF16 = 0, S2R_F16 = 1, S2R_F32 = 2 } s2r_dtype;
/* OCP 8-bit formats: e4m3 has no infinity (largest value 448), e5m2 has (57344). */
typedef enum { S2R_E4M3 = 0, S2R_E5M2 = 1 } s2r_q8_format;
/* SiLU x / (1 + e^-x); GELU x * Phi(x); GELU_TANH its tanh form
 * x/2 (1 + tanh(sqrt(2/pi) (x + 0.044715 x^3))). */
typedef enum { S2R_ACT_SILU = 0, S2R_ACT_GELU = 1, S2R_ACT_GELU_TANH = 2 } s2r_act;

typedef struct {
  void* data;      /* [rows][ld] */
  uint64_t ld;     /* elements from one row to the next */
  uint32_t dtype;  /* s2r_dtype */
} s2r_mat;

typedef struct {
  uint8_t* q;       /* [rows][ld] codes */
  uint64_t ld;      /* codes from one row to the next */
  uint8_t* scale;   /* [ceil(cols / 128)][lds] */
  uint64_t lds;     /* scale bytes from one block of columns to the next */
  uint32_t format;  /* s2r_q8_format */
} s2r_q8_mat;

/* x [M][K] -> out (row blocks).  x may be bf16, fp16 or fp32. */
s2r_status s2r_q8_save(uint64_t M, uint64_t K, const s2r_mat* x, const s2r_q8_mat* out,
                       void* stream);

/* in [M][K] (row blocks) -> x.  fp32 and bf16 hold the stored values exactly; fp16 rounds once. */
s2r_status s2r_q8_load(uint64_t M, uint64_t K, const s2r_q8_mat* in, const s2r_mat* x,
                       void* stream);

/* w [N][K] -> out (square blocks) and, unless NULL, out_t: the same codes as [K][N], with
 * the scales transposed, as s2r_q8_gemm takes them for the input gradient. */
s2r_status s2r_q8_weight(uint64_t N, uint64_t K, const s2r_mat* w, const s2r_q8_mat* out,
                         const s2r_q8_mat* out_t, void* stream);

/* Bytes of device workspace that let s2r_q8_gemm and s2r_q8_gemm_fast cut a long sum among
 * workgroups where the result alone is too small to fill the GPU; 0 where they would not. */
size_t s2r_q8_gemm_workspace_bytes(uint64_t M, uint64_t N, uint64_t K);

/* c[m][n] = sum over k < K of value(a[m][k]) * value(b[n][k]).
 * a [M][K] row blocks, b [N][K] square blocks, c [M][N] of any s2r_dtype.  Every product is
 * exact as far as fp32 reaches and every addition fp32; c is rounded once.
 * Layer output: a = X, b = W [N][K].  Input gradient: a = dY, b = the
 * transposed copy of s2r_q8_weight.  Any M from one token up.
 * workspace may be NULL (or ws_bytes 0): the sum is then never cut.  Otherwise it holds at
 * least s2r_q8_gemm_workspace_bytes(M, N, K) bytes, 16-byte aligned; contents on entry do not
 * matter. */
s2r_status s2r_q8_gemm(uint64_t M, uint64_t N, uint64_t K, const s2r_q8_mat* a,
                       const s2r_q8_mat* b, const s2r_mat* c, void* workspace, size_t ws_bytes,
                       void* stream);

/* The same call through the 8-bit matrix instruction, 1.8 times as fast for large sizes, for
 * results that may be a little off: of each eight consecutive k, 8 i .. 8 i + 7, a product is cut
 * toward zero by less than 2^-13 of the largest of the eight |a b|, where a nonzero value
 * below its format's normal range (2^-6 of its scale in e4m3, 2^-14 in e5m2) counts as the least
 * normal.  So a result is off by at most 7 * 2^-13 times the sum of those largest products, apart
 * from its fp32 additions and its rounding; on ordinary values by 2.4e-5 of its typical size (root mean
 * square, 5001 x 1000 x 4100).  Few rows of A, which memory bounds, are summed as in s2r_q8_gemm. */
s2r_status s2r_q8_gemm_fast(uint64_t M, uint64_t N, uint64_t K, const s2r_q8_mat* a,
                            const s2r_q8_mat* b, const s2r_mat* c, void* workspace,
                            size_t ws_bytes, void* stream);

/* The same for s2r_q8_wgrad. */
size_t s2r_q8_wgrad_workspace_bytes(uint64_t M, uint64_t N, uint64_t K);

/* dw[n][k] = (accumulate ? dw[n][k] : 0) + sum over m < M of dy[m][n] * value(x[m][k]).
 * dy is given as dy16 [M][N] (bf16 only: S2R_ERR_DIM otherwise) or as dy8 [M][N] (row
 * blocks), the other one NULL; x [M][K] row blocks; dw fp32 [N][lddw], lddw >= K, 4-byte
 * aligned (any element of a worker's gradient row).  The products are exact as far as fp32
 * reaches, and the sums fp32.
 * workspace as in s2r_q8_gemm, with s2r_q8_wgrad_workspace_bytes(M, N, K). */
s2r_status s2r_q8_wgrad(uint64_t M, uint64_t N, uint64_t K, const s2r_mat* dy16,
                        const s2r_q8_mat* dy8, const s2r_q8_mat* x, float* dw, uint64_t lddw,
                        int accumulate, void* workspace, size_t ws_bytes, void* stream);

/* y = act(g) * u, or y = act(g) with u == NULL, computed in fp32 from g and u [M][F] (of one
 * dtype).  Each output may be NULL, not all of them: gq and uq are the checkpoints of g and
 * u, y [M][F] of any s2r_dtype and yq the result in 8 bits (all row blocks).  uq needs u. */
s2r_status s2r_q8_glu(uint64_t M, uint64_t F, s2r_act act, const s2r_mat* g, const s2r_mat* u,
                      const s2r_q8_mat* gq, const s2r_q8_mat* uq, const s2r_mat* y,
                      const s2r_q8_mat* yq, void* stream);

/* With g and u the stored values of gq and uq (uq NULL where the forward pass had no u):
 *   dg = dy * u * act'(g)  (dy * act'(g) without u),   du = dy * act(g)
 * in fp32 from dy [M][F] of any s2r_dtype.  Outputs, each of which may be NULL but not all: dg
 * and du as matrices of any dtype, dgq and duq in 8 bits.  du and duq need uq. */
s2r_status s2r_q8_glu_grad(uint64_t M, uint64_t F, s2r_act act, const s2r_q8_mat* gq,
                           const s2r_q8_mat* uq, const s2r_mat* dy, const s2r_mat* dg,
                           const s2r_mat* du, const s2r_q8_mat* dgq, const s2r_q8_mat* duq,
                           void* stream);

#ifdef __cplusplus
}
#endif

#endif /* S2R_Q8_H */
