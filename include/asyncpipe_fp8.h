/*
 * libasyncpipe: 8-bit block-scaled operators on GB300 (sm_103a).
 *
 * The operators of a layer whose matrix products run in 8-bit floating point:
 * a root-mean-square norm that adds the residual and writes its output in
 * 8 bits, its gradient, a quantiser, and the matrix product that reads what
 * these write. The 8-bit type is e4m3 (1 sign, 4 exponent, 3 mantissa bits,
 * largest value 448, one NaN code a sign, no infinities).
 *
 * Blocks and scales. A value v of a block is held as the code
 *     q = e4m3(v * (1 / s)),   s = max(amax / 448, 2^-126),
 * amax the largest |v| of the block, every operation in 32 bits rounded to
 * nearest even; q * s stands for v. A row block is 128 consecutive values of
 * a row, columns 128 j .. 128 j + 127, the last block of a row possibly
 * shorter; a tile is 128 x 128 values, the last ones possibly smaller. A block
 * that holds a NaN has scale NaN and codes NaN; one that holds an infinity and
 * no NaN has scale infinity, code NaN where the infinity was and 0 elsewhere.
 * Scale arrays are float32, row-major without gaps: row blocks of a rows x
 * cols matrix have rows x ceil(cols / 128) scales, tiles have
 * ceil(rows / 128) x ceil(cols / 128).
 *
 * Conventions beside those of asyncpipe.h (streams, empty calls, graph
 * capture, no device memory allocated, arguments checked before any CUDA
 * call):
 *  - Matrices are row-major with a leading dimension ld (in elements, at
 *    least the columns), so they may be slices of wider ones. Any alignment
 *    of whole elements is accepted except where a call says otherwise; rows
 *    that start on 16-byte boundaries are read and written 16 bytes at a time.
 *  - An output may be the same matrix as an input of the same element size
 *    and leading dimension where the call says "in place"; any other overlap
 *    of an output with another argument is AP_ERR_ALIAS. Two matrices of one
 *    allocation whose rows interleave without sharing bytes (column slices of
 *    one wider matrix) do not overlap.
 *  - Sums, statistics and accumulators are held in 32 bits; each output is
 *    rounded once, to nearest even.
 *  - Results do not depend on timing: no sum is taken in an order that can
 *    change from call to call.
 *  - Pointers are device memory. A call may be captured into a graph once a
 *    call of the same sizes, types and alignment has run outside capture (sizes
 *    choose between kernels, and each has one-time attributes).
 */
#ifndef ASYNCPIPE_FP8_H
#define ASYNCPIPE_FP8_H

#include <stdint.h>

#include "asyncpipe.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum ap_dtype { AP_F32 = 0, AP_BF16 = 1, AP_F16 = 2 } ap_dtype;

/*
 * ap_rms_norm: for every row,
 *     h = x + residual,  r = 1 / sqrt(mean(h^2) + eps),  y = h * r * weight.
 *  x            rows x cols of `type`, leading dimension ldx.
 *  residual     rows x cols of `residual_type` (`type` or AP_F32), leading
 *               dimension ldr, or NULL: h = x.
 *  residual_out h rounded to residual_type, leading dimension ldr; NULL if
 *               and only if residual is. In place: residual. The norm itself
 *               uses h before that rounding.
 *  weight       cols values of `weight_type` (`type` or AP_F32).
 *  y            y in `type`, leading dimension ldy, or NULL. In place: x.
 *  q, q_scales  y (before any rounding) in e4m3 by row blocks, leading
 *               dimension ldq, and its scales; both NULL or neither. One of y
 *               and q is required.
 *  rstd         r of every row, or NULL.
 *  rows, cols   >= 0; no rows or no columns: nothing is written.
 */
ap_status ap_rms_norm(const void* x, int64_t ldx, ap_dtype type, const void* residual, void* residual_out,
                      int64_t ldr, ap_dtype residual_type, const void* weight, ap_dtype weight_type, float eps,
                      int64_t rows, int64_t cols, void* y, int64_t ldy, uint8_t* q, int64_t ldq, float* q_scales,
                      float* rstd, cudaStream_t stream);

/*
 * ap_rms_norm_backward: the gradient of ap_rms_norm. With n = h * r and
 * g = dy * weight, for every row
 *     dx = r * (g - n * mean(g * n)) + dresidual
 * and dweight[j] = sum over the rows of dy[., j] * n[., j].
 *  dy           rows x cols of `type`, leading dimension lddy: the gradient
 *               with respect to y.
 *  h            rows x cols of `residual_type` (`type` or AP_F32), leading
 *               dimension ldh: the forward call's residual_out, or its x
 *               where there was no residual.
 *  weight       as in the forward call; rstd the forward call's rstd.
 *  dresidual    gradient with respect to residual_out from elsewhere, of
 *               residual_type, leading dimension lddr; or NULL: 0.
 *  dx           the gradient with respect to x and to residual, of
 *               residual_type, leading dimension lddx. In place: dresidual, h
 *               or dy.
 *  dweight      cols floats, or NULL. No rows: zeros.
 *  workspace    device memory of at least ap_rms_norm_backward_workspace(rows,
 *               cols) bytes, 16-byte aligned, its contents undefined before
 *               and after the call (NULL allowed where dweight is NULL). One
 *               call at a time may use it.
 */
ap_status ap_rms_norm_backward(const void* dy, int64_t lddy, ap_dtype type, const void* h, int64_t ldh,
                               ap_dtype residual_type, const void* weight, ap_dtype weight_type, const float* rstd,
                               const void* dresidual, int64_t lddr, int64_t rows, int64_t cols, void* dx, int64_t lddx,
                               float* dweight, void* workspace, cudaStream_t stream);

/* Bytes of workspace ap_rms_norm_backward needs for these sizes; -1 if they
 * are not valid. Makes no CUDA call. */
int64_t ap_rms_norm_backward_workspace(int64_t rows, int64_t cols);

/*
 * ap_quantize: a rows x cols matrix in e4m3 with scales, as it stands (q,
 * scales), transposed (qt, scales_t), or both from one pass over x.
 *  x            rows x cols of `type`, leading dimension ldx.
 *  block_rows   1: row blocks; qt then holds row blocks of the transposed
 *               matrix, i.e. 128 consecutive rows of one column of x share a
 *               scale (an output gradient or an activation as the operands of
 *               a weight's gradient). 128: tiles, the same for q and qt (a
 *               weight).
 *  q, scales    rows x cols, leading dimension ldq; both NULL or neither.
 *  qt, scales_t cols x rows, leading dimension ldqt; scales_t as the scales of
 *               a cols x rows matrix; both NULL or neither. One of q and qt is
 *               required.
 */
ap_status ap_quantize(const void* x, int64_t ldx, ap_dtype type, int64_t rows, int64_t cols, int block_rows,
                      uint8_t* q, int64_t ldq, float* scales, uint8_t* qt, int64_t ldqt, float* scales_t,
                      cudaStream_t stream);

/*
 * ap_matmul_fp8: c = a * b^T of block-scaled 8-bit matrices,
 *     c[i, j] = sum over blocks kb of (sa sb) * sum over the block's k of a[i, k] b[j, k],
 * sa = a_scales[i, kb], sb = b_scales[j / 128, kb] (b_block_rows = 128: b in
 * tiles) or b_scales[j, kb] (b_block_rows = 1: b in row blocks).
 * The products of a block of 128 are summed by the tensor cores into 32-bit
 * accumulators; each block's sum times sa sb is added to a 32-bit sum.
 * The product sa sb is formed first, in 32 bits rounded to nearest, and is to
 * be a float: past the largest one (two scales of 2^64 and more) it is an
 * infinity and the term infinite, or NaN where the block's sum is 0; below 2^-126
 * (two of 2^-63 and less) it is subnormal and has lost bits, and so has the term.
 * Blocks whose largest magnitudes lie between 2^-54 and 2^72, or are 0, meet
 * without either.
 *  a            m x k, leading dimension lda; a_scales by row blocks.
 *  b            n x k, leading dimension ldb; b_scales as b_block_rows says.
 *  c            m x n of c_type, leading dimension ldc.
 *  a and b start on 16-byte boundaries and lda and ldb are multiples of 16
 *  (AP_ERR_ALIGN otherwise); m, n and k are any sizes up to 2^31 - 512. What a
 *  row holds past k is not read.
 *  m or n = 0: nothing is written. k = 0: c is set to zero.
 */
ap_status ap_matmul_fp8(const uint8_t* a, int64_t lda, const float* a_scales, const uint8_t* b, int64_t ldb,
                        const float* b_scales, int b_block_rows, void* c, int64_t ldc, ap_dtype c_type, int64_t m,
                        int64_t n, int64_t k, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* ASYNCPIPE_FP8_H */
