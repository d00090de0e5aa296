/*
 * libasyncpipe: a gated feed-forward block on GB300 (sm_103a).
 *
 * The operators of a block y = act(x Wg^T) * (x Wu^T), elementwise product,
 * beside those of asyncpipe_fp8.h: both projections with the activation in one
 * kernel and their gradient, in 8 bits; and products with weights of 4 bits for
 * few rows of x, where the weight's bytes are what a call costs.
 *
 * Activations. act(g) = g s(w(g)) with s(w) = 1 / (1 + exp(-w)):
 *     AP_ACT_SILU  w = g;
 *     AP_ACT_GELU  w = 2 sqrt(2 / pi) (g + 0.044715 g^3), the form with tanh:
 *                  act(g) = g / 2 (1 + tanh(sqrt(2 / pi) (g + 0.044715 g^3))).
 * act is 0 at minus infinity and infinity at infinity, its slope 0 and 1.
 * s below 2^-126, w below about -87.3, is taken as 0: act and its slope are 0
 * there, off by less than |g| 2^-126 and (1 + |g| w'(g)) 2^-126.
 *
 * 4-bit weights. A weight of n rows and k columns is stored row by row, two
 * columns a byte, the even one in the low half, an odd last column in the low
 * half of a byte of its own; row j starts at byte j * ldw. `group` columns
 * (32, 64 or 128, the last group of a row possibly shorter) share a scale and a
 * zero point: with G = ceil(k / group), scales and zeros are n x G, row-major
 * without gaps, and the code v in 0..15 stands for
 *     (v - zeros[j, i / group]) * scales[j, i / group].
 * zeros are whole numbers from 0 to 255, one a byte; NULL: 8 for every group.
 * How the codes were chosen is not the library's business.
 *
 * Conventions as in asyncpipe_fp8.h.
 */
#ifndef ASYNCPIPE_GATED_H
#define ASYNCPIPE_GATED_H

#include <stdint.h>

#include "asyncpipe_fp8.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum ap_activation { AP_ACT_SILU = 0, AP_ACT_GELU = 1 } ap_activation;

/*
 * ap_gated_matmul_fp8: both projections of a gated block, the activation and
 * the product in one kernel,
 *     g = a * Wg^T,  u = a * Wu^T,  y = act(g) * u,
 * of block-scaled 8-bit matrices. Each product is ap_matmul_fp8's with a
 * weight in tiles (what it says of scales and sums holds here); g, u and y stay
 * in 32 bits up to the rounding of each output.
 *  a            m x k, leading dimension lda; a_scales by row blocks.
 *  gate_codes, up_codes  Wg and Wu, n x k each, leading dimensions ldwg, ldwu;
 *               gate_scales, up_scales by tiles.
 *  gate, up     g and u in `type`, leading dimensions ldg, ldu, each or NULL (a
 *               training step keeps both for ap_gated_backward).
 *  y            y in `type`, leading dimension ldy, or NULL.
 *  q, q_scales  y in e4m3 by row blocks, leading dimension ldq; both NULL or
 *               neither. One of y and q is required.
 *  a and both weights start on 16-byte boundaries and lda, ldwg and ldwu are
 *  multiples of 16 (AP_ERR_ALIGN otherwise); m, n and k are any sizes up to
 *  2^31 - 512. What a row holds past k is not read.
 *  m or n = 0: nothing is written. k = 0: every output is zero.
 */
ap_status ap_gated_matmul_fp8(const uint8_t* a, int64_t lda, const float* a_scales, const uint8_t* gate_codes,
                              int64_t ldwg, const float* gate_scales, const uint8_t* up_codes, int64_t ldwu,
                              const float* up_scales, ap_activation act, void* gate, int64_t ldg, void* up, int64_t ldu,
                              void* y, int64_t ldy, ap_dtype type, uint8_t* q, int64_t ldq, float* q_scales, int64_t m,
                              int64_t n, int64_t k, cudaStream_t stream);

/*
 * ap_gated_backward: the gradient of y = act(g) * u. From dy, the gradient
 * with respect to y,
 *     dg = dy u act'(g),  du = dy act(g),
 * and h = act(g) u itself, in any of these forms (at least one of dgate, dup, q,
 * qt and ht); the three are computed in 32 bits, and each output is rounded from there.
 *  dy, gate, up rows x cols of `type`, leading dimensions lddy, ldg, ldu: the
 *               forward call's gate and up.
 *  dgate, dup   dg and du in `type`, leading dimensions lddg, lddu, each or
 *               NULL. In place: any of dy, gate, up, by one of the two, where
 *               none of q, qt and ht is asked for.
 *  q, scales    dg and du side by side, rows x (cols' + cols) with cols' = cols
 *               rounded up to a multiple of 128, in e4m3 by row blocks, leading
 *               dimension ldq: columns 0 .. cols - 1 hold dg, columns from
 *               cols' on du, those between zeros. With the two weights stacked
 *               the same way, one product gives the block's input gradient.
 *               Both NULL or neither.
 *  qt, scales_t the transpose of that matrix, (cols' + cols) x rows, by its own
 *               row blocks, leading dimension ldqt (the operand of both
 *               projections' weight gradients); both NULL or neither.
 *  ht, ht_scales h transposed, cols x rows, by row blocks, leading dimension
 *               ldht (the operand of the down projection's weight gradient);
 *               both NULL or neither.
 *  rows, cols   >= 0; no rows or no columns: nothing is written.
 */
ap_status ap_gated_backward(const void* dy, int64_t lddy, const void* gate, int64_t ldg, const void* up, int64_t ldu,
                            ap_dtype type, ap_activation act, int64_t rows, int64_t cols, void* dgate, int64_t lddg,
                            void* dup, int64_t lddu, uint8_t* q, int64_t ldq, float* scales, uint8_t* qt, int64_t ldqt,
                            float* scales_t, uint8_t* ht, int64_t ldht, float* ht_scales, cudaStream_t stream);

/*
 * ap_matmul_w4: c = x * W^T for a 4-bit weight W,
 *     c[i, j] = sum over groups of scale * sum over the group's columns of x[i, .] (code - zero);
 * every sum in 32 bits, of products of x and the whole number code - zero, which are
 * exact. A column whose code is its zero point takes no part, unless its x is
 * infinite or NaN, which make that row's result NaN; an infinity times any other
 * weight is an infinity. (So is a group's sum that passes the largest float before
 * its scale.)
 *  x            m x k of `type` (AP_BF16 or AP_F16), leading dimension ldx.
 *  codes        the weight, n x k as above: 16-byte aligned, ldw (bytes) a
 *               multiple of 16 (AP_ERR_ALIGN otherwise). What a row holds past
 *               its last column is not used, what it holds past its last byte
 *               not read.
 *  scales       n x ceil(k / group) of `type`; zeros as above or NULL.
 *  c            m x n of c_type (`type` or AP_F32), leading dimension ldc.
 *  m up to 2^20; the weight is read once for every 32 rows of x.
 *  m or n = 0: nothing is written. k = 0: c is set to zero.
 */
ap_status ap_matmul_w4(const void* x, int64_t ldx, ap_dtype type, const uint8_t* codes, int64_t ldw, const void* scales,
                       const uint8_t* zeros, int group, void* c, int64_t ldc, ap_dtype c_type, int64_t m, int64_t n,
                       int64_t k, cudaStream_t stream);

/*
 * ap_gated_matmul_w4: y = act(x * Wg^T) * (x * Wu^T) for two 4-bit weights of
 * the same sizes, group and kind of zero points, each argument as above. The
 * two sums stay in 32 bits up to the one rounding of y.
 */
ap_status ap_gated_matmul_w4(const void* x, int64_t ldx, ap_dtype type, const uint8_t* gate_codes, int64_t ldwg,
                             const void* gate_scales, const uint8_t* gate_zeros, const uint8_t* up_codes, int64_t ldwu,
                             const void* up_scales, const uint8_t* up_zeros, int group, ap_activation act, void* y,
                             int64_t ldy, ap_dtype y_type, int64_t m, int64_t n, int64_t k, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* ASYNCPIPE_GATED_H */
