/*
 * q4_mx.h -- C ABI of the operators on microscaled (MX) numbers (the same
 * libq4.so as q4.h):
 *
 *   mx_quantize, mx_dequantize  blocks of 32 values <-> codes and scales
 *   mx_linear    y = act(x . W^T + b) + r                  (and its gradients)
 *   mx_gated     h = act(x . Wg^T + bg) * (x . Wu^T + bu)  (and its gradients)
 *   block_norm_mx  block_norm whose n leaves as codes and scales
 *
 * Chained, they are the feed-forward half of a layer on 4-bit floating-point
 * weights: block_norm_mx gives the x of mx_gated, whose h mx_quantize turns
 * into the x of the down projection's mx_linear.
 *
 * An MX tensor [R][K], K a multiple of 32, is two planes:
 *   Q4_MXFP4 (e2m1: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives)
 *     codes  : uint8 [R][K/2]   byte i = c_{2i} | c_{2i+1} << 4, c = sign << 3 | magnitude
 *   Q4_MXFP8 (e4m3: largest 448, no infinity, 0x7F and 0xFF are NaN)
 *     codes  : uint8 [R][K]
 *   both
 *     scales : uint8 [R][K/32]  e8m0: 2^(s - 127), 255 is NaN
 * A value is code * scale of its block of 32 along K (the OCP Microscaling
 * Formats specification's MXFP4 and MXFP8).
 *
 * Conventions are those of q4.h and q4_block.h: device pointers owned by the
 * caller, contiguous, 16-byte aligned; calls only enqueue kernels on `stream`
 * (no allocation, copy or synchronisation: they may be captured into a HIP
 * graph); every argument is checked on the host before any HIP call and a
 * rejected call enqueues nothing; M == 0 (or N == 0, D == 0) is a no-op that
 * returns Q4_OK; calls are deterministic.  Status, dtype, activation and norm
 * codes are those of q4.h and q4_block.h.
 */
#ifndef GEMV_Q4_AFFINE_AMD_Q4_MX_H
#define GEMV_Q4_AFFINE_AMD_Q4_MX_H

#include "q4_block.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- types: these, or where said Q4_BF16 / Q4_F16 of q4.h -------------------- */
#define Q4_MXFP4  8
#define Q4_MXFP8  9

/*
 * mx_quantize -- v [M][K] to codes and scales.  With e = 2 (MXFP4) or 8 (MXFP8):
 *   scale = 2^(floor(log2 max|v|) - e), at least 2^-127 (also for a block of zeros)
 *   code  = v / scale rounded to nearest even, cut to +-6 or +-448
 * A block that holds an infinity or a NaN becomes NaN: scale 255, codes 0.
 *   v      : device, [M][K] of dtype (Q4_F32, Q4_BF16 or Q4_F16)
 *   codes, scales : device out, the planes of `type`
 *   K % 32 == 0, 0 < K <= 2^30, M <= 2^30 (else Q4_ERR_SHAPE).
 */
int mx_quantize(const void* v, int dtype, int type, uint8_t* codes, uint8_t* scales, int64_t M, int64_t K, void* stream);

/*
 * mx_dequantize -- the values that planes stand for, rounded once into dtype
 * (Q4_F32 and Q4_BF16 hold them exactly, but for overflow and, at scales
 * below 2^-120, bfloat16's smallest values).  Shapes as above.
 */
int mx_dequantize(int type, const uint8_t* codes, const uint8_t* scales, void* v, int dtype, int64_t M, int64_t K,
                  void* stream);

/*
 * mx_linear -- y = act(z) + residual, z = x . W^T + bias, W [N][K] in MXFP4.
 *   w_q, w_s : device, codes and scales of W
 *   x_type   : Q4_BF16 or Q4_F16: x is [M][K] of that type, x_s NULL and dtype
 *              the same (else Q4_ERR_DTYPE); Q4_MXFP8 or Q4_MXFP4: x and x_s are
 *              the planes of x
 *   dtype    : Q4_BF16 or Q4_F16, of bias, residual, y and pre
 *   bias, residual, y, pre : as in q4_linear (residual may be y itself)
 *   K % 32 == 0; N, K <= 2^25, M <= 2^30 (here and in the other products).
 *   workspace: mx_linear_workspace_size(x_type, M, N, K) bytes (0: may be
 *              NULL), else Q4_ERR_WORKSPACE.  Calls sharing it must not overlap.
 *
 * Sums are binary32; the operands are taken as they are: products are exact.
 * With MX x the matrix instruction adds the 64 or 128 products of a step at a
 * fixed precision below the largest of them: MXFP8 x loses what lies about 2^-16
 * under it (a sum's error is 5e-6 of it on ordinary data), MXFP4 x nothing.
 * W may have any scales.  Only with binary16 x above 64 rows are blocks of W whose
 * scale is less than 2^-36 of their row's largest rounded (to multiples of 2^-37 of
 * that one), and in the gradients blocks whose scale is less than 2^-36 of the
 * largest of the same 32 columns; dz is rounded to binary16 after a power of two for
 * each row, as in q4_linear.
 *
 * (The terms of a sum have to stay in binary32's range, 3.4e38.)
 * A row of x with an infinity or a NaN (a NaN code or scale) spoils no other
 * row of y, and a column of W with a NaN scale no other column.
 */
int64_t mx_linear_workspace_size(int x_type, int64_t M, int64_t N, int64_t K);
int mx_linear(const uint8_t* w_q, const uint8_t* w_s, const void* bias, int act, const void* residual, int x_type,
              const void* x, const uint8_t* x_s, int dtype, void* y, void* pre, int64_t M, int64_t N, int64_t K,
              void* workspace, int64_t workspace_bytes, void* stream);

/*
 * mx_linear_backward -- with dz = dy * act'(pre): dx = dz . W and dbias, as
 * q4_linear_backward (dtype Q4_BF16 only; the same dz, pre and dbias).  For an
 * x that was quantised, dx is the gradient of the values its codes stand for.
 */
int64_t mx_linear_backward_workspace_size(int64_t M, int64_t N, int64_t K);
int mx_linear_backward(const uint8_t* w_q, const uint8_t* w_s, int act, const void* pre, const void* dy, int dtype,
                       void* dx, void* dz, float* dbias, int64_t M, int64_t N, int64_t K, void* workspace,
                       int64_t workspace_bytes, void* stream);

/*
 * mx_gated -- h = act(g) * u, g = x . Wg^T + gate_bias, u = x . Wu^T + up_bias;
 * x as in mx_linear, the other arguments as in q4_gated (gate_pre and up_pre
 * both or neither).
 */
int64_t mx_gated_workspace_size(int x_type, int64_t M, int64_t N, int64_t K);
int mx_gated(const uint8_t* gate_q, const uint8_t* gate_s, const uint8_t* up_q, const uint8_t* up_s,
             const void* gate_bias, const void* up_bias, int act, int x_type, const void* x, const uint8_t* x_s,
             int dtype, void* h, void* gate_pre, void* up_pre, int64_t M, int64_t N, int64_t K, void* workspace,
             int64_t workspace_bytes, void* stream);

/* mx_gated_backward -- as q4_gated_backward. */
int64_t mx_gated_backward_workspace_size(int64_t M, int64_t N, int64_t K);
int mx_gated_backward(const uint8_t* gate_q, const uint8_t* gate_s, const uint8_t* up_q, const uint8_t* up_s, int act,
                      const void* gate_pre, const void* up_pre, const void* dh, int dtype, void* dx, void* dgate,
                      void* dup, float* dgate_bias, float* dup_bias, int64_t M, int64_t N, int64_t K,
                      void* workspace, int64_t workspace_bytes, void* stream);

/*
 * block_norm_mx -- block_norm (q4_block.h) whose n leaves quantised:
 *   p = post(y);  r' = r + scale * gate * p;  n = pre(r') as codes and scales
 * computed in binary64 from the inputs to the codes, so that these are the ones
 * that mx_quantize's rule gives for the exact n (one past binary32's range
 * counts as its largest number).
 *   y .. eps, r_out, stats : as in block_norm, pre_norm not Q4_NORM_NONE
 *             (Q4_ERR_ARG); D % 32 == 0 (Q4_ERR_SHAPE)
 *   n_type    : Q4_MXFP8 or Q4_MXFP4
 *   n_codes, n_scales : device out, the planes [M][D] of n_type
 * The gradients are block_norm_backward's, of the values before their rounding
 * to codes.
 */
int block_norm_mx(const void* y, const void* r, int dtype, int r_dtype, int64_t M, int64_t D, int post_norm,
                  const void* post_weight, const void* post_bias, const void* gate, int64_t gate_rows, float scale,
                  int pre_norm, const void* pre_weight, const void* pre_bias, float eps, void* r_out, int n_type,
                  uint8_t* n_codes, uint8_t* n_scales, float* stats, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GEMV_Q4_AFFINE_AMD_Q4_MX_H */
