/*
 * q4_block.h -- C ABI of the feed-forward operators on block-quantised
 * weights (the same libq4.so as q4.h):
 *
 *   q4_linear    y = act(x . W^T + b) + r                 (and its gradients)
 *   q4_gated     h = act(x . Wg^T + bg) * (x . Wu^T + bu) (and its gradients)
 *   block_norm   r' = r + scale * gate * post(y), n = pre(r')   (and its gradients)
 *
 * Chained, they are the feed-forward half of a layer: n of one block_norm is
 * x of q4_gated, whose h is x of the down projection's q4_linear, whose y is
 * y of the next block_norm (or whose residual is the stream itself).
 *
 * The conventions are those of q4.h: device pointers owned by the caller,
 * contiguous row-major tensors, 16-byte aligned; a stream argument on which
 * the calls only enqueue kernels (no allocation, copy or synchronisation, so
 * they may be captured into a HIP graph); every argument is checked on the
 * host before any HIP call and a rejected call enqueues nothing; M == 0 (or
 * N == 0, D == 0) is a no-op that returns Q4_OK; calls are deterministic.
 * Status, dtype and format codes are those of q4.h.  W is frozen: its planes
 * (Q4_FMT_Q4_0: w_q = qs, w_s = d, w_b unused; Q4_FMT_AFFINE4 / _AFFINE8:
 * codes, scales, biases, group 64) get no gradient.
 *
 * dtype: Q4_BF16 or Q4_F16, the type of every activation tensor of the call.
 * Up to 64 rows the forward products are exact with binary32 accumulation.  Above, and
 * in the gradients, they are binary16 x binary16 (weights dequantised to
 * binary16, rounding <= 2^-11, absolute 2^-25 below 2^-14: the dequantised weights
 * must fit binary16; x and dz scaled per row by a power of two); for binary16 outputs of
 * a gated product or under a curved activation the roundings' remainders are
 * summed too.  Either way x and dz may be anything in their type's range.  Biases,
 * activations, products of projections, residuals and norms are computed in
 * binary32 and rounded once into the output.
 *
 * A row of x (dz, r, y) with an infinity or a NaN spoils no other row of the
 * outputs.  Its own sums over k are what their infinite terms make them: an infinity
 * of their sign, NaN where they oppose each other, where the weight is zero
 * (above 64 rows and in the gradients: zero in binary16), or next to a NaN.
 */
#ifndef GEMV_Q4_AFFINE_AMD_Q4_BLOCK_H
#define GEMV_Q4_AFFINE_AMD_Q4_BLOCK_H

#include "q4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- activations ----------------------------------------------------------- */
#define Q4_ACT_NONE       0
#define Q4_ACT_SILU       1   /* z / (1 + exp(-z))                                        */
#define Q4_ACT_GELU       2   /* z * (1 + erf(z / sqrt 2)) / 2                             */
#define Q4_ACT_GELU_TANH  3   /* z * (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) / 2         */
#define Q4_ACT_RELU       4   /* max(z, 0)                                                 */

/* ---- norms ------------------------------------------------------------------- */
#define Q4_NORM_NONE   0      /* the identity (no weight, no bias)                         */
#define Q4_NORM_RMS    1      /* v * rstd * w + b,          rstd = 1 / sqrt(mean(v^2) + eps)         */
#define Q4_NORM_LAYER  2      /* (v - mean) * rstd * w + b, rstd = 1 / sqrt(mean((v - mean)^2) + eps) */

/* Largest D of block_norm. */
#define Q4_NORM_MAX_D 32768

/*
 * q4_linear -- y = act(z) + residual, z = x . W^T + bias.
 *   x        : device, [M][K] of dtype;  y : device out, [M][N] of dtype
 *   bias     : device, [N] of dtype, or NULL
 *   residual : device, [M][N] of dtype, or NULL; may be y itself
 *   pre      : device out, [M][N] of dtype: z (for the backward pass), or NULL
 *   K % 32 == 0 (Q4_0) or K % 64 == 0 (affine); N, K <= 2^25, M <= 2^30 (here
 *   and in the other products).
 *   workspace: q4_linear_workspace_size(fmt, dtype, M, N, K) bytes (0: may be NULL),
 *              else Q4_ERR_WORKSPACE.  Calls sharing it must not overlap.
 */
int64_t q4_linear_workspace_size(int fmt, int dtype, int64_t M, int64_t N, int64_t K);
int q4_linear(int fmt, const uint8_t* w_q, const uint16_t* w_s, const uint16_t* w_b, const void* bias, int act,
              const void* residual, const void* x, int dtype, void* y, void* pre, int64_t M, int64_t N, int64_t K,
              void* workspace, int64_t workspace_bytes, void* stream);

/*
 * q4_linear_backward -- with dz = dy * act'(pre): dx = dz . W, dbias = sum
 * over the rows of dz (the residual's gradient is dy itself).
 *   dy    : device, [M][N] of dtype (Q4_BF16 only: binary16 gradients would
 *           lose small values; other types return Q4_ERR_DTYPE)
 *   pre   : device, [M][N] of dtype, as q4_linear wrote it (NULL with
 *           Q4_ACT_NONE)
 *   dx    : device out, [M][K] of dtype
 *   dz    : device out, [M][N] of dtype, or NULL (what an adapter beside W or
 *           another consumer of z's gradient reads); not with Q4_ACT_NONE,
 *           where it is dy (Q4_ERR_ARG)
 *   dbias : device out, float [N], or NULL
 *   Workspace as above, q4_linear_backward_workspace_size bytes.
 */
int64_t q4_linear_backward_workspace_size(int fmt, int64_t M, int64_t N, int64_t K);
int q4_linear_backward(int fmt, const uint8_t* w_q, const uint16_t* w_s, const uint16_t* w_b, int act,
                       const void* pre, const void* dy, int dtype, void* dx, void* dz, float* dbias, int64_t M,
                       int64_t N, int64_t K, void* workspace, int64_t workspace_bytes, void* stream);

/*
 * q4_gated -- h = act(g) * u, g = x . Wg^T + gate_bias, u = x . Wu^T + up_bias.
 *   Wg, Wu   : two [N][K] matrices of the same format
 *   h        : device out, [M][N] of dtype
 *   gate_pre, up_pre : device out, [M][N] of dtype: g and u (for the backward
 *              pass), both or neither (else Q4_ERR_ARG)
 */
int64_t q4_gated_workspace_size(int fmt, int dtype, int64_t M, int64_t N, int64_t K);
int q4_gated(int fmt, const uint8_t* gate_q, const uint16_t* gate_s, const uint16_t* gate_b, const uint8_t* up_q,
             const uint16_t* up_s, const uint16_t* up_b, const void* gate_bias, const void* up_bias, int act,
             const void* x, int dtype, void* h, void* gate_pre, void* up_pre, int64_t M, int64_t N, int64_t K,
             void* workspace, int64_t workspace_bytes, void* stream);

/*
 * q4_gated_backward -- dgate = dh * u * act'(g), dup = dh * act(g),
 * dx = dgate . Wg + dup . Wu (one product over both), and the bias gradients,
 * sums over the rows.  dtype Q4_BF16 only, as in q4_linear_backward.
 *   dgate, dup           : device out, [M][N] of dtype, or NULL
 *   dgate_bias, dup_bias : device out, float [N], or NULL
 */
int64_t q4_gated_backward_workspace_size(int fmt, int64_t M, int64_t N, int64_t K);
int q4_gated_backward(int fmt, const uint8_t* gate_q, const uint16_t* gate_s, const uint16_t* gate_b,
                      const uint8_t* up_q, const uint16_t* up_s, const uint16_t* up_b, int act,
                      const void* gate_pre, const void* up_pre, const void* dh, int dtype, void* dx, void* dgate,
                      void* dup, float* dgate_bias, float* dup_bias, int64_t M, int64_t N, int64_t K,
                      void* workspace, int64_t workspace_bytes, void* stream);

/*
 * block_norm -- the residual stream between two blocks:
 *   p = post(y);  r' = r + scale * gate * p;  n = pre(r')
 * with post and pre one of Q4_NORM_*.  n is computed from r' before r' is
 * rounded into r_out.
 * Squares are summed in binary32: a row whose sum of squares passes 3.4e38 has rstd 0.
 *   y       : device, [M][D] of dtype, a block's output, or NULL (then r' = r,
 *             post_norm is Q4_NORM_NONE, gate and r_out are NULL: the norm
 *             before the first block)
 *   r       : device, [M][D] of r_dtype;  r_out : device out, [M][D] of
 *             r_dtype, may be r itself
 *   dtype   : Q4_BF16, Q4_F16 or Q4_F32;  r_dtype : dtype or Q4_F32
 *   post_weight, pre_weight : [D] of dtype, or NULL for ones; post_bias,
 *             pre_bias : [D] of dtype, or NULL for zeros; NULL where the norm
 *             is Q4_NORM_NONE (else Q4_ERR_ARG)
 *   gate    : device, [ceil(M / gate_rows)][D] of dtype, or NULL for ones; row
 *             m uses gate row m / gate_rows (gate_rows = M: one for all;
 *             1: one per row; a sequence's length: one per sequence)
 *   n       : device out, [M][D] of dtype; NULL if and only if pre_norm is
 *             Q4_NORM_NONE
 *   stats   : device out, float [M][4] = {post mean, post rstd, pre mean, pre
 *             rstd} for the backward pass (mean 0 for RMS; 0 and 1 for NONE),
 *             or NULL
 *   eps     : > 0 and finite, scale finite, else Q4_ERR_ARG.  D <= Q4_NORM_MAX_D.
 */
int block_norm(const void* y, const void* r, int dtype, int r_dtype, int64_t M, int64_t D, int post_norm,
               const void* post_weight, const void* post_bias, const void* gate, int64_t gate_rows, float scale,
               int pre_norm, const void* pre_weight, const void* pre_bias, float eps, void* r_out, void* n,
               float* stats, void* stream);

/*
 * block_norm_backward -- with G = dr_out + pre'(dn), the gradient of r':
 *   dr = G;  dgate = scale * (sum over the gate's rows of G * p);
 *   dy = post'(scale * gate * G), and the norms' weight and bias gradients.
 *   r_out, y, stats : as block_norm wrote (read) them (r_out: r where y is NULL)
 *   dn      : [M][D] of dtype, NULL if and only if pre_norm is Q4_NORM_NONE
 *   dr_out  : [M][D] of r_dtype, or NULL for zeros; not NULL where dn is
 *   dr      : device out, [M][D] of r_dtype;  dy : device out, [M][D] of
 *             dtype (NULL if and only if y is NULL)
 *   dgate   : device out, [ceil(M / gate_rows)][D] of dtype, or NULL (gate
 *             NULL: must be NULL)
 *   pre_dw, pre_db, post_dw, post_db : device out, float [D], or NULL; NULL
 *             where the norm is Q4_NORM_NONE (else Q4_ERR_ARG)
 *   workspace: block_norm_backward_workspace_size(M, D, gate_rows) bytes.
 */
int64_t block_norm_backward_workspace_size(int64_t M, int64_t D, int64_t gate_rows);
int block_norm_backward(const void* y, const void* r_out, const float* stats, const void* dn, const void* dr_out,
                        int dtype, int r_dtype, int64_t M, int64_t D, int post_norm, const void* post_weight,
                        const void* post_bias, const void* gate, int64_t gate_rows, float scale, int pre_norm,
                        const void* pre_weight, void* dr, void* dy, void* dgate, float* pre_dw, float* pre_db,
                        float* post_dw, float* post_db, void* workspace, int64_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GEMV_Q4_AFFINE_AMD_Q4_BLOCK_H */
