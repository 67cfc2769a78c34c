/*
 * ecc_train.h -- C ABI of the operators in libecc_mi355.so that train a
 * network through the curves: group norm with an activation over
 * channels-last features, the same norm read out to the scalar grid a curve
 * takes, Newton-Schulz orthogonalisation, and the momentum update built on it.
 *
 * Conventions are those of ecc.h (device pointers owned by the caller, work
 * enqueued on `stream`, status codes, ecc_last_error), except the workspace:
 *   - `ws` is scratch of at least the bytes its size function gives, 256-byte
 *     aligned.  It need not be cleared before a call and holds nothing after
 *     it; calls that overlap in time must not share one.
 *   - The library allocates nothing and clears nothing with a memset, so every
 *     call may be captured into a graph.
 * Every output is written in full, and its value does not depend on
 * scheduling: sums are formed in a fixed order and no floating-point atomics
 * are used.
 */
#ifndef ECC_TRAIN_MI355_H
#define ECC_TRAIN_MI355_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* status codes beyond those of ecc.h */
#define ECC_E_GROUPS 9 /* groups < 1 or channels not a multiple of groups     */
#define ECC_E_ACT 10   /* act is not one of ECC_ACT_*                         */
#define ECC_E_VALUE 11 /* a scalar argument is out of range or not finite     */

/* element types of features, parameters and matrices */
#define ECC_T_F32 0
#define ECC_T_F16 1
#define ECC_T_BF16 2

/* activations */
#define ECC_ACT_NONE 0
#define ECC_ACT_RELU 1
#define ECC_ACT_SILU 2 /* u / (1 + exp(-u))                                   */
#define ECC_ACT_GELU 3 /* u Phi(u), Phi the normal distribution function      */
/* (at an infinite u, their limits: infinity or 0, with slope 1 or 0)         */

#define ECC_MAX_CHANNELS 8192          /* of the norm                         */
#define ECC_MAX_READOUT_CHANNELS 1024  /* of the norm read out to a grid      */
#define ECC_MAX_NORM_BATCH 32768
#define ECC_MAX_MATRIX 32768           /* rows and columns of one matrix      */
#define ECC_MAX_NS_STEPS 64

/*
 * Group norm with an activation, channels last.
 *   x       device, dtype elements, [batch][voxels][channels]
 *   weight, bias  device, pdtype elements, [channels]; NULL stands for 1 / 0
 *   y       device, dtype elements, x's shape (must not overlap x):
 *           xhat = (x - mean) / sqrt(var + eps) over the voxels and the
 *           channels / groups channels of one group of one sample (var with
 *           the divisor voxels * channels / groups), u = xhat * weight + bias,
 *           y = act(u)
 *   stats   device float32 [batch][groups][3]: the mean, 1/sqrt(var + eps), and
 *           what rounding to float32 left of the mean; written by the forward
 *           call and read by the backward one
 *   pdtype  ECC_T_F32 or dtype
 * Moments are accumulated in float32 about a pivot per thread and joined in
 * float64 about a value of the group, and x - mean takes the mean with more
 * digits than float32 has, so that values a few ulps apart are normalised to
 * float32's digits too; everything else is float32, rounded once to dtype.
 * x and y need only the alignment of their elements.  Two kernel launches,
 * three or four where the features are many.
 */
int ecc_norm_fwd(const void* x, int dtype, int64_t batch, int64_t voxels, int64_t channels, int64_t groups,
                 const void* weight, const void* bias, int pdtype, int act, float eps, void* y, float* stats,
                 void* ws, size_t ws_bytes, void* stream);

/*
 * Its backward pass.  grad_y: dL/dy, dtype elements.  grad_x (dtype),
 * grad_weight and grad_bias (pdtype) are OVERWRITTEN; each may be NULL (not
 * wanted), but not all of them.  With
 * du = grad_y act'(u) (act'(0) = 0 for relu),
 *   grad_bias = sum du, grad_weight = sum du xhat   over samples and voxels,
 *   grad_x = rstd (du weight - m1 - xhat m2), m1 and m2 the means over the
 *   group of du weight and of du weight xhat.
 * Three or four kernel launches.
 */
int ecc_norm_bwd(const void* x, int dtype, int64_t batch, int64_t voxels, int64_t channels, int64_t groups,
                 const void* weight, const void* bias, int pdtype, int act, const float* stats, const void* grad_y,
                 void* grad_x, void* grad_weight, void* grad_bias, void* ws, size_t ws_bytes, void* stream);

/*
 * The same norm contracted to a scalar grid:
 *   field[b][v] = offset + sum over c of readout[c] act(u[b][v][c]),
 * float32 [batch][voxels], ready for a curve.  readout: [channels], offset:
 * [1] or NULL (0), both pdtype.  channels <= ECC_MAX_READOUT_CHANNELS.  The
 * activated features are never written.
 */
int ecc_norm_readout_fwd(const void* x, int dtype, int64_t batch, int64_t voxels, int64_t channels, int64_t groups,
                         const void* weight, const void* bias, const void* readout, const void* offset, int pdtype,
                         int act, float eps, float* field, float* stats, void* ws, size_t ws_bytes, void* stream);

/*
 * Its backward pass from grad_field = dL/dfield, float32 [batch][voxels]:
 * grad_readout = sum grad_field act(u), grad_offset = sum grad_field, and the
 * gradients of ecc_norm_bwd for grad_y = grad_field readout.  Gradients that
 * are not wanted are NULL.
 */
int ecc_norm_readout_bwd(const void* x, int dtype, int64_t batch, int64_t voxels, int64_t channels, int64_t groups,
                         const void* weight, const void* bias, const void* readout, int pdtype, int act,
                         const float* stats, const float* grad_field, void* grad_x, void* grad_weight,
                         void* grad_bias, void* grad_readout, void* grad_offset, void* ws, size_t ws_bytes,
                         void* stream);

/* Workspace bytes of the four calls above (0 for invalid sizes). */
size_t ecc_norm_workspace_bytes(int64_t batch, int64_t voxels, int64_t channels, int64_t groups);

/*
 * Newton-Schulz orthogonalisation of a stack of matrices g[batch][rows][cols]
 * (dtype), each on its own: X = g / (|g|_F + eps), then `steps` times
 *   A = X X^T,  X <- a X + (b A + c A A) X
 * (with X^T in place of X where rows > cols), written to out (dtype, g's
 * shape; g itself, or memory that does not overlap it).  The singular vectors stay, the singular values are
 * driven towards 1 by the polynomial a s + b s^3 + c s^5.
 * The norm is summed in float64.  Products take operands of 22 significant bits
 * (pairs of float16) and sum in float32; where the short side is at most 64, or
 * small beside the long one, and the steps let an error of X X^T grow by less
 * than 2^26, X X^T is carried through the steps in float64 instead and the long
 * side passed twice only.  Either way the result has the error of float32
 * arithmetic, rounded once to dtype, in every row and column down to 1e-5 of the
 * largest; the pairs' last bit leaves an error of up to 1e-10 of the largest in
 * smaller ones.  (Short sides up to 64 that are carried have no such limit.)
 * Refused with ECC_E_VALUE: steps outside [1, ECC_MAX_NS_STEPS], eps < 0, a
 * coefficient that is not finite, and coefficients under which a singular
 * value in [0, 1] leaves [-16, 16] within the steps.
 */
int ecc_orthogonalize(const void* g, int dtype, int64_t batch, int64_t rows, int64_t cols, int32_t steps, float eps,
                      float a, float b, float c, void* out, void* ws, size_t ws_bytes, void* stream);

/*
 * Momentum, orthogonalisation and update of a stack of matrices, in place:
 *   buffer <- momentum buffer + (1 - momentum) grad               (float32)
 *   u = nesterov ? momentum buffer + (1 - momentum) grad : buffer
 *   param <- (1 - lr weight_decay) param - lr scale orthogonalize(u)
 * param: pdtype, grad: gdtype, buffer: float32, all [batch][rows][cols]; none
 * overlaps another.
 * Refused with ECC_E_VALUE besides the above: lr, momentum, weight_decay or
 * scale not finite, or momentum, 1 - lr weight_decay or lr scale beyond float32.
 */
int ecc_muon_step(void* param, int pdtype, const void* grad, int gdtype, float* buffer, int64_t batch, int64_t rows,
                  int64_t cols, double lr, double momentum, int nesterov, double weight_decay, double scale,
                  int32_t steps, float eps, float a, float b, float c, void* ws, size_t ws_bytes, void* stream);

/* Workspace bytes of the two calls above (0 for invalid sizes). */
size_t ecc_orth_workspace_bytes(int64_t batch, int64_t rows, int64_t cols);

#ifdef __cplusplus
}
#endif

#endif /* ECC_TRAIN_MI355_H */
