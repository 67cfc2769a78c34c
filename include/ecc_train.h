/*
 * ecc_train.h -- C ABI of the operators in libecc_mi355.so that train a
 * network through the curves: group norm with an activation over
 * channels-last features, the same norm read out to the scalar grid a curve
 * takes, Newton-Schulz orthogonalisation, and the momentum update built on it;
 * and those of a residual block over curves or other channels-last features:
 * the norms around a block with its gate and residual scale, the gated pair of
 * projections of a feed-forward block, and a gated linear recurrence along the
 * steps of a sequence.
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
#define ECC_MAX_RECURRENCE_CHANNELS 1048576

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

/*
 * The norms after a block and before the next one, with the block's gate and
 * the residual scale between them.  A row is one position of one sample, of
 * `channels` (<= ECC_MAX_CHANNELS) numbers; there are batch x inner of them.
 *   x       device, xdtype elements, [batch][inner][channels]: the residual stream
 *   branch  device, dtype elements, of x's shape: the block's output; NULL for
 *           the norm alone, z of x (gate, branch_weight and norm_branch are
 *           then NULL and 0, and scale is not used)
 *   gate    pdtype elements, [channels], or [batch][channels] where
 *           gate_per_sample (batch <= ECC_MAX_NORM_BATCH); NULL stands for 1
 *   weight, branch_weight  pdtype elements, [channels]; NULL stands for 1
 *   xdtype  ECC_T_F32 or dtype; pdtype: ECC_T_F32 or dtype
 * With n(v) = v / sqrt(mean v^2 + eps) over a row,
 *   y = scale x + gate n(branch) branch_weight   (xdtype; with branch in place
 *       of n(branch) unless norm_branch),
 *   z = n(y) weight                              (dtype; y as it was before rounding).
 * stats: float32 [batch][inner][2], the factors 1 / sqrt(..) of both norms for
 * the backward pass, or NULL.  No output overlaps an input.  One launch, no
 * workspace.
 * Squares are summed in float64, everything else is float32, rounded once (so
 * are the factors: beyond a root mean square of 2^126 they have fewer bits, below
 * 2^-128 with eps = 0 they are infinite).
 */
int ecc_residual_norm_fwd(const void* x, int xdtype, const void* branch, int dtype, int64_t batch, int64_t inner,
                          int64_t channels, const void* gate, int gate_per_sample, const void* weight,
                          const void* branch_weight, int pdtype, int norm_branch, float scale, float eps, void* y, void* z,
                          float* stats, void* stream);

/*
 * Its backward pass.  grad_y (xdtype), grad_z (dtype): either may be NULL (0).
 * grad_x (xdtype), grad_branch (dtype), grad_gate, grad_weight and
 * grad_branch_weight (pdtype, of their arguments' shapes) are OVERWRITTEN; each
 * may be NULL (not wanted), but not all of them.  One launch, two where a
 * parameter's gradient is wanted.
 */
int ecc_residual_norm_bwd(const void* x, int xdtype, const void* branch, int dtype, int64_t batch, int64_t inner,
                          int64_t channels, const void* gate, int gate_per_sample, const void* weight,
                          const void* branch_weight, int pdtype, int norm_branch, float scale, const float* stats,
                          const void* grad_y, const void* grad_z, void* grad_x, void* grad_branch, void* grad_gate,
                          void* grad_weight, void* grad_branch_weight, void* ws, size_t ws_bytes, void* stream);

/* Workspace bytes of the backward pass (0 for invalid sizes). */
size_t ecc_residual_norm_workspace_bytes(int64_t batch, int64_t inner, int64_t channels, int gate_per_sample);

/*
 * The gated linear recurrence along a sequence's steps (the thresholds of a
 * curve, say): with k_t = 1 / (1 + exp(-gate_t)),
 *   h_t = k_t h_(t-1) + (1 - k_t) x_t,  h_(-1) = state, for every channel.
 *   x, gate  device, dtype elements, [batch][steps][channels];
 *            channels <= ECC_MAX_RECURRENCE_CHANNELS, batch < 2^31
 *   state    device float32 [batch][channels]; NULL stands for 0
 *   lengths  device int64 [batch], or NULL: sequence b has the steps before
 *            lengths[b] (taken as 0 below it and as `steps` beyond them); x and
 *            gate behind them are not read, h there is 0, and the state, infinite
 *            or not, stays as it is
 *   h        dtype, x's shape
 *   last     float32 [batch][channels]: the state after the last step (the
 *            initial one where there is none), to be carried to a next call
 *   saved    float32, ecc_gated_recurrence_saved_bytes: states that the backward
 *            pass starts from; NULL where there will be none
 * No output overlaps an input.  States are float32.  A step is formed from
 * x_t - h_(t-1): where that is beyond float32, an infinite x or state among
 * others, h is not finite from there on.  One launch, three where batch x
 * channels is small beside the card and the sequence is cut into parts, and one
 * for every 2^24 - 1 sequences where there are more.
 */
int ecc_gated_recurrence_fwd(const void* x, const void* gate, int dtype, int64_t batch, int64_t steps, int64_t channels,
                             const float* state, const int64_t* lengths, void* h, float* last, float* saved, void* ws,
                             size_t ws_bytes, void* stream);

/*
 * Its backward pass.  grad_h (dtype; not read behind a sequence's length) and
 * grad_last (float32): either may be NULL (0).  grad_x, grad_gate (dtype; 0
 * behind a sequence's length) and grad_state (float32) are OVERWRITTEN; each may
 * be NULL (not wanted), but not all of them.
 */
int ecc_gated_recurrence_bwd(const void* x, const void* gate, int dtype, int64_t batch, int64_t steps, int64_t channels,
                             const int64_t* lengths, const float* saved, const void* grad_h, const float* grad_last,
                             void* grad_x, void* grad_gate, float* grad_state, void* ws, size_t ws_bytes, void* stream);

/* Workspace bytes of the two calls above, and the bytes of `saved` (0 for invalid sizes). */
size_t ecc_gated_recurrence_workspace_bytes(int64_t batch, int64_t steps, int64_t channels, int dtype);
size_t ecc_gated_recurrence_saved_bytes(int64_t batch, int64_t steps, int64_t channels, int dtype);

/*
 * The gated pair of projections of a feed-forward block:
 *   h = act(x w_gate^T + b_gate) (x w_up^T + b_up)
 *   x             device, dtype elements, [rows][channels]
 *   w_gate, w_up  dtype, [hidden][channels]
 *   b_gate, b_up  dtype, [hidden]; each may be NULL (0)
 *   act           of the first projection, ECC_ACT_*
 *   h             dtype, [rows][hidden]; overlaps no input
 * channels, hidden <= ECC_MAX_MATRIX.  Sums are float32, h is rounded once.  One
 * launch; one more, and a workspace, only where rows > 64 and x's rows are not
 * whole 16-byte chunks (ws may be NULL otherwise).
 */
int ecc_gated_linear_fwd(const void* x, int dtype, int64_t rows, int64_t channels, int64_t hidden, const void* w_gate,
                         const void* w_up, const void* b_gate, const void* b_up, int act, void* h, void* ws, size_t ws_bytes,
                         void* stream);

/*
 * Its backward pass from grad_h = dL/dh (dtype, [rows][hidden]); the two
 * projections are formed again.  With a and b the projections,
 *   da = grad_h b act'(a), db = grad_h act(a)   (act'(0) = 0 for relu), float32,
 *   or where dtype has 16 bits two numbers of dtype, with twice its bits, as
 *   operands of
 *   grad_x = da w_gate + db w_up, grad_w_gate = da^T x, grad_w_up = db^T x;
 *   grad_b_gate = sum da, grad_b_up = sum db, of the values before that rounding.
 * In float16 da and db may be up to 2^20, and are kept to 2^-32 at least.
 * All of dtype and OVERWRITTEN; each may be NULL (not wanted), but not all.
 */
int ecc_gated_linear_bwd(const void* x, int dtype, int64_t rows, int64_t channels, int64_t hidden, const void* w_gate,
                         const void* w_up, const void* b_gate, const void* b_up, int act, const void* grad_h, void* grad_x,
                         void* grad_w_gate, void* grad_w_up, void* grad_b_gate, void* grad_b_up, void* ws, size_t ws_bytes,
                         void* stream);

/* Workspace bytes of either call (0 for invalid sizes). */
size_t ecc_gated_linear_workspace_bytes(int64_t rows, int64_t channels, int64_t hidden, int dtype, int backward);

#ifdef __cplusplus
}
#endif

#endif /* ECC_TRAIN_MI355_H */
