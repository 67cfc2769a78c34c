"""Thin PyTorch binding of the operators of a residual block (include/ecc_train.h).

Features are channels last, ``[batch, *space, channels]`` or, for curves and other sequences, ``[batch, steps,
channels]``.  Every function takes tensors that live on a ROCm device and calls the C entry points on the current torch
stream; argument checks and autograd nodes are in csrc/ecc_torch_block.cpp, all arithmetic is in the HIP kernels.
Scratch comes from torch's allocator per call, so calls may run on any stream and be captured into a graph.  Strided
tensors are copied once.  Forward-mode derivatives and torch.jit.trace are refused, and gradients of gradients raise an
error.  A backward pass is not captured while a graph made on the default stream holds a leaf whose gradient it forms.
"""

from . import _torch
from ._lib import EccError
from .train import _ACTS

__all__ = ["residual_norm", "rms_norm", "gated_linear", "gated_recurrence", "EccError"]


def residual_norm(x, branch, gate=None, weight=None, branch_weight=None, norm_branch=True, scale=1.0, eps=1e-6):
    """What stands between two blocks of a residual network, in one pass: the norm after a block, its gate, the residual
    sum and the norm before the next block.

        y = scale * x + gate * n(branch) * branch_weight,   z = n(y) * weight,   n(v) = v / sqrt(mean(v^2) + eps)

    with the means over the channels of one position.  x: the residual stream, float32, float16 or bfloat16 [batch,
    *space, channels]; branch: the block's output, of x's shape and type, or 16-bit beside a float32 x; gate: [channels],
    or [batch, channels] for a gate per sample; gate, weight and branch_weight are float32 or branch's dtype, all alike,
    and 1 where they are None.  norm_branch=False leaves n(branch) out of y.

    Returns (y, z), y like x and z like branch.  Differentiable in the five tensors (see include/ecc_train.h).
    """
    return _torch.residual_norm(x, branch, gate, weight, branch_weight, scale, eps, norm_branch)


def rms_norm(x, weight=None, eps=1e-6, dtype=None):
    """The norm before the first block: x / sqrt(mean(x^2) + eps) * weight over the channels, [batch, *space, channels].

    weight: [channels], float32 or the result's dtype, or None (1); dtype: of the result, x's by default; a float32 x may
    have a 16-bit result.  Differentiable in x and weight.
    """
    return _torch.rms_norm(x, weight, eps, dtype)


def gated_linear(x, w_gate, w_up, b_gate=None, b_up=None, act="silu"):
    """Both projections of a gated feed-forward block, the activation and their product:

        h = act(x @ w_gate.T + b_gate) * (x @ w_up.T + b_up)

    x: float32, float16 or bfloat16 [*space, channels]; w_gate, w_up: [hidden, channels]; b_gate, b_up: [hidden] or None;
    all of x's type; act: "none", "relu", "silu" or "gelu".  Returns [*space, hidden], like x.  Sums are float32; the
    backward pass forms the projections again, so that nothing but the arguments is kept.  Differentiable in all five
    tensors (see include/ecc_train.h).
    """
    if act not in _ACTS:
        raise ValueError(f"act must be one of {sorted(_ACTS)} (got {act!r})")
    return _torch.gated_linear(x, w_gate, w_up, b_gate, b_up, _ACTS[act])


def gated_recurrence(x, gate, state=None, lengths=None):
    """A gated linear recurrence along the steps of a sequence, such as the thresholds of a curve:

        h_t = k_t h_(t-1) + (1 - k_t) x_t,   k_t = 1 / (1 + exp(-gate_t)),   h_(-1) = state

    x, gate: float32, float16 or bfloat16 [batch, steps, channels] of one type; state: float32 [batch, channels], or None
    (0); lengths: int64 [batch] on the device, how many steps each sequence has (all of them where None): what x and gate
    hold behind them is not read, and h is 0 there.

    Returns (h, last): h like x, and the float32 state after every sequence's last step, [batch, channels], which a next
    call takes as its state.  Differentiable in x, gate and state (see include/ecc_train.h).
    """
    return _torch.gated_recurrence(x, gate, state, lengths)
