"""Thin PyTorch binding of the training operators (include/ecc_train.h).

Features are channels last, ``[batch, *space, channels]``; every function takes
tensors that live on a ROCm device, checks them, and calls the C entry points
on the current torch stream (the norms through their autograd nodes in
csrc/ecc_torch.cpp).  All arithmetic happens in the HIP kernels.
Scratch comes from torch's allocator per call, so calls may run on any stream
and be captured into a graph.  torch.jit.trace is refused by the norms.
"""

import torch

from . import _lib, _torch
from ._lib import EccError, check, lib
from .ecc import _dev_tensor, _ptr, _stream

__all__ = ["group_norm_act", "group_norm_readout", "orthogonalize", "muon_step", "EccError"]

_DTYPES = {torch.float32: _lib.ECC_T_F32, torch.float16: _lib.ECC_T_F16, torch.bfloat16: _lib.ECC_T_BF16}
_ACTS = {"none": _lib.ECC_ACT_NONE, "relu": _lib.ECC_ACT_RELU, "silu": _lib.ECC_ACT_SILU, "gelu": _lib.ECC_ACT_GELU}


def _on_device(t):
    """Runs the call on the tensor's GPU (a no-op where that is the current one)."""
    return torch.cuda.device(t.device) if t.get_device() != torch.cuda.current_device() else _NULL_CONTEXT


class _NullContext:
    def __enter__(self):
        return None

    def __exit__(self, *exc):
        return False


_NULL_CONTEXT = _NullContext()


class _NormPlan:
    """What a norm call needs besides its tensors, checked.  Strided tensors are made contiguous where the kernels are
    called, once."""

    __slots__ = ("sizes", "dtype", "pdtype", "act", "nbytes")

    def __init__(self, x, groups, weight, bias, act, readout=None, offset=None, read=False):
        _dev_tensor(x, "x", strided=True)
        if x.dtype not in _DTYPES:
            raise TypeError(f"x dtype {x.dtype} not supported (float32, float16 or bfloat16)")
        if x.dim() < 3:
            raise ValueError("x must be [batch, *space, channels]")
        if act not in _ACTS:
            raise ValueError(f"act must be one of {sorted(_ACTS)} (got {act!r})")
        shape = x.shape
        B, C = shape[0], shape[-1]
        if isinstance(groups, bool) or not isinstance(groups, int):
            raise TypeError(f"groups must be an int (got {type(groups).__name__})")
        if groups < 1 or C < 1 or C % groups:
            raise ValueError(f"groups={groups} does not divide channels={C}")
        if read and readout is None:
            raise TypeError("readout must be a torch.Tensor")
        pdtype = None
        for t, name, n in ((weight, "weight", C), (bias, "bias", C), (readout, "readout", C), (offset, "offset", 1)):
            if t is None:
                continue
            _dev_tensor(t, name, None, x.device, strided=True)
            if t.dim() != 1 or t.numel() != n:
                raise ValueError(f"{name} must be [{n}] (got {list(t.shape)})")
            if t.dtype != torch.float32 and t.dtype != x.dtype:
                raise TypeError(f"{name} must be torch.float32 or x's {x.dtype} (got {t.dtype})")
            if pdtype is not None and t.dtype != pdtype:
                raise TypeError(f"{name} is {t.dtype}, the parameters before it {pdtype}")
            pdtype = t.dtype
        numel = x.numel()
        self.sizes = (B, numel // (B * C) if B else 0, C, groups)
        self.dtype, self.act = _DTYPES[x.dtype], _ACTS[act]
        self.pdtype = _DTYPES[pdtype or torch.float32]
        self.nbytes = 0
        if numel:
            self.nbytes = lib.ecc_norm_workspace_bytes(*self.sizes)
            if not self.nbytes:
                raise EccError(_lib.ECC_E_SHAPE, "group norm: " + lib.ecc_last_error().decode(errors="replace"))


def _norm(x, groups, weight, bias, readout, offset, act, eps, read):
    plan = _NormPlan(x, groups, weight, bias, act, readout, offset, read)
    return _torch.norm(x, weight, bias, readout, offset, plan.sizes, plan.dtype, plan.pdtype, plan.act, plan.nbytes,
                       float(eps), read)


def group_norm_act(x, groups, weight=None, bias=None, act="none", eps=1e-5):
    """act(group_norm(x) * weight + bias) over channels-last features, differentiable in x, weight and bias.

    x: float32, float16 or bfloat16 [batch, *space, channels]; weight and bias: [channels], float32 or x's dtype, or
    None (1 and 0); act: "none", "relu", "silu" or "gelu".  Returns a tensor like x (see include/ecc_train.h).  Forward-mode
    derivatives are refused.
    """
    return _norm(x, groups, weight, bias, None, None, act, eps, False)


def group_norm_readout(x, groups, weight, bias, readout, offset=None, act="none", eps=1e-5):
    """The features group_norm_act gives, contracted with ``readout`` [channels] plus ``offset`` [1] to the float32 grid
    [batch, *space] that a curve takes.  Differentiable in x and all four parameters; the features are not stored."""
    return _norm(x, groups, weight, bias, readout, offset, act, eps, True)


# ------------------------------------------------- orthogonalised updates
_COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def _matrix_sizes(t, name):
    """(batch, rows, cols) of a matrix or a stack of matrices."""
    if t.dim() not in (2, 3):
        raise ValueError(f"{name} must be [rows, cols] or [batch, rows, cols] (got {list(t.shape)})")
    return (1, *t.shape) if t.dim() == 2 else tuple(t.shape)


def _matrix_dtype(t, name):
    if t.dtype not in _DTYPES:
        raise TypeError(f"{name} dtype {t.dtype} not supported (float32, float16 or bfloat16)")
    return _DTYPES[t.dtype]


def _overlap(a, b):
    """Whether two contiguous tensors share memory."""
    x, y = a.data_ptr(), b.data_ptr()
    return x < y + b.numel() * b.element_size() and y < x + a.numel() * a.element_size()


def _orth_bytes(sizes):
    nbytes = lib.ecc_orth_workspace_bytes(*sizes)
    if not nbytes:
        raise EccError(_lib.ECC_E_SHAPE, "orthogonalize: " + lib.ecc_last_error().decode(errors="replace"))
    return nbytes


def _polynomial(coefficients):
    a, b, c = coefficients
    return float(a), float(b), float(c)


def _whole(steps):
    """steps as an int that fits the C argument; one that does not stays out of range there."""
    n = int(steps)
    if isinstance(steps, bool) or n != steps:
        raise TypeError(f"steps must be a whole number (got {steps!r})")
    return max(-1, min(n, 2 ** 31 - 1))


def orthogonalize(g, steps=5, eps=1e-7, coefficients=_COEFFICIENTS, out=None):
    """The Newton-Schulz iterate of a matrix, or of each matrix of a stack (see ecc_orthogonalize in
    include/ecc_train.h): g with its singular values driven towards 1.  Not differentiable.

    g: float32, float16 or bfloat16, [rows, cols] or [batch, rows, cols]; out: a tensor like g, written in place; it is
    g itself or has no memory in common with it.
    """
    g, given = g.detach(), out is not None
    if not given:
        g = g.contiguous()
    _dev_tensor(g, "g")
    dtype, sizes = _matrix_dtype(g, "g"), _matrix_sizes(g, "g")
    if not given:
        out = torch.empty_like(g)
    _dev_tensor(out, "out", g.dtype, g.device)
    if out.shape != g.shape:
        raise ValueError("out must have g's shape")
    if out.data_ptr() != g.data_ptr() and _overlap(out, g):
        raise ValueError("out shares a part of g's memory: workgroups would write what others have yet to read")
    a, b, c = _polynomial(coefficients)
    steps = _whole(steps)
    if not g.numel():
        return out
    with _on_device(g):
        nbytes = _orth_bytes(sizes)
        if given:  # a backward pass that saved it is to notice
            torch.autograd.graph.increment_version(out)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=g.device)
        check(lib.ecc_orthogonalize(_ptr(g), dtype, *sizes, steps, float(eps), a, b, c, _ptr(out), _ptr(ws), nbytes,
                                    _stream(g).cuda_stream), "ecc_orthogonalize")
    return out


def muon_step(params, grads, buffers, lr, momentum=0.95, nesterov=True, weight_decay=0.0, scale=None, steps=5, eps=1e-7,
              coefficients=_COEFFICIENTS):
    """One step of momentum with orthogonalised updates, in place on ``params`` and ``buffers`` (see ecc_muon_step in
    include/ecc_train.h).

    params, grads, buffers: sequences of one length; entry i of each is [rows, cols] or a stack [batch, rows, cols] of
    matrices (layers of one shape), contiguous, without memory in common; buffers are float32.  scale: factor of the
    update, by default sqrt(max(1, rows / cols)).  Every argument is checked before anything is changed.
    """
    params, grads, buffers = list(params), list(grads), list(buffers)
    if not len(params) == len(grads) == len(buffers):
        raise ValueError(f"{len(params)} params, {len(grads)} grads, {len(buffers)} buffers")
    a, b, c = _polynomial(coefficients)
    steps = _whole(steps)
    calls = []
    for p, g, m in zip(params, grads, buffers):
        _dev_tensor(p, "param")
        _dev_tensor(g, "grad", None, p.device)
        _dev_tensor(m, "buffer", torch.float32, p.device)
        sizes = _matrix_sizes(p, "param")
        if g.shape != p.shape or m.shape != p.shape:
            raise ValueError(f"param {list(p.shape)}, grad {list(g.shape)} and buffer {list(m.shape)} must agree")
        for t, other, names in ((p, g, "param and grad"), (p, m, "param and buffer"), (g, m, "grad and buffer")):
            if _overlap(t, other):
                raise ValueError(f"{names} share memory")
        calls.append((p, _matrix_dtype(p, "param"), g, _matrix_dtype(g, "grad"), m, sizes,
                      _orth_bytes(sizes) if p.numel() else 0))
    for p, pdtype, g, gdtype, m, sizes, nbytes in calls:
        if not nbytes:
            continue
        s = float(scale) if scale is not None else max(1.0, sizes[1] / sizes[2]) ** 0.5
        with _on_device(p):
            ws = torch.empty(nbytes, dtype=torch.uint8, device=p.device)
            check(lib.ecc_muon_step(_ptr(p), pdtype, _ptr(g), gdtype, _ptr(m), *sizes, float(lr), float(momentum),
                                    1 if nesterov else 0, float(weight_decay), s, steps, float(eps), a, b, c,
                                    _ptr(ws), nbytes, _stream(p).cuda_stream), "ecc_muon_step")
        torch.autograd.graph.increment_version(p)
        torch.autograd.graph.increment_version(m)
