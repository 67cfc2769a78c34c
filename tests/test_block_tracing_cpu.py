"""Traced calls of the operators that the binding holds are refused: a trace would hold their results' allocation alone."""

import pytest
import torch

import euler_characteristic_curves_amd as E

X, W, V = torch.zeros(2, 3, 8), torch.zeros(5, 8), torch.zeros(8)
CALLS = {"residual": lambda x: E.residual_norm(x, x, V, V)[1], "rms": lambda x: E.rms_norm(x, V),
         "linear": lambda x: E.gated_linear(x, W, W), "recurrence": lambda x: E.gated_recurrence(x, x)[0]}


@pytest.mark.parametrize("which", CALLS)
def test_tracing_is_refused(which):
    with pytest.raises(NotImplementedError, match="cannot be traced"):
        torch.jit.trace(CALLS[which], (X,), check_trace=False)
    with pytest.raises(ValueError, match="ROCm device"):   # outside of a trace, the call's own checks
        CALLS[which](X)


@pytest.mark.gpu
@pytest.mark.parametrize("which", [*CALLS, "norm", "readout"])
def test_tracing_is_refused_on_the_gpu(which):
    if not torch.cuda.is_available():
        pytest.skip("no ROCm GPU visible")
    x, w, v = X.cuda(), W.cuda(), V.cuda()
    calls = {"residual": lambda x: E.residual_norm(x, x, v, v)[1], "rms": lambda x: E.rms_norm(x, v),
             "linear": lambda x: E.gated_linear(x, w, w), "recurrence": lambda x: E.gated_recurrence(x, x)[0],
             "norm": lambda x: E.group_norm_act(x, 2, v, v), "readout": lambda x: E.group_norm_readout(x, 2, v, v, v)}
    with pytest.raises(NotImplementedError, match="cannot be traced"):
        torch.jit.trace(calls[which], (x,), check_trace=False)
    assert torch.isfinite(calls[which](x)).all()
