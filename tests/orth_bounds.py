"""Newton-Schulz orthogonalisation in float64, with a bound in the Frobenius
norm of what float32 arithmetic may leave of it.

A step maps X to f(X), f(s) = a s + b s^3 + c s^5 on the singular values; an
error in X grows at most by max |f'| over the attained singular values (the
Frobenius norm of the derivative of an odd matrix function).  The step itself
adds, relative to |X|_F and to the sizes |a| + 3|b| r^2 + 5|c| r^4 of its terms
(r the largest singular value), the rounding of its operands, 2^-22, and of
sums of K float32 products, whose errors add up at random: 4 sqrt(K) 2^-24.
"""

import torch

E = 2.0 ** -24
HALF = {torch.float32: E, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def orthogonal(g, steps=5, eps=1e-7, coefficients=COEFFICIENTS):
    """(iterate, Frobenius bound) of one matrix, float64 on the CPU."""
    g = g.detach().double().cpu()
    if g.shape[0] > g.shape[1]:
        x, bound = orthogonal(g.T, steps, eps, coefficients)
        return x.T, bound
    a, b, c = coefficients
    x = g / (torch.linalg.matrix_norm(g) + eps)
    K = max(g.shape)
    unit = 2.0 ** -22 + 4 * K ** 0.5 * E
    bound = 2 * E * float(torch.linalg.matrix_norm(x))
    for _ in range(steps):
        s = torch.linalg.svdvals(x)
        r = float(s.max())
        t = torch.linspace(0, 1.01 * r, 1000, dtype=torch.float64)
        growth = float((a + 3 * b * t ** 2 + 5 * c * t ** 4).abs().max())
        size = abs(a) + 3 * abs(b) * r ** 2 + 5 * abs(c) * r ** 4
        bound = growth * bound + unit * size * float(torch.linalg.matrix_norm(x))
        gram = x @ x.T
        x = a * x + (b * gram + c * gram @ gram) @ x
    return x, bound


def check(got, g, dtype, **kw):
    """Asserts that one matrix agrees with its iterate; returns error over bound."""
    want, bound = orthogonal(g, **kw)
    got = got.detach().double().cpu()
    assert got.shape == want.shape
    total = bound + HALF[dtype] * float(torch.linalg.matrix_norm(want)) + 1e-7 * HALF[dtype] * want.numel() ** 0.5
    err = float(torch.linalg.matrix_norm(got - want))
    assert err <= total, (err, total)
    return err / total
