"""Stacks of matrices that between them take every way a product of the direct
iteration is shared out (tests/test_orth_products_cpu.py holds the list to
that), and their iterates in float64 on the GPU."""

import torch

from tests.orth_bounds import COEFFICIENTS, E

# (batch, rows, cols): one tile of 64 to many, whole and shared; 128-tiles two a CU, whole and shared; one a CU ("deep");
# two to a workgroup, whole, shared and both, with an odd number of tile columns above the diagonal left out
STACKS = [(1, 70, 75), (1, 257, 771), (1, 1000, 790), (12, 257, 771), (32, 260, 257), (32, 129, 257), (24, 129, 645),
          (32, 129, 645), (8, 513, 520), (3, 769, 771), (1, 769, 1153), (6, 1537, 769), (40, 640, 800), (3, 385, 1925),
          (4, 1411, 1409), (4, 1411, 1000), (1, 1409, 1411), (1, 2817, 1409), (2, 1409, 2817), (1, 65, 195), (6, 193, 450)]


def orthogonal_on_device(g, steps=5, eps=1e-7, coefficients=COEFFICIENTS):
    """orth_bounds.orthogonal for one matrix on the GPU: the singular values, which its bound asks for at every step, are
    taken once and follow the scalar polynomial."""
    g = g.detach().double()
    if g.shape[0] > g.shape[1]:
        x, bound = orthogonal_on_device(g.T.contiguous(), steps, eps, coefficients)
        return x.T, bound
    a, b, c = coefficients
    x = g / (g.square().sum().sqrt() + eps)
    s = torch.linalg.eigvalsh((x @ x.T).cpu()).clamp_min(0).sqrt()
    unit = 2.0 ** -22 + 4 * g.shape[1] ** 0.5 * E
    bound = 2 * E * float(s.square().sum().sqrt())
    for _ in range(steps):
        r = float(s.max())
        t = torch.linspace(0, 1.01 * r, 1000, dtype=torch.float64)
        growth = float((a + 3 * b * t ** 2 + 5 * c * t ** 4).abs().max())
        size = abs(a) + 3 * abs(b) * r ** 2 + 5 * abs(c) * r ** 4
        bound = growth * bound + unit * size * float(s.square().sum().sqrt())
        gram = x @ x.T
        x = a * x + (b * gram + c * gram @ gram) @ x
        s = (s * (a + s ** 2 * (b + s ** 2 * c))).abs()
    return x, bound
