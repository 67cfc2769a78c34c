"""Trains a small network whose output is read through soft Euler characteristic curves.

A scalar volume goes through a 3 x 3 x 3 layer, group norm with an activation, a pointwise layer, and group norm read out
to a new scalar volume; the soft curve of that volume feeds a linear head.  The network learns to tell smooth random
volumes from rough ones.  Matrices are updated by ``muon_step`` (layers of one shape as one stack), vectors by plain
gradient steps.

    python examples/train_through_curves.py --steps 60
"""

import argparse
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import euler_characteristic_curves_amd as E  # noqa: E402

SIDE, CHANNELS, GROUPS, THRESHOLDS, LAM = 24, 32, 8, 64, 8.0


def volumes(batch, gen, device):
    """Random volumes [batch, SIDE, SIDE, SIDE] of unit variance, and 1 where they were smoothed."""
    label = torch.randint(0, 2, (batch,), generator=gen).to(device)
    noise = torch.randn(batch, 1, SIDE, SIDE, SIDE, generator=gen).to(device)
    smooth = F.avg_pool3d(noise, 3, stride=1, padding=1, count_include_pad=False)
    x = torch.where(label.bool()[:, None, None, None, None], smooth, noise)[:, 0]
    return x / x.std(dim=(1, 2, 3), keepdim=True), label


def taps(x):
    """The 27 neighbours of every voxel, [batch, SIDE, SIDE, SIDE, 27]."""
    p = F.pad(x[:, None], (1,) * 6, mode="replicate")[:, 0]
    n = SIDE
    return torch.stack([p[:, a:a + n, b:b + n, c:c + n] for a in range(3) for b in range(3) for c in range(3)], dim=-1)


class Network:
    def __init__(self, gen, device):
        rnd = lambda *s: torch.randn(*s, generator=gen).to(device)  # noqa: E731
        c = CHANNELS
        self.matrices = [rnd(27, c) / 27 ** 0.5, rnd(c, c) / c ** 0.5, rnd(THRESHOLDS, 2) / THRESHOLDS ** 0.5]
        one, zero = torch.ones(c, device=device), torch.zeros(c, device=device)
        self.vectors = [one.clone(), zero.clone(), one.clone(), zero.clone(), rnd(c) / c ** 0.5,
                        torch.zeros(1, device=device), torch.zeros(2, device=device)]
        for t in self.matrices + self.vectors:
            t.requires_grad_()
        self.buffers = [torch.zeros_like(t) for t in self.matrices]
        self.tau = torch.linspace(-2.5, 2.5, THRESHOLDS, device=device)

    def __call__(self, x):
        first, mix, head = self.matrices
        w1, b1, w2, b2, readout, offset, bias = self.vectors
        h = E.group_norm_act(taps(x) @ first, GROUPS, w1, b1, act="silu")
        field = E.group_norm_readout(h @ mix, GROUPS, w2, b2, readout, offset, act="gelu")
        curve = E.soft_ecc_batched(field, self.tau, LAM) / SIDE ** 2
        return curve @ head + bias

    def step(self, loss, lr):
        grads = torch.autograd.grad(loss, self.matrices + self.vectors)
        k = len(self.matrices)
        with torch.no_grad():
            E.muon_step(self.matrices, [g.contiguous() for g in grads[:k]], self.buffers, lr=lr)
            for t, g in zip(self.vectors, grads[k:]):
                t.sub_(lr * g)


def train(steps, batch=16, lr=0.02, seed=0, device="cuda", report=None):
    """Losses of the steps."""
    gen = torch.Generator().manual_seed(seed)
    net, losses = Network(gen, device), []
    for i in range(steps):
        x, label = volumes(batch, gen, device)
        loss = F.cross_entropy(net(x), label)
        net.step(loss, lr)
        losses.append(float(loss.detach()))
        if report and (i % 10 == 0 or i + 1 == steps):
            report(f"step {i}: loss {losses[-1]:.4f}")
    return losses


if __name__ == "__main__":
    parser = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    parser.add_argument("--steps", type=int, default=60)
    train(parser.parse_args().steps, report=lambda line: print(line, flush=True))
