"""The gradients of residual_norm's parameters where a thread has many rows, all different: sums over turns, over runs of
turns in LDS, over the rows of a workgroup and over workgroups, against float64; and rms_norm by itself."""

import pytest
import torch

import euler_characteristic_curves_amd as E
from tests.block_bounds import residual
from tests.gpu_util import banner, need_gpu
from tests.norm_bounds import rounded, worst
from tests.norm_bounds import E as STEP
from tests.test_gpu_residual import IDS, TYPES, make

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def parameter_sums(t, gy, gz, eps=1e-6):
    """{name: (value, bound)} of the three parameters' gradients, in float64 on the GPU, with the bounds of
    block_bounds.residual but for the sums over rows: 16 rows of a run, 16 runs, and a tree over at most 256 rows, 40
    roundings, and every 2^-24 once more for the product."""
    x, b, gy, gz = (v.double() for v in (t["x"], t["branch"], gy, gz))
    x, b, gy, gz = (v.reshape(x.shape[0], -1, x.shape[-1]) for v in (x, b, gy, gz))
    g, w, wb = (t[k].double() for k in ("gate", "weight", "branch_weight"))
    per_sample = g.dim() == 2
    if per_sample:
        g = g[:, None]

    def rms(v):
        return 1 / torch.sqrt((v * v).mean(dim=-1, keepdim=True) + eps)

    hb = b * rms(b)
    n = hb * wb
    y = x + g * n
    y_ = 4 * STEP * (g * n).abs() + STEP * (x.abs() + y.abs())
    ry = rms(y)
    rel = (y.abs() * y_).sum(dim=-1, keepdim=True) / (y * y).sum(dim=-1, keepdim=True) + 2 * STEP
    hy = y * ry
    hy_ = y_ * ry + hy.abs() * (rel + STEP)
    q = gz * w
    m = (q * hy).mean(dim=-1, keepdim=True)
    m_ = (q.abs() * hy_ + 30 * STEP * (q * hy).abs()).mean(dim=-1, keepdim=True)
    inner = q - hy * m
    inner_ = 3 * STEP * (q.abs() + (hy * m).abs()) + hy_ * m.abs() + hy.abs() * m_
    dy = gy + ry * inner
    dy_ = ry * (inner_ + (rel + 2 * STEP) * inner.abs()) + STEP * dy.abs()
    out = {}
    for name, term, term_ in (("gate", dy * n, dy_ * n.abs() + 4 * STEP * (dy * n).abs()), ("weight", gz * hy, gz.abs() * hy_),
                              ("branch_weight", dy * g * hb, dy_ * (g * hb).abs() + 4 * STEP * (dy * g * hb).abs())):
        dims = 1 if name == "gate" and per_sample else (0, 1)
        v, bound = term.sum(dim=dims), (term_ + 41 * STEP * term.abs()).sum(dim=dims)
        out[name] = (v.cpu(), rounded(v, bound, t[name].dtype).cpu())
    return out


# (turns of a thread beyond 16, the last one in part; lanes of a row and vectors of a lane as the channels give them)
CASES = [("f32", F32, F32, (1, 70001, 260), "channel"), ("f32-bf16", F32, BF16, (1, 70001, 260), "channel"),
         ("f32-sample", F32, F32, (3, 25003, 260), "sample"), ("bf16", BF16, BF16, (1, 1200001, 24), "channel"),
         ("f16-sample", F16, F16, (5, 240001, 24), "sample"), ("f32-few", F32, F32, (1, 4300001, 3), "channel"),
         ("f32-12", F32, F32, (1, 17001, 4100), "channel"), ("f32-16", F32, F16, (1, 17001, 6200), "channel"),
         ("f16-16", F16, F16, (1, 17001, 4104), "channel"), ("bf16-16", BF16, BF16, (2, 8701, 8192), "sample")]


@pytest.mark.parametrize("name,xt,bt,shape,gate", CASES, ids=[c[0] for c in CASES])
def test_sums_over_many_rows(name, xt, bt, shape, gate):
    banner("residual turns", name, shape)
    gen = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    C = shape[-1]
    t = {"x": rnd(*shape).to(xt), "branch": (rnd(*shape) * (0.3 + rnd(C).abs())).to(bt),
         "gate": 0.5 + 0.5 * rnd(*((C,) if gate == "channel" else (shape[0], C))), "weight": 1 + 0.2 * rnd(C),
         "branch_weight": 1 + 0.2 * rnd(C)}
    gy, gz = rnd(*shape).to(xt), rnd(*shape).to(bt)
    want = parameter_sums(t, gy, gz)
    leaves = {k: t[k].requires_grad_() for k in ("gate", "weight", "branch_weight")}
    outs = E.residual_norm(t["x"], t["branch"], **leaves)
    grads = torch.autograd.grad(outs, list(leaves.values()), [gy, gz])
    for k, v in zip(leaves, grads):
        ratio = worst(v, want[k])
        assert ratio <= 1, (k, ratio)


@pytest.mark.parametrize("types", TYPES, ids=IDS)
@pytest.mark.parametrize("shape", [(1, 1, 1), (2, 7), (3, 5, 8), (2, 70, 9), (2, 3, 5, 24), (4, 33, 64), (3, 37, 411),
                                   (2, 6, 1024), (1, 3, 2051), (2, 2, 8192)], ids=lambda s: "x".join(map(str, s)))
def test_norm_by_itself(shape, types):
    banner("rms norm", shape, types)
    t, _, gz = make(shape, *types, seed=sum(shape))
    want = residual(t["x"], None, weight=t["weight"], gz=gz, ztype=types[1])
    x, w = t["x"].cuda().requires_grad_(), t["weight"].cuda().requires_grad_()
    z = E.rms_norm(x, w, dtype=types[1])
    gx, gw = torch.autograd.grad(z, [x, w], gz.cuda())
    for name, v in (("z", z), ("x", gx), ("weight", gw)):
        ratio = worst(v, want[name])
        assert ratio <= 1, (name, ratio)
