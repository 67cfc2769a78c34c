"""Cases and plain forms of the operators that train a network through the curves.

Four operators are covered, each in the forms a training or an inference program calls:

* ``group_norm_act``: group norm with an activation over channels-last features, forward and with its gradient;
* ``group_norm_readout``: the same norm, contracted with one weight per channel to the float32 grid a curve reads;
* ``orthogonalize``: Newton-Schulz orthogonalisation of a matrix or a stack of matrices;
* ``muon_step``: momentum, orthogonalisation and the weight update of a stack of matrices, in place.

``own`` selects between the plain form (elementary torch operations in 32 bits) and the framework's entry points.
"""

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
STEPS = 5
NORM_EPS = 1e-5
ORTH_EPS = 1e-7


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the first feature map of one small image at inference: launch latency
        {"name": "norm_fwd_128sq_f32", "op": "norm", "train": False, "batch": 1, "space": "128x128", "channels": 32,
         "groups": 8, "act": "silu", "dtype": "f32", "params": "f32"},
        # a middle layer of a volume network at inference
        {"name": "norm_fwd_64cube_bf16", "op": "norm", "train": False, "batch": 2, "space": "64x64x64", "channels": 128,
         "groups": 32, "act": "silu", "dtype": "bf16", "params": "f32"},
        # training on crops of odd sizes, float16
        {"name": "norm_train_odd_f16", "op": "norm", "train": True, "batch": 3, "space": "37x41x43", "channels": 96,
         "groups": 12, "act": "gelu", "dtype": "f16", "params": "f32"},
        # training at full resolution, parameters kept in bfloat16 as the features are
        {"name": "norm_train_128cube_bf16", "op": "norm", "train": True, "batch": 2, "space": "128x128x128",
         "channels": 64, "groups": 16, "act": "silu", "dtype": "bf16", "params": "bf16"},
        # a batch of small images to their grids at inference
        {"name": "readout_fwd_64sq_f32", "op": "readout", "train": False, "batch": 8, "space": "64x64", "channels": 24,
         "groups": 4, "act": "silu", "dtype": "f32", "params": "f32"},
        # training a volume network in float32, ragged rows
        {"name": "readout_train_95cube_f32", "op": "readout", "train": True, "batch": 2, "space": "95x96x97",
         "channels": 48, "groups": 6, "act": "gelu", "dtype": "f32", "params": "f32"},
        # training at the size of the soft curve's own benchmark grid
        {"name": "readout_train_256cube_bf16", "op": "readout", "train": True, "batch": 1, "space": "256x256x256",
         "channels": 32, "groups": 8, "act": "silu", "dtype": "bf16", "params": "f32"},
        # the kernel taps of one 3x3x3 layer from a scalar grid: latency
        {"name": "orth_27x64_f32", "op": "orth", "batch": 1, "rows": 27, "cols": 64, "dtype": "f32"},
        # a few ragged layers of one shape, gradients in bfloat16, more rows than columns
        {"name": "orth_4x1411x1000_bf16", "op": "orth", "batch": 4, "rows": 1411, "cols": 1000, "dtype": "bf16"},
        # one large square layer
        {"name": "orth_4096sq_f32", "op": "orth", "batch": 1, "rows": 4096, "cols": 4096, "dtype": "f32"},
        # the 3x3x3 kernels of a volume network, 64 channels to 64, all layers stacked
        {"name": "muon_24x64x1728_f32", "op": "muon", "batch": 24, "rows": 64, "cols": 1728, "dtype": "f32",
         "grads": "f32", "nesterov": True, "decay": 0.0},
        # the first layer of a head over 64 directions of 256 thresholds, gradients in bfloat16
        {"name": "muon_512x16384_bf16", "op": "muon", "batch": 1, "rows": 512, "cols": 16384, "dtype": "f32",
         "grads": "bf16", "nesterov": True, "decay": 0.01},
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "readout", "readout", "orth", "muon"])
    if op in ("norm", "readout"):
        dtype = rng.choice(["f32", "bf16", "f16"])
        channels = rng.choice([8, 12, 16, 24, 32, 40, 48, 51, 64, 80, 96, 128, 160, 192, 256, 320, 384, 512])
        groups = rng.choice([g for g in range(1, channels + 1) if channels % g == 0])
        batch = _spread(rng, 1, 8)
        # one pass touches at most about a quarter of the largest listed case
        voxels = _spread(rng, 64, max(65, (1 << 27) // (batch * channels)))
        if rng.random() < 0.5:
            ny = max(1, _spread(rng, max(1, math.isqrt(voxels) // 2), 2 * math.isqrt(voxels)))
            space = "%dx%d" % (ny, max(1, voxels // ny))
        else:
            nz = max(1, round(voxels ** (1 / 3) * rng.uniform(0.6, 1.6)))
            ny = max(1, round(math.sqrt(voxels / nz) * rng.uniform(0.6, 1.6)))
            space = "%dx%dx%d" % (nz, ny, max(1, voxels // (nz * ny)))
        train = rng.random() < 0.6
        # relu's slope jumps at 0, where two roundings of one value fall on either side: forward only
        acts = ["none", "silu", "gelu"] + ([] if train else ["relu"])
        return {"op": op, "train": train, "batch": batch, "space": space, "channels": channels, "groups": groups,
                "act": rng.choice(acts), "dtype": dtype, "params": rng.choice(["f32", dtype])}
    rows, cols = _spread(rng, 3, 4000), _spread(rng, 16, 4000)
    small, large = min(rows, cols), max(rows, cols)
    most = min(32, max(1, int(2e10 / (small * small * (3 * large + small)))), max(1, (1 << 25) // (rows * cols)))
    case = {"op": op, "batch": _spread(rng, 1, most) if most > 1 else 1, "rows": rows, "cols": cols,
            "dtype": rng.choice(["f32", "bf16"])}
    if op == "muon":
        case.update(grads=rng.choice(["f32", "bf16"]), nesterov=rng.random() < 0.5, decay=rng.choice([0.0, 0.01, 0.1]))
    return case


# ----------------------------------------------------------------- inputs
def _space(case):
    return [int(n) for n in case["space"].split("x")]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    if case["op"] in ("norm", "readout"):
        dt, pdt, c = DTYPES[case["dtype"]], DTYPES[case["params"]], case["channels"]
        shape = [case["batch"], *_space(case), c]
        # features as a convolution leaves them: every channel with an offset and a scale of its own
        scale, offset = 0.5 + normal(c).abs(), 0.7 * normal(c)
        x = normal(*shape).mul_(scale).add_(offset).to(dt)
        state = {"case": case, "x": x, "weight": (1 + 0.2 * normal(c)).to(pdt), "bias": (0.2 * normal(c)).to(pdt)}
        if case["op"] == "readout":
            state["readout"] = (normal(c) / math.sqrt(c)).to(pdt)
            state["offset"] = (0.1 * normal(1)).to(pdt)
        if case["train"]:
            state["grad"] = normal(*(shape if case["op"] == "norm" else shape[:-1]))
            if case["op"] == "norm":
                state["grad"] = state["grad"].to(dt)
            for name in ("x", "weight", "bias", "readout", "offset"):
                if name in state:
                    state[name].requires_grad_()
        return state

    b, m, n = case["batch"], case["rows"], case["cols"]
    gdt = DTYPES[case["grads"] if case["op"] == "muon" else case["dtype"]]

    def gradient():
        # a few strong directions over a weak background, as gradients of matrices have them
        r = max(1, min(m, n) // 8)
        strong = torch.matmul(normal(b, m, r) * torch.linspace(1, 0.05, r, device="cuda"), normal(b, r, n))
        return (strong / math.sqrt(r) + 0.3 * normal(b, m, n)).mul_(1e-3)

    state = {"case": case, "grad": gradient().to(gdt)}
    if case["op"] == "muon":
        state["param"] = (normal(b, m, n) / math.sqrt(n)).to(DTYPES[case["dtype"]])
        state["buffer"] = gradient()
    return state


# ------------------------------------------------------------- plain forms
def _activation(u, act):
    if act == "relu":
        return u.clamp_min(0)
    if act == "silu":
        return u / (1 + torch.exp(-u))
    if act == "gelu":
        return 0.5 * u * (1 + torch.erf(u * math.sqrt(0.5)))
    return u


def _slope(u, act):
    if act == "relu":
        return (u > 0).to(u.dtype)
    if act == "silu":
        s = 1 / (1 + torch.exp(-u))
        return s * (1 + u * (1 - s))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(u * math.sqrt(0.5))) + u * torch.exp(-0.5 * u * u) / math.sqrt(2 * math.pi)
    return torch.ones_like(u)


def _plain_norm(state):
    case, x = state["case"], state["x"]
    b, c, g = case["batch"], case["channels"], case["groups"]
    w, bias = state["weight"].float(), state["bias"].float()
    v = x.float().reshape(b, -1, g, c // g)
    count = v.shape[1] * v.shape[3]
    centred = v - v.sum(dim=(1, 3), keepdim=True) / count
    rstd = ((centred * centred).sum(dim=(1, 3), keepdim=True) / count + NORM_EPS).rsqrt()
    xhat = (centred * rstd).reshape(b, -1, c)
    u = xhat * w + bias
    y = _activation(u, case["act"])
    outs = {}
    if case["op"] == "norm":
        outs["y"] = y.reshape(x.shape).to(x.dtype)
    else:
        r = state["readout"].float()
        outs["field"] = ((y * r).sum(dim=2) + state["offset"].float()).reshape(x.shape[:-1])
    if not case["train"]:
        return outs
    if case["op"] == "norm":
        dy = state["grad"].float().reshape(b, -1, c)
    else:
        df = state["grad"].reshape(b, -1, 1)
        outs["readout"] = (df * y).sum(dim=(0, 1)).to(state["readout"].dtype)
        outs["offset"] = df.sum().reshape(1).to(state["offset"].dtype)
        dy = df * r
    du = dy * _slope(u, case["act"])
    outs["bias"] = du.sum(dim=(0, 1)).to(state["bias"].dtype)
    outs["weight"] = (du * xhat).sum(dim=(0, 1)).to(state["weight"].dtype)
    dxhat = (du * w).reshape(b, -1, g, c // g)
    xhat = xhat.reshape(b, -1, g, c // g)
    first = dxhat.sum(dim=(1, 3), keepdim=True) / count
    second = (dxhat * xhat).sum(dim=(1, 3), keepdim=True) / count
    outs["x"] = ((dxhat - first - xhat * second) * rstd).reshape(x.shape).to(x.dtype)
    return outs


def _plain_orthogonal(g):
    """Newton-Schulz iterates of a stack of float32 matrices."""
    tall = g.shape[1] > g.shape[2]
    x = g.transpose(1, 2).contiguous() if tall else g
    norm = x.double().square().sum(dim=(1, 2), keepdim=True).sqrt()
    x = (x / (norm + ORTH_EPS)).float()
    a, b, c = COEFFICIENTS
    for _ in range(STEPS):
        gram = torch.matmul(x, x.transpose(1, 2).contiguous())
        x = a * x + torch.matmul(b * gram + c * torch.matmul(gram, gram), x)
    return x.transpose(1, 2).contiguous() if tall else x


LR, MOMENTUM = 0.02, 0.95


def _scale(rows, cols):
    return math.sqrt(max(1.0, rows / cols))


def _plain_muon(state):
    case, p, buf, g = state["case"], state["param"], state["buffer"], state["grad"].float()
    buf.mul_(MOMENTUM).add_(g, alpha=1 - MOMENTUM)
    update = g * (1 - MOMENTUM) + buf * MOMENTUM if case["nesterov"] else buf
    step = _plain_orthogonal(update) * (LR * _scale(case["rows"], case["cols"]))
    p.copy_(p.float() * (1 - LR * case["decay"]) - step)
    return {"param": p, "buffer": buf}


# -------------------------------------------------------------------- run
def run(state):
    case = state["case"]
    if own:
        return _own(state)
    with torch.no_grad():
        if case["op"] in ("norm", "readout"):
            return _plain_norm(state)
        if case["op"] == "orth":
            return _plain_orthogonal(state["grad"].float()).to(state["grad"].dtype)
        return _plain_muon(state)


def _own(state):
    import euler_characteristic_curves_amd as E

    case = state["case"]
    if case["op"] == "orth":
        return E.orthogonalize(state["grad"], steps=STEPS, eps=ORTH_EPS, coefficients=COEFFICIENTS)
    if case["op"] == "muon":
        E.muon_step([state["param"]], [state["grad"]], [state["buffer"]], lr=LR, momentum=MOMENTUM,
                    nesterov=case["nesterov"], weight_decay=case["decay"], scale=_scale(case["rows"], case["cols"]),
                    steps=STEPS, eps=ORTH_EPS, coefficients=COEFFICIENTS)
        return {"param": state["param"], "buffer": state["buffer"]}
    if case["op"] == "norm":
        leaves = ["x", "weight", "bias"]
        out = E.group_norm_act(state["x"], case["groups"], state["weight"], state["bias"], act=case["act"], eps=NORM_EPS)
        outs = {"y": out}
    else:
        leaves = ["x", "weight", "bias", "readout", "offset"]
        out = E.group_norm_readout(state["x"], case["groups"], state["weight"], state["bias"], state["readout"],
                                   state["offset"], act=case["act"], eps=NORM_EPS)
        outs = {"field": out}
    if case["train"]:
        outs.update(zip(leaves, torch.autograd.grad(out, [state[k] for k in leaves], state["grad"])))
    return outs


# ------------------------------------------------------------------- work
def work(case):
    """Bytes with every input read and every output written once; operations of the formulas (symmetric products
    counted once for both halves, an exponential or an error function as one)."""
    size = {"f32": 4, "bf16": 2, "f16": 2}
    if case["op"] in ("norm", "readout"):
        voxels = case["batch"] * math.prod(_space(case))
        n, c, p = voxels * case["channels"], case["channels"], size[case["params"]]
        e = size[case["dtype"]]
        if case["op"] == "norm":
            moved, flops = 2 * n * e + 2 * c * p, 12 * n
            if case["train"]:
                moved, flops = moved + 2 * n * e + 2 * c * p, flops + 22 * n
        else:
            moved, flops = n * e + 4 * voxels + 3 * c * p, 14 * n
            if case["train"]:
                moved, flops = moved + n * e + 4 * voxels + 3 * c * p, flops + 26 * n
        return {"bytes": moved, "flops": flops}
    b, m, n = case["batch"], min(case["rows"], case["cols"]), max(case["rows"], case["cols"])
    flops = b * STEPS * (m * m * n + m * m * m + 2 * m * m * n)
    if case["op"] == "orth":
        return {"bytes": 2 * b * m * n * size[case["dtype"]], "flops": flops}
    return {"bytes": b * m * n * (size[case["grads"]] + 2 * size[case["dtype"]] + 8), "flops": flops + 8 * b * m * n}


# ------------------------------------------------------------------ exact
def exact(case, seed):
    """The definitions in 64 bits: the norm through torch's double-precision autograd, the orthogonalisation as an odd
    polynomial of the rows."""
    state = prepare(case, seed)
    if case["op"] in ("norm", "readout"):
        return _exact_norm(case, state)
    g = state["grad"].double()
    if case["op"] == "orth":
        return _exact_orthogonal(g)
    buf = MOMENTUM * state["buffer"].double() + (1 - MOMENTUM) * g
    update = (1 - MOMENTUM) * g + MOMENTUM * buf if case["nesterov"] else buf
    param = state["param"].double()
    param = param - LR * case["decay"] * param - LR * _scale(case["rows"], case["cols"]) * _exact_orthogonal(update)
    return {"param": param, "buffer": buf}


def _exact_norm(case, state):
    names = [k for k in ("x", "weight", "bias", "readout", "offset") if k in state]
    v = {k: state[k].detach().double().requires_grad_(case["train"]) for k in names}
    x = v["x"]
    split = x.reshape(case["batch"], -1, case["groups"], case["channels"] // case["groups"])
    var, mean = torch.var_mean(split, dim=(1, 3), correction=0, keepdim=True)
    u = ((split - mean) / torch.sqrt(var + NORM_EPS)).reshape(x.shape) * v["weight"] + v["bias"]
    if case["act"] == "relu":
        y = torch.where(u > 0, u, torch.zeros_like(u))
    elif case["act"] == "silu":
        y = u * torch.sigmoid(u)
    elif case["act"] == "gelu":
        y = u * torch.special.ndtr(u)
    else:
        y = u
    if case["op"] == "norm":
        outs = {"y": y.detach()}
    else:
        y = torch.tensordot(y, v["readout"], dims=1) + v["offset"]
        outs = {"field": y.detach()}
    if case["train"]:
        outs.update(zip(names, torch.autograd.grad(y, [v[k] for k in names], state["grad"].double())))
    return outs


def _exact_orthogonal(g):
    if g.shape[1] > g.shape[2]:
        return _exact_orthogonal(g.mT.contiguous()).mT.contiguous()
    x = g / (torch.linalg.matrix_norm(g)[:, None, None] + ORTH_EPS)
    a, b, c = COEFFICIENTS
    for _ in range(STEPS):
        gram = x @ x.mT.contiguous()
        cubic = gram @ x
        x = a * x + b * cubic + c * (gram @ cubic)
    return x
