"""Cases and plain forms of the operators that read curves as sequences and mix channels at every position.

Three operators are covered, each in the forms a training or an inference program calls:

* ``residual_norm``: the gate, the norm and the residual scale after a block and the norm before the next one, in one pass;
* ``gated_linear``: both projections of a gated feed-forward block, the activation and the product;
* ``gated_recurrence``: a gated linear recurrence along the thresholds of a curve (or any sequence), with a state.

``own`` selects between the plain form (elementary torch operations in 32 bits) and the framework's entry points.
"""

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one position of a sequence model at inference: launch latency
        {"name": "resnorm_fwd_token_bf16", "op": "resnorm", "train": False, "batch": 1, "inner": 1, "channels": 1024,
         "dtype": "bf16", "stream": "bf16", "params": "bf16", "gate": "channel", "after": True, "scale": 1.0},
        # ragged rows of an odd width at inference, no norm after the block
        {"name": "resnorm_fwd_odd_f16", "op": "resnorm", "train": False, "batch": 3, "inner": 1337, "channels": 411,
         "dtype": "f16", "stream": "f16", "params": "f32", "gate": "channel", "after": False, "scale": 0.7},
        # curves along 64 directions of 256 thresholds, residual stream kept in 32 bits
        {"name": "resnorm_train_curves_bf16", "op": "resnorm", "train": True, "batch": 64, "inner": 256, "channels": 1024,
         "dtype": "bf16", "stream": "f32", "params": "f32", "gate": "channel", "after": True, "scale": 1.0},
        # every voxel of two volumes, gates conditioned on the sample
        {"name": "resnorm_train_voxels_bf16", "op": "resnorm", "train": True, "batch": 2, "inner": 96 ** 3, "channels": 64,
         "dtype": "bf16", "stream": "bf16", "params": "bf16", "gate": "sample", "after": True, "scale": 1.0},
        # one position at inference: the weights are read once
        {"name": "glu_fwd_token_bf16", "op": "glu", "train": False, "rows": 1, "channels": 1024, "hidden": 2816,
         "dtype": "bf16", "bias": False, "act": "silu"},
        # training in float32 with odd sizes throughout
        {"name": "glu_train_odd_f32", "op": "glu", "train": True, "rows": 1999, "channels": 333, "hidden": 877,
         "dtype": "f32", "bias": True, "act": "gelu"},
        # every voxel of two volumes through a narrow block
        {"name": "glu_train_voxels_f16", "op": "glu", "train": True, "rows": 2 * 64 ** 3, "channels": 64, "hidden": 160,
         "dtype": "f16", "bias": True, "act": "silu"},
        # curves along 64 directions of 256 thresholds through a wide block
        {"name": "glu_train_curves_bf16", "op": "glu", "train": True, "rows": 64 * 256, "channels": 1024, "hidden": 2816,
         "dtype": "bf16", "bias": False, "act": "silu"},
        # one threshold more for a batch of running sequences: states are carried from call to call
        {"name": "recur_step_bf16", "op": "recur", "train": False, "batch": 64, "steps": 1, "channels": 1024,
         "dtype": "bf16", "state": True, "lengths": False},
        # one long sequence of few channels
        {"name": "recur_fwd_long_f32", "op": "recur", "train": False, "batch": 1, "steps": 65536, "channels": 96,
         "dtype": "f32", "state": False, "lengths": False},
        # curves of as many thresholds as a curve may have, padded to the longest, an odd number of channels
        {"name": "recur_train_ragged_f16", "op": "recur", "train": True, "batch": 12, "steps": 8192, "channels": 201,
         "dtype": "f16", "state": True, "lengths": True},
        # curves along 64 directions of 256 thresholds
        {"name": "recur_train_curves_bf16", "op": "recur", "train": True, "batch": 64, "steps": 256, "channels": 1024,
         "dtype": "bf16", "state": False, "lengths": False},
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["resnorm", "glu", "recur"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    train = rng.random() < 0.6
    if op == "resnorm":
        channels = _spread(rng, 8, 4096)
        batch = _spread(rng, 1, 16)
        inner = _spread(rng, 1, max(2, (1 << 25) // (batch * channels)))
        return {"op": op, "train": train, "batch": batch, "inner": inner, "channels": channels, "dtype": dtype,
                "stream": rng.choice(["f32", dtype]), "params": rng.choice(["f32", dtype]),
                "gate": rng.choice(["none", "channel", "sample"]), "after": rng.random() < 0.6,
                "scale": rng.choice([1.0, 0.5, 1.7])}
    if op == "glu":
        channels, hidden = _spread(rng, 16, 2048), _spread(rng, 16, 4096)
        # a tenth of the largest listed case's products
        rows = _spread(rng, 1, max(2, min(200000, int(5e9 / (channels * hidden)))))
        # relu's slope jumps at 0, where two roundings of one value fall on either side: forward only
        acts = ["none", "silu", "gelu"] + ([] if train else ["relu"])
        return {"op": op, "train": train, "rows": rows, "channels": channels, "hidden": hidden, "dtype": dtype,
                "bias": rng.random() < 0.5, "act": rng.choice(acts)}
    channels, batch = _spread(rng, 8, 2048), _spread(rng, 1, 64)
    steps = _spread(rng, 1, min(65536, max(2, (1 << 24) // (batch * channels))))
    return {"op": op, "train": train, "batch": batch, "steps": steps, "channels": channels, "dtype": dtype,
            "state": rng.random() < 0.5, "lengths": rng.random() < 0.4}


# ----------------------------------------------------------------- inputs
LEAVES = {"resnorm": ("x", "branch", "gate", "weight", "branch_weight"),
          "glu": ("x", "w_gate", "w_up", "b_gate", "b_up"), "recur": ("x", "gate", "state")}


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    dt, c, op = DTYPES[case["dtype"]], case["channels"], case["op"]
    state = {"case": case}
    if op == "resnorm":
        sdt, pdt = DTYPES[case["stream"]], DTYPES[case["params"]]
        shape = [case["batch"], case["inner"], c]
        # a stream that has grown over some blocks, with louder channels, and a block's output
        state["x"] = normal(*shape).mul_(1 + 2 * normal(c).abs()).to(sdt)
        state["branch"] = normal(*shape).mul_(0.3 + normal(c).abs()).to(dt)
        if case["gate"] != "none":
            state["gate"] = (0.5 + 0.5 * normal(*([c] if case["gate"] == "channel" else [case["batch"], c]))).to(pdt)
        state["weight"] = (1 + 0.2 * normal(c)).to(pdt)
        if case["after"]:
            state["branch_weight"] = (1 + 0.2 * normal(c)).to(pdt)
        if case["train"]:
            state["grads"] = [normal(*shape).to(sdt), normal(*shape).to(dt)]
    elif op == "glu":
        f = case["hidden"]
        state["x"] = normal(case["rows"], c).to(dt)
        state["w_gate"], state["w_up"] = ((normal(f, c) / math.sqrt(c)).to(dt) for _ in range(2))
        if case["bias"]:
            state["b_gate"], state["b_up"] = ((0.2 * normal(f)).to(dt) for _ in range(2))
        if case["train"]:
            state["grads"] = [normal(case["rows"], f).to(dt)]
    else:
        b, t = case["batch"], case["steps"]
        state["x"] = normal(b, t, c).to(dt)
        # memories from a step or two to some hundreds of them, by channel
        state["gate"] = normal(b, t, c).add_(torch.rand(c, generator=gen, device="cuda") * 7 - 1).to(dt)
        if case["state"]:
            state["state"] = normal(b, c)
        if case["lengths"]:
            n = torch.randint(0, t + 1, (b,), generator=gen, device="cuda")
            n[0] = t
            state["lengths"] = n
        if case["train"]:
            state["grads"] = [normal(b, t, c).to(dt), normal(b, c)]
    if case["train"]:
        for name in LEAVES[op]:
            if name in state:
                state[name].requires_grad_()
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
    if act == "silu":
        s = 1 / (1 + torch.exp(-u))
        return s * (1 + u * (1 - s))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(u * math.sqrt(0.5))) + u * torch.exp(-0.5 * u * u) / math.sqrt(2 * math.pi)
    return torch.ones_like(u)


def _rms(v):
    return (v * v).sum(dim=-1, keepdim=True).div_(v.shape[-1]).add_(EPS).rsqrt_()


def _rms_back(dn, v, r):
    """Gradient of v r(v) where dn is that of the result."""
    return r * (dn - v * (r * r * (dn * v).sum(dim=-1, keepdim=True) / v.shape[-1]))


def _plain_resnorm(state):
    case = state["case"]
    x, branch = state["x"].float(), state["branch"].float()
    weight = state["weight"].float()
    gate = state["gate"].float() if "gate" in state else torch.ones_like(weight)
    if case["gate"] == "sample":
        gate = gate[:, None]
    if case["after"]:
        after = state["branch_weight"].float()
        rb = _rms(branch)
        hat = branch * rb
        n = hat * after
    else:
        n = branch
    y = case["scale"] * x + gate * n
    ry = _rms(y)
    outs = {"y": y.to(state["x"].dtype), "z": (y * ry * weight).to(state["branch"].dtype)}
    if not case["train"]:
        return outs
    dy, dz = state["grads"][0].float(), state["grads"][1].float()
    outs["weight"] = (dz * y * ry).sum(dim=(0, 1)).to(state["weight"].dtype)
    dy = dy + _rms_back(dz * weight, y, ry)
    outs["x"] = (case["scale"] * dy).to(state["x"].dtype)
    if case["gate"] != "none":
        outs["gate"] = (dy * n).sum(dim=1 if case["gate"] == "sample" else (0, 1)).to(state["gate"].dtype)
    dn = dy * gate
    if case["after"]:
        outs["branch_weight"] = (dn * hat).sum(dim=(0, 1)).to(state["branch_weight"].dtype)
        dn = _rms_back(dn * after, branch, rb)
    outs["branch"] = dn.to(state["branch"].dtype)
    return outs


def _plain_glu(state):
    case = state["case"]
    x, wg, wu = (state[k].float() for k in ("x", "w_gate", "w_up"))
    a, b = torch.matmul(x, wg.t()), torch.matmul(x, wu.t())
    if case["bias"]:
        a, b = a + state["b_gate"].float(), b + state["b_up"].float()
    dt = state["x"].dtype
    value = _activation(a, case["act"])
    outs = {"h": (value * b).to(dt)}
    if not case["train"]:
        return outs
    dh = state["grads"][0].float()
    da, db = dh * b * _slope(a, case["act"]), dh * value
    outs["x"] = (torch.matmul(da, wg) + torch.matmul(db, wu)).to(dt)
    outs["w_gate"], outs["w_up"] = torch.matmul(da.t(), x).to(dt), torch.matmul(db.t(), x).to(dt)
    if case["bias"]:
        outs["b_gate"], outs["b_up"] = da.sum(dim=0).to(dt), db.sum(dim=0).to(dt)
    return outs


def _scan(a, b):
    """h_t = a_t h_(t-1) + b_t from h = 0 along the second axis, and the products of a from the start, by doubling."""
    step = 1
    while step < a.shape[1]:
        b = torch.cat([b[:, :step], b[:, step:] + a[:, step:] * b[:, :-step]], dim=1)
        a = torch.cat([a[:, :step], a[:, step:] * a[:, :-step]], dim=1)
        step *= 2
    return a, b


def _plain_recur(state):
    case, x, gate = state["case"], state["x"].float(), state["gate"].float()
    b, t, c = x.shape
    keep, blend = 1 / (1 + torch.exp(-gate)), 1 / (1 + torch.exp(gate))
    first = state["state"] if case["state"] else torch.zeros(b, c, device=x.device)
    inside = None
    if case["lengths"]:
        inside = (torch.arange(t, device=x.device) < state["lengths"][:, None])[:, :, None]
        keep, blend = torch.where(inside, keep, 1.0), torch.where(inside, blend, 0.0)
        x = torch.where(inside, x, 0.0)
    prod, h = _scan(keep, blend * x)
    h = h + prod * first[:, None]
    shown = h if inside is None else torch.where(inside, h, 0.0)
    outs = {"h": shown.to(state["x"].dtype), "last": h[:, -1].clone()}
    if not case["train"]:
        return outs
    dh, dlast = state["grads"][0].float(), state["grads"][1]
    if inside is not None:
        dh = torch.where(inside, dh, 0.0)
    # gradients run backwards: D_t = dh_t + a_(t+1) D_(t+1), the last one with the state's
    later = torch.cat([keep[:, 1:], torch.ones_like(keep[:, :1])], dim=1).flip(1)
    prod, d = _scan(later, dh.flip(1))
    d = (d + prod * dlast[:, None]).flip(1)
    before = torch.cat([first[:, None], h[:, :-1]], dim=1)
    outs["x"] = (blend * d).to(state["x"].dtype)
    outs["gate"] = (d * (before - x) * keep * blend).to(state["gate"].dtype)
    if case["state"]:
        outs["state"] = keep[:, 0] * d[:, 0]
    return outs


PLAIN = {"resnorm": _plain_resnorm, "glu": _plain_glu, "recur": _plain_recur}


# -------------------------------------------------------------------- run
def run(state):
    if own:
        return _own(state)
    with torch.no_grad():
        return PLAIN[state["case"]["op"]](state)


def _own(state):
    import euler_characteristic_curves_amd as E

    case = state["case"]
    if case["op"] == "resnorm":
        y, z = E.residual_norm(state["x"], state["branch"], gate=state.get("gate"), weight=state["weight"],
                               branch_weight=state.get("branch_weight"), norm_branch=case["after"], scale=case["scale"],
                               eps=EPS)
        outs = {"y": y, "z": z}
    elif case["op"] == "glu":
        outs = {"h": E.gated_linear(state["x"], state["w_gate"], state["w_up"], state.get("b_gate"), state.get("b_up"),
                                    act=case["act"])}
    else:
        h, last = E.gated_recurrence(state["x"], state["gate"], state=state.get("state"), lengths=state.get("lengths"))
        outs = {"h": h, "last": last}
    if case["train"]:
        leaves = [k for k in LEAVES[case["op"]] if k in state]
        got = torch.autograd.grad(list(outs.values()), [state[k] for k in leaves], state["grads"])
        outs.update(zip(leaves, got))
    return outs


# ------------------------------------------------------------------- work
def work(case):
    """Bytes with every input read and every output written once; operations of the formulas (an exponential or an
    error function as one)."""
    size = {"f32": 4, "bf16": 2, "f16": 2}
    e, c, ways = size[case["dtype"]], case["channels"], 2 if case["train"] else 1
    if case["op"] == "resnorm":
        n, p = case["batch"] * case["inner"] * c, size[case["params"]]
        params = c * p * (1 + case["after"] + {"none": 0, "channel": 1, "sample": case["batch"]}[case["gate"]])
        return {"bytes": ways * (2 * n * (e + size[case["stream"]]) + params), "flops": n * (9 + 20 * (ways - 1))}
    if case["op"] == "glu":
        n, f = case["rows"], case["hidden"]
        params = (2 * c * f + (2 * f if case["bias"] else 0)) * e
        return {"bytes": ways * (n * (c + f) * e + params), "flops": 4 * n * c * f * (3 if case["train"] else 1)
                + n * f * (6 + 8 * (ways - 1))}
    n, states = case["batch"] * case["steps"] * c, case["batch"] * c * 4
    return {"bytes": ways * (3 * n * e + states * (1 + case["state"])), "flops": n * (6 + 10 * (ways - 1))}


# ------------------------------------------------------------------ exact
def exact(case, seed):
    """The definitions in 64 bits: norms and products through double-precision autograd, the recurrence step by step."""
    state = prepare(case, seed)
    if case["op"] == "recur":
        return _exact_recur(case, state)
    names = [k for k in LEAVES[case["op"]] if k in state]
    v = {k: state[k].detach().double().requires_grad_(case["train"]) for k in names}
    if case["op"] == "resnorm":
        def unit(t):
            return t / torch.sqrt(t.square().mean(dim=-1, keepdim=True) + EPS)

        n = unit(v["branch"]) * v["branch_weight"] if case["after"] else v["branch"]
        if case["gate"] == "channel":
            n = n * v["gate"]
        elif case["gate"] == "sample":
            n = n * v["gate"].unsqueeze(1)
        y = v["x"] * case["scale"] + n
        outs = {"y": y, "z": unit(y) * v["weight"]}
    else:
        a, b = v["x"] @ v["w_gate"].mT, v["x"] @ v["w_up"].mT
        if case["bias"]:
            a, b = a + v["b_gate"], b + v["b_up"]
        if case["act"] == "relu":
            a = torch.where(a > 0, a, torch.zeros_like(a))
        elif case["act"] == "silu":
            a = a * torch.sigmoid(a)
        elif case["act"] == "gelu":
            a = a * torch.special.ndtr(a)
        outs = {"h": a * b}
    done = {k: t.detach() for k, t in outs.items()}
    if case["train"]:
        grads = torch.autograd.grad(list(outs.values()), [v[k] for k in names], [g.double() for g in state["grads"]])
        done.update(zip(names, grads))
    return done


def _exact_recur(case, state):
    # time first, so that a step is one contiguous slice
    x, gate = (state[k].detach().double().transpose(0, 1).contiguous() for k in ("x", "gate"))
    t, b, c = x.shape
    a, one_minus = torch.sigmoid(gate), torch.sigmoid(-gate)
    h = torch.zeros(b, c, dtype=torch.float64, device=x.device)
    if case["state"]:
        h = state["state"].detach().double()
    on = None
    if case["lengths"]:
        on = (torch.arange(t, device=x.device)[:, None] < state["lengths"])[:, :, None]
        a, one_minus = torch.where(on, a, 1.0), torch.where(on, one_minus, 0.0)
    drive = one_minus * x
    before = torch.empty_like(x)
    for i in range(t):
        before[i] = h
        h = torch.addcmul(drive[i], a[i], h)
    every = torch.cat([before[1:], h[None]])
    if on is not None:
        every = torch.where(on, every, 0.0)
    outs = {"h": every.transpose(0, 1).contiguous(), "last": h}
    if not case["train"]:
        return outs
    dh, d = state["grads"][0].double().transpose(0, 1).contiguous(), state["grads"][1].double()
    if on is not None:
        dh = torch.where(on, dh, 0.0)
    total = torch.empty_like(x)
    for i in range(t - 1, -1, -1):
        total[i] = d = d + dh[i]
        d = d * a[i]
    outs["x"] = (total * one_minus).transpose(0, 1).contiguous()
    outs["gate"] = (total * (before - x) * a * one_minus).transpose(0, 1).contiguous()
    if case["state"]:
        outs["state"] = d
    return outs
