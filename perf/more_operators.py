"""Timed cases of a gated feed-forward block's operators: the gated layer on
DFP-8 products (forward and backward), the norms around a block with its gate
and residual scale (forward and backward) and the Muon step.

A case is a dict of plain values; prepare() makes its inputs on the GPU from
a seed, run() makes one pass (the plain form in elementary torch operations,
or, where `own` is true, the library's calls) and exact() computes the same
outputs in 64 bits.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
NORMS = ("none", "layer", "rms")
EPS = 1e-5
NS = (3.4445, -4.7750, 2.0315)  # the quintic of Muon's Newton-Schulz steps
NS_STEPS = 5
DEV = "cuda:0"


def _gated(name, op, B, IN, H, act, dtype, bias=True, save_z=False):
    return {"name": name, "op": op, "B": B, "IN": IN, "H": H, "act": act, "dtype": dtype, "bias": bias, "save_z": save_z}


def _norm(name, op, rows, cols, norm_a, norm_y, dtype, gate_rows=0, alpha=1.0):
    return {"name": name, "op": op, "rows": rows, "cols": cols, "norm_a": norm_a, "norm_y": norm_y, "dtype": dtype,
            "gate_rows": gate_rows, "alpha": alpha}


def listed():
    return [
        # one token through the gate and up projections: both weights' bytes and the launch
        _gated("gated fwd 1x4096x4096", "gated_fwd", 1, 4096, 4096, "silu", "bf16", bias=False),
        # a small layer, the sizes of the 784-256-128-10 perceptron's first, FP32 activations
        _gated("gated fwd 256x784x256", "gated_fwd", 256, 784, 256, "relu", "f32"),
        # a ragged batch: odd rows, columns and reduction
        _gated("gated fwd 1000x1023x2049", "gated_fwd", 1000, 1023, 2049, "gelu_tanh", "f16"),
        # a training step over 8192 tokens, which keeps what its backward pass needs
        _gated("gated fwd 8192x4096x4096", "gated_fwd", 8192, 4096, 4096, "silu", "bf16", save_z=True),
        # the backward passes of the small layer and of the 8192 tokens
        _gated("gated bwd 256x784x256", "gated_bwd", 256, 784, 256, "relu", "f32"),
        _gated("gated bwd 8192x4096x4096", "gated_bwd", 8192, 4096, 4096, "silu", "bf16"),
        # one token between two blocks: the norm after the one, the gate, the residual and the norm before the other
        _norm("norms fwd 1x4096", "norms_fwd", 1, 4096, "rms", "rms", "bf16", gate_rows=1),
        # the same of a training step over 8192 tokens, and its gradient
        _norm("norms fwd 8192x4096", "norms_fwd", 8192, 4096, "rms", "rms", "bf16", gate_rows=8192),
        _norm("norms bwd 8192x4096", "norms_bwd", 8192, 4096, "rms", "rms", "bf16", gate_rows=8192),
        # short rows in FP32: 128 samples of 196 positions, each sample with a gate of its own
        _norm("norms bwd 25088x256", "norms_bwd", 25088, 256, "layer", "layer", "f32", gate_rows=196, alpha=0.5),
        # the optimiser step of the perceptron's three weights
        {"name": "muon 784-256-128-10", "op": "muon", "shapes": "256x784,128x256,10x128", "grad": "f32"},
        # the optimiser step of one 4096 x 4096 layer, bfloat16 gradients
        {"name": "muon 4096x4096", "op": "muon", "shapes": "4096x4096", "grad": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gated_fwd", "gated_bwd", "norms_fwd", "norms_bwd", "muon"])
    dtype = rng.choice(list(DT))
    if op == "muon":
        shapes = [(_log(rng, 8, 4096), _log(rng, 8, 4096)) for _ in range(rng.randint(1, 4))]
        while sum(m * n * min(m, n) for m, n in shapes) > 4096 ** 3:
            shapes.pop()
        return {"op": op, "shapes": ",".join("%dx%d" % s for s in shapes or [(4096, 1024)]), "grad": dtype}
    if op.startswith("norms"):
        rows = _log(rng, 1, 8192)
        return {"op": op, "rows": rows, "cols": _log(rng, 8, 4096), "norm_a": rng.choice(NORMS),
                "norm_y": rng.choice(NORMS[1:]), "dtype": dtype, "gate_rows": rng.choice([0, rows, _log(rng, 1, rows)]),
                "alpha": rng.choice([1.0, 0.5])}
    return {"op": op, "B": _log(rng, 1, 8192), "IN": _log(rng, 16, 4096), "H": _log(rng, 16, 4096),
            # FP32 gradients go with activations whose products are exact:
            # elsewhere one step of the 8-bit error weighs more than FP32 resolves
            "act": rng.choice(("none", "relu") if op == "gated_bwd" and dtype == "f32" else ACTS), "dtype": dtype,
            "bias": op == "gated_bwd" or rng.random() < 0.5, "save_z": op == "gated_fwd" and rng.random() < 0.5}


# ---- inputs -----------------------------------------------------------------

def _pow2(e):
    """2^e as float32 for an int32 tensor e in [-126, 127]."""
    return ((e + 127) << 23).view(torch.float32)


def _prepare_gated(c, g):
    B, IN, H, t = c["B"], c["IN"], c["H"], DT[c["dtype"]]
    new = lambda *shape: torch.randn(*shape, generator=g, device=DEV)  # noqa: E731
    ints = lambda rows, std: new(rows, IN).mul_(std).round_().clamp_(-128, 127).to(torch.int8)  # noqa: E731
    # activations of unit scale at 2^-5, weights at the exponent that keeps z near 1
    s = {"X": ints(B, 32.0), "W": ints(2 * H, 24.0), "eX": torch.tensor([-5], dtype=torch.int32, device=DEV),
         "eW": torch.tensor([-round(math.log2(24.0 * math.sqrt(IN)))], dtype=torch.int32, device=DEV)}
    if c["op"] == "gated_fwd":
        s["bias"] = new(2 * H) * 0.5 if c["bias"] else None
    else:
        s["Z"] = new(B, 2 * H).to(t)
        # per-token error of varying size, as a loss leaves it
        s["dY"] = (new(B, H) * (0.02 + 0.05 * torch.rand(B, 1, generator=g, device=DEV))).to(t)
    return s


def _stats(x, kind):
    """Mean and reciprocal deviation of the rows of a float64 tensor."""
    mean = x.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(x[:, :1])
    return mean, ((x - mean).square().mean(1, keepdim=True) + EPS).rsqrt()


def _prepare_norms(c, g):
    n, m, t = c["rows"], c["cols"], DT[c["dtype"]]
    new = lambda *shape: torch.randn(*shape, generator=g, device=DEV)  # noqa: E731
    a, x = new(n, m) + 0.25 * new(n, 1), new(n, m) * 1.5 + 0.25 * new(n, 1)
    x[:, torch.randint(0, m, (max(1, m // 128),), generator=g, device=DEV)] *= 8.0  # outlier channels of the stream
    groups = -(-n // c["gate_rows"]) if c["gate_rows"] else 0
    s = {"a": a.to(t), "x": x.to(t), "gate": 0.5 + 0.2 * new(groups, m) if groups else None}
    for k in "ay":
        kind = c["norm_" + k]
        s["gamma_" + k] = 1.0 + 0.1 * new(m) if kind != "none" else None
        s["beta_" + k] = 0.1 * new(m) if kind == "layer" else None
    if c["op"] == "norms_bwd":
        ad = s["a"].double()
        p = ad
        for k, v in (("a", ad), ("y", None)):
            if k == "y":
                gate = s["gate"].double().repeat_interleave(c["gate_rows"], 0)[:n] if groups else 1.0
                v = c["alpha"] * s["x"].double() + gate * p
                s["y"] = v.to(t)
            s["mean_" + k] = s["rstd_" + k] = None
            if c["norm_" + k] != "none":
                mean, rstd = _stats(v, c["norm_" + k])
                s["rstd_" + k] = rstd[:, 0].float()
                s["mean_" + k] = mean[:, 0].float() if c["norm_" + k] == "layer" else None
                p = (v - mean) * rstd * s["gamma_" + k] + (s["beta_" + k] if s["beta_" + k] is not None else 0.0)
        del s["x"]
        s["dy"], s["dn"] = (0.05 * new(n, m)).to(t), (0.05 * new(n, m)).to(t)
    return s


def _prepare_muon(c, g):
    shapes = [tuple(map(int, x.split("x"))) for x in c["shapes"].split(",")]
    s = {"lr": 0.02, "momentum": 0.95, "wd": 0.01, "eps": 1e-7, "p": [], "m": [], "g": []}
    for rows, cols in shapes:
        new = lambda *shape: torch.randn(*shape, generator=g, device=DEV)  # noqa: E731
        s["p"].append(new(rows, cols) / math.sqrt(cols))
        # a momentum of a few strong directions over the noise of many batches
        k = min(8, rows, cols)
        s["m"].append(1e-3 * new(rows, cols) + 5e-4 * new(rows, k) @ new(k, cols))
        s["g"].append((1e-3 * new(rows, cols)).to(DT[c["grad"]]))
    return s


def _buffers(c, s):
    """Outputs and workspaces that a program allocates once."""
    from integer_only_nn_amd import ops, steps
    empty = lambda *shape, dtype=torch.float32: torch.empty(shape, dtype=dtype, device=DEV)  # noqa: E731
    if c["op"].startswith("gated"):
        B, IN, H, t = c["B"], c["IN"], c["H"], DT[c["dtype"]]
        if c["op"] == "gated_fwd":
            s["Y"], s["Zout"] = empty(B, H, dtype=t), empty(B, 2 * H, dtype=t) if c["save_z"] else None
            s["ws"] = empty(ops.dfp8_gated_fwd_workspace_bytes(B, IN, H), dtype=torch.uint8)
        else:
            s["dZ8"], s["edZ"] = empty(B, 2 * H, dtype=torch.int8), empty(1, dtype=torch.int32)
            s["dX"], s["G"], s["gb"] = empty(B, IN, dtype=t), empty(2 * H, IN, dtype=t), empty(2 * H)
            s["ws"] = empty(ops.dfp8_gated_bwd_workspace_bytes(B, IN, H), dtype=torch.uint8)
    elif c["op"] == "muon":
        s["opt"] = steps.Muon(s["p"], s["m"], lr=s["lr"], momentum=s["momentum"], weight_decay=s["wd"], eps=s["eps"])
        s["opt"].bind_grads(s["g"])
    else:
        n, m, t = c["rows"], c["cols"], DT[c["dtype"]]
        if c["op"] == "norms_fwd":
            s["y"], s["n"] = empty(n, m, dtype=t), empty(n, m, dtype=t)
            for k in "ay":
                s["mean_" + k] = empty(n) if c["norm_" + k] == "layer" else None
                s["rstd_" + k] = empty(n) if c["norm_" + k] != "none" else None
        else:
            s["da"], s["dx"] = empty(n, m, dtype=t), empty(n, m, dtype=t)
            s["dgate"] = torch.empty_like(s["gate"]) if s["gate"] is not None else None
            for k in ("gamma_a", "beta_a", "gamma_y", "beta_y"):
                s["d" + k] = empty(m) if s[k] is not None else None
            s["ws"] = empty(ops.ionn_residual_norm_bwd_workspace_bytes(n, m, c["gate_rows"] or n), dtype=torch.uint8)


MAKE = {"gated": _prepare_gated, "norms": _prepare_norms, "muon": _prepare_muon}


def _inputs(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return MAKE[case["op"].split("_")[0]](case, g)


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = dict(case)
    if own:
        _buffers(case, s)
    return s


# ---- the plain forms --------------------------------------------------------

def _act(z, act):
    if act == "relu":
        return z.clamp_min(0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * math.sqrt(0.5 / math.pi)
    if act == "gelu_tanh":
        k = math.sqrt(2 / math.pi)
        t = torch.tanh(k * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * k * (1 + 3 * 0.044715 * z * z)
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    return torch.ones_like(z)


def _gated_fwd(s, c):
    t, H = DT[c["dtype"]], c["H"]
    z = (s["X"].float() @ s["W"].float().t()) * _pow2(s["eX"] + s["eW"])
    if s["bias"] is not None:
        z = z + s["bias"]
    y = _act(z[:, :H], c["act"]) * z[:, H:]
    return [y.to(t), z.to(t)] if c["save_z"] else [y.to(t)]


def _gated_bwd(s, c):
    t, H = DT[c["dtype"]], c["H"]
    # a product of two float32 values next to a rounding's border needs 64 bits; of 16-bit ones it is exact in 32
    wide = torch.float64 if t == torch.float32 else torch.float32
    dy, z = s["dY"].to(wide), s["Z"].to(wide)
    g, u = z[:, :H], z[:, H:]
    dz = torch.cat([dy * u * _act_grad(g, c["act"]), dy * _act(g, c["act"])], 1)
    bits = dz.abs().amax().float().view(torch.int32)
    e = torch.where(bits == 0, 0, (bits >> 23) - 133)
    q = (dz * _pow2(-e)).round().clamp(-128, 127).float()
    return [((q @ s["W"].float()) * _pow2(e + s["eW"])).to(t), ((q.t() @ s["X"].float()) * _pow2(e + s["eX"])).to(t),
            dz.sum(0).float()]


def _gates(s, c):
    """The gate of each row, or 1."""
    if s["gate"] is None:
        return 1.0
    return s["gate"] if s["gate"].shape[0] == 1 else s["gate"].repeat_interleave(c["gate_rows"], 0)[:c["rows"]]


def _normed(v, kind, gamma, beta):
    if kind == "none":
        return v, []
    mean = v.mean(1, keepdim=True) if kind == "layer" else 0.0
    d = v - mean
    rstd = 1 / torch.sqrt(d.square().mean(1, keepdim=True) + EPS)
    h = d * rstd * gamma
    return (h + beta, [mean[:, 0], rstd[:, 0]]) if kind == "layer" else (h, [rstd[:, 0]])


def _norms_fwd(s, c):
    t = DT[c["dtype"]]
    p, stats_a = _normed(s["a"].float(), c["norm_a"], s["gamma_a"], s["beta_a"])
    y = c["alpha"] * s["x"].float() + _gates(s, c) * p
    n, stats_y = _normed(y, c["norm_y"], s["gamma_y"], s["beta_y"])
    return [y.to(t), n.to(t)] + stats_a + stats_y


def _norm_back(d, v, kind, mean, rstd, gamma):
    """The gradient of a norm's input, and its normalised rows, for the error d of its output."""
    if kind == "none":
        return d, v
    h = (v - mean[:, None] if kind == "layer" else v) * rstd[:, None]
    e = d * gamma
    dx = e - h * (e * h).mean(1, keepdim=True)
    if kind == "layer":
        dx = dx - e.mean(1, keepdim=True)
    return rstd[:, None] * dx, h


def _norms_bwd(s, c):
    t, m = DT[c["dtype"]], c["cols"]
    dn = s["dn"].float()
    back, hy = _norm_back(dn, s["y"].float(), c["norm_y"], s["mean_y"], s["rstd_y"], s["gamma_y"])
    d = s["dy"].float() + back
    gate = _gates(s, c)
    e = d * gate
    da, ha = _norm_back(e, s["a"].float(), c["norm_a"], s["mean_a"], s["rstd_a"], s["gamma_a"])
    out = [da.to(t), (c["alpha"] * d).to(t)]
    if s["gate"] is not None:
        p = ha if s["gamma_a"] is None else ha * s["gamma_a"]
        p = p if s["beta_a"] is None else p + s["beta_a"]
        groups = s["gate"].shape[0]
        dg = torch.nn.functional.pad(d * p, (0, 0, 0, groups * c["gate_rows"] - c["rows"]))
        out.append(dg.view(groups, c["gate_rows"], m).sum(1))
    for k, x, h in (("a", e, ha), ("y", dn, hy)):
        if s["gamma_" + k] is not None:
            out.append((x * h).sum(0))
        if s["beta_" + k] is not None:
            out.append(x.sum(0))
    return out


def _muon(s, c):
    a, b, k = NS
    for p, m, g in zip(s["p"], s["m"], s["g"]):
        g = g.float()
        m.mul_(s["momentum"]).add_(g)
        u = g + s["momentum"] * m
        rows, cols = u.shape
        x = u.t() if rows > cols else u
        x = x / (torch.sqrt(x.square().sum()) + s["eps"])
        for _ in range(NS_STEPS):
            A = x @ x.t()
            x = a * x + (b * A + k * (A @ A)) @ x
        x = x.t() if rows > cols else x
        p.mul_(1 - s["lr"] * s["wd"]).sub_(x * (s["lr"] * math.sqrt(max(1.0, rows / cols))))
    return [s["p"], s["m"]]


PLAIN = {"gated_fwd": _gated_fwd, "gated_bwd": _gated_bwd, "norms_fwd": _norms_fwd, "norms_bwd": _norms_bwd,
         "muon": _muon}


# ---- the library's calls ----------------------------------------------------

def _given(*xs):
    return [x for x in xs if x is not None]


def _own(s, c):
    from integer_only_nn_amd import ops
    if c["op"] == "gated_fwd":
        ops.dfp8_gated_fwd(s["X"], s["eX"], s["W"], s["eW"], s["Y"], bias=s["bias"], act=c["act"], Z=s["Zout"],
                           workspace=s["ws"])
        return [s["Y"], s["Zout"]] if c["save_z"] else [s["Y"]]
    if c["op"] == "gated_bwd":
        ops.dfp8_gated_bwd(s["dY"], s["Z"], c["act"], s["X"], s["eX"], s["W"], s["eW"], s["dZ8"], s["edZ"],
                           dX=s["dX"], G=s["G"], gb=s["gb"], workspace=s["ws"])
        return [s["dX"], s["G"], s["gb"]]
    if c["op"] == "norms_fwd":
        ops.ionn_residual_norm_fwd(s["a"], s["x"], s["y"], s["n"], norm_a=c["norm_a"], gamma_a=s["gamma_a"],
                                   beta_a=s["beta_a"], gate=s["gate"], gate_rows=c["gate_rows"], alpha=c["alpha"],
                                   norm_y=c["norm_y"], gamma_y=s["gamma_y"], beta_y=s["beta_y"], eps=EPS,
                                   mean_a=s["mean_a"], rstd_a=s["rstd_a"], mean_y=s["mean_y"], rstd_y=s["rstd_y"])
        return [s["y"], s["n"]] + _given(s["mean_a"], s["rstd_a"], s["mean_y"], s["rstd_y"])
    if c["op"] == "norms_bwd":
        ops.ionn_residual_norm_bwd(s["dy"], s["dn"], s["a"], s["y"], s["da"], s["dx"], norm_a=c["norm_a"],
                                   gamma_a=s["gamma_a"], beta_a=s["beta_a"], gate=s["gate"], gate_rows=c["gate_rows"],
                                   alpha=c["alpha"], norm_y=c["norm_y"], gamma_y=s["gamma_y"], mean_a=s["mean_a"],
                                   rstd_a=s["rstd_a"], mean_y=s["mean_y"], rstd_y=s["rstd_y"], dgamma_a=s["dgamma_a"],
                                   dbeta_a=s["dbeta_a"], dgate=s["dgate"], dgamma_y=s["dgamma_y"],
                                   dbeta_y=s["dbeta_y"], workspace=s["ws"])
        return [s["da"], s["dx"]] + _given(s["dgate"], s["dgamma_a"], s["dbeta_a"], s["dgamma_y"], s["dbeta_y"])
    s["opt"].step()
    return [s["p"], s["m"]]


def run(state):
    c = state["case"]
    return _own(state, c) if own else PLAIN[c["op"]](state, c)


# ---- what a pass has to do --------------------------------------------------

def work(case):
    if case["op"] == "muon":
        shapes = [tuple(map(int, x.split("x"))) for x in case["shapes"].split(",")]
        t = DT[case["grad"]].itemsize
        # A and A A are symmetric: half of each
        return {"bytes": sum(r * c * (16 + t) for r, c in shapes),
                "flops": NS_STEPS * sum(3 * r * c * min(r, c) + min(r, c) ** 3 for r, c in shapes)}
    t = DT[case["dtype"]].itemsize
    if case["op"].startswith("norms"):
        n, fwd = case["rows"] * case["cols"], case["op"] == "norms_fwd"
        groups = -(-case["rows"] // case["gate_rows"]) if case["gate_rows"] else 0
        vectors = (1 if fwd else 2) * 4 * case["cols"] * (groups + sum(
            {"none": 0, "rms": 1, "layer": 2}[case[k]] for k in ("norm_a", "norm_y")))
        return {"bytes": (4 if fwd else 6) * t * n + vectors + 16 * case["rows"], "flops": (20 if fwd else 40) * n}
    B, IN, H = case["B"], case["IN"], case["H"]
    if case["op"] == "gated_fwd":
        return {"bytes": B * IN + 2 * H * IN + 8 * H * case["bias"] + (3 if case["save_z"] else 1) * t * B * H,
                "flops": 4 * B * IN * H}
    return {"bytes": 3 * t * B * H + (1 + t) * (B * IN + 2 * H * IN) + 8 * H, "flops": 8 * B * IN * H}


# ---- the definitions in 64 bits ---------------------------------------------

def _gelu_cdf(z):
    return 0.5 * torch.special.erfc(-z / math.sqrt(2.0))


def _exact_act(z, act):
    """The activation and its derivative."""
    if act == "relu":
        return torch.relu(z), (z > 0).double()
    if act == "gelu":
        return z * _gelu_cdf(z), _gelu_cdf(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":  # tanh(w) = 2 sigmoid(2 w) - 1
        w = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
        p, dw = torch.sigmoid(w), 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * z ** 2)
        return z * p, p + z * p * (1 - p) * dw
    if act == "silu":
        p = torch.sigmoid(z)
        return z * p, p + z * p * (1 - p)
    return z, torch.ones_like(z)


def _exact_gated(c, s):
    scale = lambda *es: 2.0 ** sum(int(e) for e in es)  # noqa: E731
    H, X, W = c["H"], s["X"].double(), s["W"].double()
    if c["op"] == "gated_fwd":
        z = torch.matmul(X, W.t().contiguous()) * scale(s["eX"], s["eW"])
        z = z + (s["bias"].double() if s["bias"] is not None else 0.0)
        gate, up = z.split(H, 1)
        y = _exact_act(gate, c["act"])[0] * up
        return [y, z] if c["save_z"] else [y]
    gate, up = s["Z"].double().split(H, 1)
    f, df = _exact_act(gate, c["act"])
    dz = torch.cat([s["dY"].double() * up * df, s["dY"].double() * f], 1)
    top = float(dz.abs().max())
    e = math.frexp(top)[1] - 7 if top else 0  # top = f 2^q with f in [1, 2): q - 6
    q = torch.clamp(torch.round(torch.ldexp(dz, torch.tensor(-e, device=DEV))), -128, 127)
    return [torch.matmul(q, W) * scale(e, s["eW"]), torch.matmul(q.t().contiguous(), X) * scale(e, s["eX"]), dz.sum(0)]


def _exact_norms(c, s):
    n = c["rows"]
    at = torch.arange(n, device=DEV) // (c["gate_rows"] or n)
    gate = s["gate"].double()[at] if s["gate"] is not None else torch.ones((), dtype=torch.float64, device=DEV)
    wide = {k: (s[k].double() if s[k] is not None else None) for k in ("gamma_a", "beta_a", "gamma_y", "beta_y")}
    a = s["a"].double()
    if c["op"] == "norms_fwd":
        outs, stats, v = [], [], a
        for k in "ay":
            if k == "y":
                v = c["alpha"] * s["x"].double() + gate * v
                outs.append(v)
            if c["norm_" + k] != "none":
                mean, rstd = _stats(v, c["norm_" + k])
                stats += [mean[:, 0], rstd[:, 0]] if c["norm_" + k] == "layer" else [rstd[:, 0]]
                v = (v - mean) * rstd * wide["gamma_" + k]
                v = v if wide["beta_" + k] is None else v + wide["beta_" + k]
        return outs + [v] + stats

    def rows(v, k):
        if c["norm_" + k] == "none":
            return v, None
        mean = s["mean_" + k].double()[:, None] if c["norm_" + k] == "layer" else 0.0
        rstd = s["rstd_" + k].double()[:, None]
        return (v - mean) * rstd, rstd

    def project(d, h, rstd, k):
        # the error off the normalised row and, for a layer norm, off the constant one
        if rstd is None:
            return d
        d = d * wide["gamma_" + k]
        off = h * ((d * h).sum(1, keepdim=True) / c["cols"])
        if c["norm_" + k] == "layer":
            off = off + d.sum(1, keepdim=True) / c["cols"]
        return (d - off) * rstd

    (ha, ra), (hy, ry) = rows(a, "a"), rows(s["y"].double(), "y")
    dn = s["dn"].double()
    t = s["dy"].double() + project(dn, hy, ry, "y")
    out = [project(t * gate, ha, ra, "a"), c["alpha"] * t]
    if s["gate"] is not None:
        p = ha if wide["gamma_a"] is None else ha * wide["gamma_a"]
        p = p if wide["beta_a"] is None else p + wide["beta_a"]
        out.append(torch.zeros_like(s["gate"], dtype=torch.float64).index_add_(0, at, t * p))
    for k, d, h in (("a", t * gate, ha), ("y", dn, hy)):
        out += [(d * h).sum(0)] if wide["gamma_" + k] is not None else []
        out += [d.sum(0)] if wide["beta_" + k] is not None else []
    return out


def _exact_muon(c, s):
    out = [[], []]
    for p, m, g in zip(s["p"], s["m"], s["g"]):
        m = s["momentum"] * m.double() + g.double()
        u = g.double() + s["momentum"] * m
        tall = u.shape[0] > u.shape[1]
        x = (u.t() if tall else u).contiguous()
        x = x / (torch.linalg.vector_norm(x) + s["eps"])
        for _ in range(NS_STEPS):  # c A (A x) for c (A A) x
            A = torch.matmul(x, x.t().contiguous())
            AX = torch.matmul(A, x)
            x = NS[0] * x + NS[1] * AX + NS[2] * torch.matmul(A, AX)
        x = x.t() if tall else x
        out[0].append((1 - s["lr"] * s["wd"]) * p.double() - s["lr"] * max(1.0, u.shape[0] / u.shape[1]) ** 0.5 * x)
        out[1].append(m)
    return out


def exact(case, seed):
    s = _inputs(case, seed)
    return {"gated": _exact_gated, "norms": _exact_norms, "muon": _exact_muon}[case["op"].split("_")[0]](case, s)
