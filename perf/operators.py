"""Timed cases of the operators around the DFP-8 products: the Linear layer
with its epilogue (forward and backward), layer norm (forward and backward)
and the AdamW step.

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
BLOCK = 256          # values that share one exponent of an 8-bit optimiser state
TINY = 2.0 ** -9     # the smallest E4M3 value
DEV = "cuda:0"

# The weights of the 20 layers of a CIFAR ResNet-20.
RESNET20 = [432] + [2304] * 6 + [4608] + [9216] * 5 + [18432] + [36864] * 5 + [640]


def _linear(name, op, B, IN, OUT, act, dtype, bias=True, residual=False, save_z=False):
    return {"name": name, "op": op, "B": B, "IN": IN, "OUT": OUT, "act": act, "dtype": dtype, "bias": bias,
            "residual": residual, "save_z": save_z}


def listed():
    return [
        # one token through the up projection of a transformer block: the weights' bytes and the launch
        _linear("linear fwd 1x4096x4096", "linear_fwd", 1, 4096, 4096, "gelu", "bf16"),
        # the first layer of the 784-256-128-10 perceptron, its batch of 256, FP32 activations
        _linear("linear fwd 256x784x256", "linear_fwd", 256, 784, 256, "relu", "f32"),
        # the down projection of a ragged batch: odd rows, columns and reduction, added to the residual stream
        _linear("linear fwd 1000x1023x2049", "linear_fwd", 1000, 1023, 2049, "none", "f16", residual=True),
        # the up projection of a training step over 8192 tokens, which keeps what its backward pass needs
        _linear("linear fwd 8192x4096x4096", "linear_fwd", 8192, 4096, 4096, "gelu", "bf16", save_z=True),
        # the backward pass of that perceptron layer
        _linear("linear bwd 256x784x256", "linear_bwd", 256, 784, 256, "relu", "f32"),
        # the backward pass of the 8192-token up projection
        _linear("linear bwd 8192x4096x4096", "linear_bwd", 8192, 4096, 4096, "gelu", "bf16"),
        # the norm before one token's projection
        {"name": "norm fwd 1x4096", "op": "norm_fwd", "rows": 1, "cols": 4096, "dtype": "bf16"},
        # the norm of a training step over 8192 tokens, and its gradient
        {"name": "norm fwd 8192x4096", "op": "norm_fwd", "rows": 8192, "cols": 4096, "dtype": "bf16"},
        {"name": "norm bwd 8192x4096", "op": "norm_bwd", "rows": 8192, "cols": 4096, "dtype": "bf16"},
        # many short rows (25088 positions of 256 channels) in FP32
        {"name": "norm bwd 25088x256", "op": "norm_bwd", "rows": 25088, "cols": 256, "dtype": "f32"},
        # the optimiser step of a small model: many small tensors, states in 32 bits
        {"name": "adamw 32-bit 268k", "op": "adamw", "sizes": ",".join(map(str, RESNET20)), "bits": 32,
         "grad": "f32"},
        # the optimiser step of four 4096 x 4096 layers, states in 8 bits, bfloat16 gradients
        {"name": "adamw 8-bit 67M", "op": "adamw", "sizes": ",".join(["16777216"] * 4), "bits": 8, "grad": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear_fwd", "linear_bwd", "norm_fwd", "norm_bwd", "adamw"])
    if op == "adamw":
        sizes = [_log(rng, 64, 1 << 22) for _ in range(rng.randint(1, 16))]
        return {"op": op, "sizes": ",".join(map(str, sizes)), "bits": rng.choice([8, 32]),
                "grad": rng.choice(["f32", "bf16", "f16"])}
    if op.startswith("norm"):
        return {"op": op, "rows": _log(rng, 1, 8192), "cols": _log(rng, 8, 4096), "dtype": rng.choice(list(DT))}
    dtype = rng.choice(list(DT))
    case = {"op": op, "B": _log(rng, 1, 8192), "IN": _log(rng, 16, 4096), "OUT": _log(rng, 16, 4096),
            # FP32 gradients of the backward pass go with activations whose
            # derivative is exact: elsewhere one step of the 8-bit delta
            # weighs more than FP32 resolves
            "act": rng.choice(("none", "relu") if op == "linear_bwd" and dtype == "f32" else ACTS), "dtype": dtype,
            "bias": rng.random() < 0.7, "residual": rng.random() < 0.5, "save_z": rng.random() < 0.5}
    if op == "linear_bwd":
        case.update(bias=True, residual=False, save_z=False)
    return case


# ---- inputs -----------------------------------------------------------------

def _pow2(e):
    """2^e as float32 for an int32 tensor e in [-126, 127]."""
    return ((e + 127) << 23).view(torch.float32)


def _mantissas(g, rows, cols, std):
    return torch.randn(rows, cols, generator=g, device=DEV).mul_(std).round_().clamp_(-128, 127).to(torch.int8)


def _prepare_linear(c, g):
    B, IN, OUT, t = c["B"], c["IN"], c["OUT"], DT[c["dtype"]]
    # activations of unit scale at 2^-5, weights at the exponent that keeps z near 1
    s = {"X": _mantissas(g, B, IN, 32.0), "W": _mantissas(g, OUT, IN, 24.0),
         "eX": torch.tensor([-5], dtype=torch.int32, device=DEV),
         "eW": torch.tensor([-round(math.log2(24.0 * math.sqrt(IN)))], dtype=torch.int32, device=DEV)}
    if c["op"] == "linear_fwd":
        s["bias"] = torch.randn(OUT, generator=g, device=DEV) * 0.5 if c["bias"] else None
        s["R"] = torch.randn(B, OUT, generator=g, device=DEV).to(t) if c["residual"] else None
    else:
        s["Z"] = torch.randn(B, OUT, generator=g, device=DEV).to(t)
        # per-token error of varying size, as a loss leaves it
        s["dY"] = (torch.randn(B, OUT, generator=g, device=DEV)
                   * (0.02 + 0.05 * torch.rand(B, 1, generator=g, device=DEV))).to(t)
    return s


def _prepare_norm(c, g):
    n, m, t = c["rows"], c["cols"], DT[c["dtype"]]
    x = torch.randn(n, m, generator=g, device=DEV) * 1.5 + 0.25 * torch.randn(n, 1, generator=g, device=DEV)
    x[:, torch.randint(0, m, (max(1, m // 128),), generator=g, device=DEV)] *= 8.0  # outlier channels
    s = {"x": x.to(t), "gamma": 1.0 + 0.1 * torch.randn(m, generator=g, device=DEV),
         "beta": 0.1 * torch.randn(m, generator=g, device=DEV)}
    if c["op"] == "norm_bwd":
        xd = s["x"].double()
        mean = xd.mean(1, keepdim=True)
        s["rstd"] = ((xd - mean).square().mean(1) + 1e-5).rsqrt().float()
        s["mean"] = mean[:, 0].float()
        s["dy"] = (0.05 * torch.randn(n, m, generator=g, device=DEV)).to(t)
    return s


def _encode(x):
    """E4M3 codes of x [blocks, BLOCK] with one exponent per block, in float32."""
    bits = x.abs().amax(1).view(torch.int32)
    e = ((bits >> 23) - 135 + ((bits & 0x7fffff) > 0x600000).int()).clamp_min(-126)
    e = torch.where(bits == 0, 0, e)
    return (x * _pow2(-e)[:, None]).to(torch.float8_e4m3fn), e.to(torch.int8)


def _encode_root(r):
    """The same for roots of second moments: a positive one never becomes 0."""
    q, e = _encode(r)
    return torch.where((q.float() == 0) & (r > 0), TINY, q.float()).to(torch.float8_e4m3fn), e


def _blocks(ts, dtype=torch.float32):
    """The tensors one after the other as [blocks, BLOCK], each padded to whole blocks."""
    return torch.cat([torch.nn.functional.pad(t.reshape(-1).to(dtype), (0, -t.numel() % BLOCK)) for t in ts]).view(-1, BLOCK)


def _split(x, sizes):
    """Undoes _blocks: one flat tensor for each size."""
    parts = x.reshape(-1).split([-(-n // BLOCK) * BLOCK for n in sizes])
    return [p[:n] for p, n in zip(parts, sizes)]


def _prepare_adamw(c, g):
    sizes = [int(n) for n in c["sizes"].split(",")]
    s = {"sizes": sizes, "t": 1000, "lr": 1e-3, "beta1": 0.9, "beta2": 0.999, "eps": 1e-8, "wd": 0.01}
    new = lambda: [torch.randn(n, generator=g, device=DEV) for n in sizes]  # noqa: E731
    s["p"] = [0.02 * p for p in new()]
    s["g"] = [(1e-3 * x).to(DT[c["grad"]]) for x in new()]
    m, r = [3e-4 * x for x in new()], [1e-3 * x.abs() + 1e-7 for x in new()]
    if c["bits"] == 32:
        s["m"], s["v"] = m, [x * x for x in r]
        return s
    s["m"], s["r"], s["e"] = [], [], []
    for a, b in zip(m, r):
        (qa, ea), (qb, eb) = _encode(_blocks([a])), _encode_root(_blocks([b]))
        s["m"].append(qa.reshape(-1)[:a.numel()].clone())
        s["r"].append(qb.reshape(-1)[:b.numel()].clone())
        s["e"].append(torch.stack([ea, eb], 1).contiguous())  # [blocks][2]: of m, of r
    return s


def _buffers(c, s):
    """Outputs and workspaces that a program allocates once."""
    from integer_only_nn_amd import ops, steps
    empty = lambda *shape, dtype=torch.float32: torch.empty(shape, dtype=dtype, device=DEV)  # noqa: E731
    if c["op"].startswith("linear"):
        B, IN, OUT, t = c["B"], c["IN"], c["OUT"], DT[c["dtype"]]
        s["act"] = ops.ACTIVATIONS[c["act"]]
        if c["op"] == "linear_fwd":
            s["Y"], s["Zout"] = empty(B, OUT, dtype=t), empty(B, OUT, dtype=t) if c["save_z"] else None
            s["ws"] = empty(ops.dfp8_linear_fwd_workspace_bytes(B, IN, OUT), dtype=torch.uint8)
        else:
            s["dZ8"], s["edZ"] = empty(B, OUT, dtype=torch.int8), empty(1, dtype=torch.int32)
            s["dX"], s["G"], s["gb"] = empty(B, IN, dtype=t), empty(OUT, IN, dtype=t), empty(OUT)
            s["ws"] = empty(ops.dfp8_linear_bwd_workspace_bytes(B, IN, OUT), dtype=torch.uint8)
    elif c["op"] == "adamw":
        s["opt"] = steps.AdamW(s["p"], s["m"], s["v"] if c["bits"] == 32 else s["r"], s.get("e"), lr=s["lr"],
                               betas=(s["beta1"], s["beta2"]), eps=s["eps"], weight_decay=s["wd"], t=s["t"] - 1)
        s["opt"].bind_grads(s["g"])
    else:
        n, m, t = c["rows"], c["cols"], DT[c["dtype"]]
        if c["op"] == "norm_fwd":
            s["y"], s["mean"], s["rstd"] = empty(n, m, dtype=t), empty(n), empty(n)
        else:
            s["dx"], s["dgamma"], s["dbeta"] = empty(n, m, dtype=t), empty(m), empty(m)
            s["ws"] = empty(ops.ionn_layer_norm_bwd_workspace_bytes(n, m), dtype=torch.uint8)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    kind = case["op"].split("_")[0]
    s = {"linear": _prepare_linear, "norm": _prepare_norm, "adamw": _prepare_adamw}[kind](case, g)
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


def _linear_fwd(s, c):
    t = DT[c["dtype"]]
    z = (s["X"].float() @ s["W"].float().t()) * _pow2(s["eX"] + s["eW"])
    if s["bias"] is not None:
        z = z + s["bias"]
    y = _act(z, c["act"])
    if s["R"] is not None:
        y = y + s["R"].float()
    return [y.to(t), z.to(t)] if c["save_z"] else [y.to(t)]


def _linear_bwd(s, c):
    t = DT[c["dtype"]]
    dz = s["dY"].float() * _act_grad(s["Z"].float(), c["act"])
    bits = dz.abs().amax().view(torch.int32)
    e = torch.where(bits == 0, 0, (bits >> 23) - 133)
    q = (dz * _pow2(-e)).round().clamp(-128, 127)
    return [((q @ s["W"].float()) * _pow2(e + s["eW"])).to(t), ((q.t() @ s["X"].float()) * _pow2(e + s["eX"])).to(t),
            dz.sum(0)]


def _norm_fwd(s, c):
    x = s["x"].float()
    mean = x.mean(1, keepdim=True)
    d = x - mean
    rstd = 1 / torch.sqrt(d.square().mean(1, keepdim=True) + 1e-5)
    return [(d * rstd * s["gamma"] + s["beta"]).to(s["x"].dtype), mean[:, 0], rstd[:, 0]]


def _norm_bwd(s, c):
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    h = (s["x"].float() - s["mean"][:, None]) * rstd
    d = dy * s["gamma"]
    dx = rstd * (d - d.mean(1, keepdim=True) - h * (d * h).mean(1, keepdim=True))
    return [dx.to(s["x"].dtype), (dy * h).sum(0), dy.sum(0)]


def _adamw(s, c):
    sizes, t = s["sizes"], s["t"]
    p, g, m = _blocks(s["p"]), _blocks(s["g"]), _blocks(s["m"])
    if c["bits"] == 8:
        e = torch.cat(s["e"]).int()
        m = m * _pow2(e[:, :1])
        r = _blocks(s["r"]) * _pow2(e[:, 1:])
        v = r * r
    else:
        v = _blocks(s["v"])
    m = m * s["beta1"] + g * (1 - s["beta1"])
    v = v * s["beta2"] + (g * (1 - s["beta2"])) * g
    r = torch.sqrt(v)
    u = m / (r * (1 / math.sqrt(1 - s["beta2"] ** t)) + s["eps"])
    p = p * (1 - s["lr"] * s["wd"]) - u * (s["lr"] / (1 - s["beta1"] ** t))
    s["t"] = t + 1
    torch._foreach_copy_(s["p"], _split(p, sizes))
    if c["bits"] == 32:
        torch._foreach_copy_(s["m"], _split(m, sizes))
        torch._foreach_copy_(s["v"], _split(v, sizes))
        return [s["p"], s["m"], s["v"]]
    (qm, em), (qr, er) = _encode(m), _encode_root(r)
    s["m"], s["r"] = _split(qm, sizes), _split(qr, sizes)
    s["e"] = list(torch.stack([em, er], 1).split([-(-n // BLOCK) for n in sizes]))
    return [s["p"], s["m"], s["r"], s["e"]]


PLAIN = {"linear_fwd": _linear_fwd, "linear_bwd": _linear_bwd, "norm_fwd": _norm_fwd, "norm_bwd": _norm_bwd,
         "adamw": _adamw}


# ---- the library's calls ----------------------------------------------------

def _own(s, c):
    from integer_only_nn_amd import ops
    if c["op"] == "linear_fwd":
        ops.dfp8_linear_fwd(s["X"], s["eX"], s["W"], s["eW"], s["Y"], bias=s["bias"], act=s["act"], residual=s["R"],
                            Z=s["Zout"], workspace=s["ws"])
        return [s["Y"], s["Zout"]] if c["save_z"] else [s["Y"]]
    if c["op"] == "linear_bwd":
        ops.dfp8_linear_bwd(s["dY"], s["Z"], s["act"], s["X"], s["eX"], s["W"], s["eW"], s["dZ8"], s["edZ"],
                            dX=s["dX"], G=s["G"], gb=s["gb"], workspace=s["ws"])
        return [s["dX"], s["G"], s["gb"]]
    if c["op"] == "norm_fwd":
        ops.ionn_layer_norm_fwd(s["x"], s["y"], gamma=s["gamma"], beta=s["beta"], eps=1e-5, mean=s["mean"],
                                rstd=s["rstd"])
        return [s["y"], s["mean"], s["rstd"]]
    if c["op"] == "norm_bwd":
        ops.ionn_layer_norm_bwd(s["dy"], s["x"], s["mean"], s["rstd"], s["dx"], gamma=s["gamma"], dgamma=s["dgamma"],
                                dbeta=s["dbeta"], workspace=s["ws"])
        return [s["dx"], s["dgamma"], s["dbeta"]]
    s["opt"].step()
    return [s["p"], s["m"], s["v"]] if c["bits"] == 32 else [s["p"], s["m"], s["r"], s["e"]]


def run(state):
    c = state["case"]
    return _own(state, c) if own else PLAIN[c["op"]](state, c)


# ---- what a pass has to do --------------------------------------------------

def work(case):
    if case["op"] == "adamw":
        n = sum(map(int, case["sizes"].split(",")))
        state = 16 if case["bits"] == 32 else 4 + 4 / BLOCK
        return {"bytes": n * (8 + DT[case["grad"]].itemsize + state), "flops": 14 * n}
    t = DT[case["dtype"]].itemsize
    if case["op"].startswith("norm"):
        n = case["rows"] * case["cols"]
        fwd = case["op"] == "norm_fwd"
        return {"bytes": (2 if fwd else 3) * t * n + 8 * case["rows"] + (8 if fwd else 12) * case["cols"],
                "flops": (8 if fwd else 14) * n}
    B, IN, OUT = case["B"], case["IN"], case["OUT"]
    if case["op"] == "linear_fwd":
        outs = 1 + case["residual"] + case["save_z"]
        return {"bytes": B * IN + OUT * IN + 4 * OUT * case["bias"] + outs * t * B * OUT, "flops": 2 * B * IN * OUT}
    return {"bytes": (2 * t * B * OUT) + (1 + t) * (B * IN + OUT * IN) + 4 * OUT, "flops": 4 * B * IN * OUT}


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


def _exact_linear(c, s):
    scale = lambda *es: 2.0 ** sum(int(e) for e in es)  # noqa: E731
    X, W = s["X"].double(), s["W"].double()
    if c["op"] == "linear_fwd":
        z = torch.matmul(X, W.t().contiguous()) * scale(s["eX"], s["eW"])
        z = z + (s["bias"].double() if s["bias"] is not None else 0.0)
        y = _exact_act(z, c["act"])[0] + (s["R"].double() if s["R"] is not None else 0.0)
        return [y, z] if c["save_z"] else [y]
    dz = s["dY"].double() * _exact_act(s["Z"].double(), c["act"])[1]
    top = float(dz.abs().max())
    e = math.frexp(top)[1] - 7 if top else 0  # top = f 2^q with f in [1, 2): q - 6
    q = torch.clamp(torch.round(torch.ldexp(dz, torch.tensor(-e, device=DEV))), -128, 127)
    return [torch.matmul(q, W) * scale(e, s["eW"]), torch.matmul(q.t().contiguous(), X) * scale(e, s["eX"]), dz.sum(0)]


def _exact_norm(c, s):
    x = s["x"].double()
    if c["op"] == "norm_fwd":
        var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
        rstd = (var + 1e-5) ** -0.5
        return [(x - mean) * rstd * s["gamma"].double() + s["beta"].double(), mean[:, 0], rstd[:, 0]]
    rstd, dy = s["rstd"].double().unsqueeze(1), s["dy"].double()
    h = (x - s["mean"].double().unsqueeze(1)) * rstd
    d, n = dy * s["gamma"].double(), x.shape[1]
    # the projection of d off the constant vector and off h, row by row
    dx = rstd * (d - d.sum(1, keepdim=True) / n - h * ((d * h).sum(1, keepdim=True) / n))
    return [dx, (dy * h).sum(0), dy.sum(0)]


def _exact_e4m3(x, n, positive):
    """The value that a flat x of n elements stands for in codes, and the codes' own values."""
    b = torch.zeros(-(-n // BLOCK) * BLOCK, dtype=torch.float64, device=DEV)
    b[:n] = x
    b = b.view(-1, BLOCK)
    top = b.abs().max(1, keepdim=True).values
    f, q = torch.frexp(top)  # f in [0.5, 1)
    e = torch.where(top > 0, (q - 9 + (f > 0.875).int()).clamp(min=-126), 0)
    a = torch.ldexp(b.abs(), -e)
    step = torch.ldexp(torch.ones_like(a), torch.frexp(a)[1].clamp(min=-5) - 4)
    a = torch.round(a / step) * step
    if positive:
        a = torch.where((a == 0) & (b > 0), TINY, a)
    return torch.where(b < 0, -a, a).reshape(-1)[:n]


def _exact_adamw(c, s):
    out = [[], [], []] + ([[]] if c["bits"] == 8 else [])
    t = s["t"]
    for i, n in enumerate(s["sizes"]):
        p, g = s["p"][i].double(), s["g"][i].double()
        if c["bits"] == 8:
            e = s["e"][i].int().repeat_interleave(BLOCK, 0)[:n]
            m, v = torch.ldexp(s["m"][i].double(), e[:, 0]), torch.ldexp(s["r"][i].double(), e[:, 1]) ** 2
        else:
            m, v = s["m"][i].double(), s["v"][i].double()
        m = s["beta1"] * m + (1 - s["beta1"]) * g
        v = s["beta2"] * v + (1 - s["beta2"]) * g * g
        step = (m / (1 - s["beta1"] ** t)) / ((v / (1 - s["beta2"] ** t)).sqrt() + s["eps"])
        out[0].append(p - s["lr"] * s["wd"] * p - s["lr"] * step)
        out[1].append(_exact_e4m3(m, n, False) if c["bits"] == 8 else m)
        out[2].append(_exact_e4m3(v.sqrt(), n, True) if c["bits"] == 8 else v)
        if c["bits"] == 8:
            out[3].append(None)
    return out


def exact(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    kind = case["op"].split("_")[0]
    if kind == "linear":
        return _exact_linear(case, _prepare_linear(case, g))
    if kind == "norm":
        return _exact_norm(case, _prepare_norm(case, g))
    return _exact_adamw(case, _prepare_adamw(case, g))
