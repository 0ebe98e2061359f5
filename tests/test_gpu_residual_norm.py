"""GPU: the norms around a block with its gate and residual scale
(ionn_residual_norm_fwd / _bwd) against the oracle.

Tolerances, with u = 2^-24 and sums over a row of at most 40 roundings one
after the other (16 columns in a thread, 6 steps in a wavefront, 16 wavefronts,
the division): a deviation from the mean is off by D = 42 u (|v| + mean |v|), a
row's rstd by rstd rms(D) + 25 u of itself, and the formulas carry those on (in
forward_bounds and backward_bounds, each line beside its formula).  The
statistics that the backward pass is given are exact inputs.  A column's sum is
off by (rows + 40) u of its terms' magnitudes at most.  The store adds half a
step of the output's type and of its smallest value."""
import itertools

import numpy as np
import pytest
import torch

from gpu_helpers import dev, host, say, to_dev
from integer_only_nn_amd import ops
from oracle import floats as of
from test_gpu_dfp8_linear import SMALLEST, TYPES, _half, _np, _round, _typed, _ws

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
EPS = 1e-5


def _case(rows, cols, name, norm_a, norm_y, gate_rows=None, alpha=1.0, far=0.0, seed=0, block=True):
    """gate_rows None: no gate."""
    rng = np.random.default_rng(seed + 31 * rows + cols)
    f32 = lambda *s: rng.standard_normal(s).astype(np.float32)  # noqa: E731
    share = gate_rows if gate_rows and gate_rows < rows else max(rows, 1)
    d = dict(a=_round(far + rng.standard_normal((rows, cols)), name) if block else None,
             x=_round(far + 2.0 * rng.standard_normal((rows, cols)), name), norm_a=norm_a, norm_y=norm_y, alpha=alpha,
             gate=None if gate_rows is None else f32(-(-rows // share), cols), gate_rows=gate_rows or 0)
    for k, kind in (("a", norm_a), ("y", norm_y)):
        d["gamma_" + k] = 1 + 0.1 * f32(cols) if kind != "none" else None
        d["beta_" + k] = 0.1 * f32(cols) if kind == "layer" else None
    return d


FWD = ("norm_a", "gamma_a", "beta_a", "gate", "gate_rows", "alpha", "norm_y", "gamma_y", "beta_y")


def _oracle(d):
    return of.residual_norm_fwd(d["a"], d["x"], *(d[k] for k in FWD), EPS)


def _args(d):
    """The vectors and settings of a call, on the device."""
    return {k: to_dev(d[k]) if isinstance(d[k], np.ndarray) else d[k] for k in FWD}


def _forward(d, name, inplace=None, stream=None):
    rows, cols = d["x"].shape
    a, x = _typed(d["a"], name), _typed(d["x"], name)
    new = lambda *s, t=torch.float32: torch.full(s, 3.0, dtype=t, device=dev())  # noqa: E731
    y = {"y=x": x, "y=a": a}.get(inplace, None)
    y = new(rows, cols, t=TYPES[name]) if y is None else y
    n = {"y=x": a, "n=x": x}.get(inplace, None) if inplace else None
    n = (new(rows, cols, t=TYPES[name]) if n is None else n) if d["norm_y"] != "none" else None
    s = {}
    for k in "ay":
        s["mean_" + k] = new(rows) if d["norm_" + k] == "layer" else None
        s["rstd_" + k] = new(rows) if d["norm_" + k] != "none" else None
    m = torch.zeros(1, dtype=torch.int32, device=dev()) if n is not None else None
    say("residual norm fwd", rows, cols, name, d["norm_a"], d["norm_y"], d["gate_rows"])
    ops.ionn_residual_norm_fwd(a, x, y, n, **_args(d), eps=EPS, **s, absmax_n=m, stream=stream)
    return dict(y=y, n=n, m=m, **s)


def _norm_bounds(v, err, kind, gamma, beta):
    """Of the mean, the rstd and the output of a norm of v known to err."""
    if kind == "none":
        return None, None, err
    lay = kind == "layer"
    mean = v.mean(1, keepdims=True) if lay else 0.0
    dmean = (err.mean(1, keepdims=True) + 41 * U * np.abs(v).mean(1, keepdims=True)) if lay else 0.0
    D = err + dmean + U * (np.abs(v) + np.abs(mean))
    d = v - mean
    rstd = 1 / np.sqrt(np.square(d).mean(1, keepdims=True) + EPS)
    rel = rstd * np.sqrt(np.square(D).mean(1, keepdims=True)) + 25 * U  # |d rms| rstd <= 1
    h = d * rstd
    dh = rstd * D * (1 + rel) + np.abs(h) * (rel + 2 * U)
    g = 1.0 if gamma is None else np.abs(gamma.astype(np.float64))
    b = 0.0 if beta is None else np.abs(beta.astype(np.float64))
    return (dmean[:, 0] if lay else None), (rstd * rel)[:, 0], g * dh + 3 * U * (g * np.abs(h) + b)


def forward_bounds(d, want):
    x = np.abs(d["alpha"] * d["x"])
    out, err = {}, 2 * U * x
    if d["a"] is not None:
        out["mean_a"], out["rstd_a"], dp = _norm_bounds(d["a"], 0 * x, d["norm_a"], d["gamma_a"], d["beta_a"])
        gate = of._per_row(d["gate"], d["gate_rows"], len(x))
        p = want["y"] - d["alpha"] * d["x"]
        err = err + np.abs(gate) * dp + 4 * U * (x + np.abs(p))
    out["y"] = err
    out["mean_y"], out["rstd_y"], out["n"] = _norm_bounds(want["y"], err, d["norm_y"], d["gamma_y"], d["beta_y"])
    return out


def _close(got, want, tol, name, what):
    got = _np(got)
    bad = np.abs(got - want) - tol - _half(name) * (np.abs(want) + tol) - SMALLEST[name]
    assert (bad <= 0).all(), f"{what}: off by {bad.max()} beyond the tolerance"


def _check_forward(d, name, **kw):
    got, want = _forward(d, name, **kw), _oracle(d)
    tol = forward_bounds(d, want)
    for k in ("y", "n"):
        if got[k] is not None:
            _close(got[k], want[k], tol[k], name, k)
    for k in ("mean_a", "rstd_a", "mean_y", "rstd_y"):
        if got[k] is not None:
            _close(got[k], want[k], tol[k], "f32", k)
    if got["m"] is not None and want["n"].size:
        top = np.abs(want["n"]).max()
        assert abs(float(host(got["m"]).view(np.float32)[0]) - top) <= tol["n"].max() + U * top


SHAPES = [(1, 1), (1, 8), (3, 7), (5, 64), (2, 100), (17, 256), (9, 257), (33, 512), (4, 513), (65, 1000), (5, 1025), (3, 2049),
          (6, 4096), (2, 4097), (3, 8192), (2, 8200), (2, 16384), (1500, 130), (700, 1024)]
KINDS = list(itertools.product(("none", "layer", "rms"), repeat=2))


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("name", list(TYPES))
def test_forward(rows, cols, name):
    for i, (ka, ky) in enumerate(KINDS):
        gate_rows = (None, 0, 1, 3, rows)[i % 5]
        _check_forward(_case(rows, cols, name, ka, ky, gate_rows, alpha=(1.0, 0.5, -2.0)[i % 3]), name)


# several rows in a wavefront: parts of 8, 16 and 32 threads, gates that end among a wavefront's rows, more
# gates than workgroups, rows behind the last that fill no part, a second round of rows
SHORT = [(1, 2, 0), (77, 5, 3), (1003, 31, 5), (1003, 33, 1), (700, 63, 300), (700, 65, 0), (130, 127, 7), (2001, 129, 2),
         (61, 255, 60), (40000, 24, 600), (40000, 9, 70)]


@pytest.mark.parametrize("rows,cols,gate_rows", SHORT)
@pytest.mark.parametrize("name", list(TYPES))
def test_forward_of_short_rows(rows, cols, gate_rows, name):
    for ka, ky in (("layer", "rms"), ("rms", "layer"), ("none", "rms")):
        _check_forward(_case(rows, cols, name, ka, ky, gate_rows or None, alpha=0.5), name)


# rows of three, five, six, ten and twelve wavefronts, full and not (16-bit types)
WIDE = [(70, 1500, 9), (70, 2560, 70), (33, 2300, 1), (20, 3000, 7), (600, 5120, 1), (40, 5000, 0), (9, 6000, 2), (6, 6144, 6)]


@pytest.mark.parametrize("rows,cols,gate_rows", WIDE)
@pytest.mark.parametrize("name", ["bf16", "f16"])
def test_rows_of_some_wavefronts(rows, cols, gate_rows, name):
    for ka, ky in (("layer", "rms"), ("rms", "layer"), ("rms", "rms")):
        d = _case(rows, cols, name, ka, ky, gate_rows or None, alpha=0.5)
        _check_forward(d, name)
        _check_backward(_errors(d, name), name)


@pytest.mark.parametrize("name", list(TYPES))
def test_forward_of_the_first_norm(name):
    """No block yet: the norm of the stream alone."""
    for kind in ("layer", "rms", "none"):
        for rows, cols in ((1, 1), (7, 300), (40, 4096)):
            _check_forward(_case(rows, cols, name, "none", kind, block=False), name)


def test_forward_far_from_zero():
    """Rows whose mean is a thousand deviations."""
    for rows, cols in ((5, 64), (9, 1000), (4, 4096)):
        _check_forward(_case(rows, cols, "f32", "layer", "layer", 2, far=1000.0), "f32")


def test_forward_in_place():
    for inplace in ("y=x", "y=a", "n=x"):
        for rows, cols in ((300, 100), (600, 4096), (3, 9000)):
            _check_forward(_case(rows, cols, "bf16", "rms", "layer", 7), "bf16", inplace=inplace)


def test_forward_outputs_are_optional():
    d = _case(6, 70, "f32", "rms", "rms", 2)
    whole = _forward(d, "f32")
    a, x = to_dev(d["a"]).float(), to_dev(d["x"]).float()
    for keep in "yn":
        out = torch.full((6, 70), 3.0, device=dev())
        ops.ionn_residual_norm_fwd(a, x, out if keep == "y" else None, out if keep == "n" else None, **_args(d), eps=EPS)
        assert torch.equal(out, whole[keep])


def test_forward_empty_and_constant_rows():
    for rows, cols in ((0, 8), (4, 0)):
        assert tuple(_forward(_case(rows, cols, "f32", "rms", "rms"), "f32")["y"].shape) == (rows, cols)
    d = _case(3, 50, "f32", "layer", "rms")
    d["a"][:], d["x"][:] = 0.0, 0.0  # no deviation: rstd = 1 / sqrt(eps), n = the shift's norm
    _check_forward(d, "f32")


def test_what_is_not_finite_stays_in_its_row():
    for cols in (100, 4096):
        d = _case(6, cols, "f32", "layer", "rms", 2)
        d["a"][2, 5], d["x"][4, 7] = np.inf, np.nan
        got = _forward(d, "f32")
        bad = np.array([False, False, True, False, True, False])
        assert (np.isnan(host(got["n"])).any(1) == bad).all() and np.isfinite(host(got["n"])[~bad]).all()
        assert int(host(got["m"])[0]) > 0x7f800000


def test_what_lies_behind_the_rows_is_left():
    for rows, cols in ((3, 70), (5, 513), (2, 4096)):
        d = _case(rows, cols, "f16", "rms", "layer", 1)
        y, n = (torch.full((rows * cols + 40,), 5.0, dtype=torch.float16, device=dev()) for _ in range(2))
        ops.ionn_residual_norm_fwd(_typed(d["a"], "f16"), _typed(d["x"], "f16"), y[:rows * cols].view(rows, cols),
                                   n[:rows * cols].view(rows, cols), **_args(d), eps=EPS)
        assert (y[rows * cols:] == 5).all() and (n[rows * cols:] == 5).all()


# ---- backward ----------------------------------------------------------------

BWD = ("norm_a", "gamma_a", "beta_a", "gate", "gate_rows", "alpha", "norm_y", "gamma_y")
SUMS = ("dgate", "dgamma_a", "dbeta_a", "dgamma_y", "dbeta_y")


def _errors(d, name, dy=True, seed=1):
    """The case with its errors, y as stored and float32 statistics."""
    rows, cols = d["x"].shape
    rng = np.random.default_rng(seed)
    w = _oracle(d)
    d = dict(d, y=_round(w["y"], name), dy=_round(0.1 * rng.standard_normal((rows, cols)), name) if dy else None,
             dn=_round(0.1 * rng.standard_normal((rows, cols)), name) if d["norm_y"] != "none" else None)
    for k in ("mean_a", "rstd_a", "mean_y", "rstd_y"):
        keep = w[k] is not None and (k[0] == "r" or d["norm_" + k[-1]] == "layer")
        d[k] = w[k].astype(np.float32) if keep else None
    return d


def _oracle_bwd(d):
    return of.residual_norm_bwd(d["dy"], d["dn"], d["a"], d["y"], *(d[k] for k in BWD),
                                *(d[k] for k in ("mean_a", "rstd_a", "mean_y", "rstd_y")))


def _wanted(d):
    """The outputs that the case has."""
    w = ["dx"] + (["da"] if d["a"] is not None else [])
    w += ["dgate"] if d["gate"] is not None else []
    for k in "ay":
        w += ["dgamma_" + k] if d["norm_" + k] != "none" else []
        w += ["dbeta_" + k] if d["norm_" + k] == "layer" else []
    return w


def _run(d, name, want=None, inplace=(), stream=None):
    rows, cols = d["x"].shape
    want = _wanted(d) if want is None else want
    t = {k: _typed(d[k], name) for k in ("dy", "dn", "a", "y")}
    out = dict.fromkeys(("da", "dx") + SUMS)
    for k in want:
        if k in SUMS:
            out[k] = torch.full(d["gate"].shape if k == "dgate" else (cols,), 7.0, device=dev())
        else:
            at = dict(inplace).get(k)
            out[k] = t[at] if at else torch.full((rows, cols), 7.0, dtype=TYPES[name], device=dev())
    stats = {k: None if d[k] is None else to_dev(d[k]) for k in ("mean_a", "rstd_a", "mean_y", "rstd_y")}
    kw = {k: to_dev(d[k]) if isinstance(d[k], np.ndarray) else d[k] for k in BWD}
    ws = _ws(ops.ionn_residual_norm_bwd_workspace_bytes(rows, cols, d["gate_rows"] if d["gate"] is not None else 0))
    say("residual norm bwd", rows, cols, name, d["norm_a"], d["norm_y"], d["gate_rows"])
    ops.ionn_residual_norm_bwd(t["dy"], t["dn"], t["a"], t["y"], out["da"], out["dx"], **kw, **stats,
                               **{k: out[k] for k in SUMS}, workspace=ws, stream=stream)
    return out


def backward_bounds(d):
    rows = len(d["x"])
    one = lambda v: 1.0 if v is None else np.abs(v.astype(np.float64))  # noqa: E731
    m = lambda v: v.mean(1, keepdims=True)  # noqa: E731

    def norm(v, kind, mean, rstd):
        if kind == "none":
            return v, None
        r = rstd.astype(np.float64)[:, None]
        return (v - (mean.astype(np.float64)[:, None] if kind == "layer" else 0.0)) * r, r

    def back(e, de, h, r, lay):
        """rstd (e - mean e - h mean(e h)), e known to de, h to 2 u of itself: 60 u covers the sums and the rest."""
        if r is None:
            return de
        e, h = np.abs(e), np.abs(h)
        sure = e + (m(e) if lay else 0.0) + h * m(e * h)
        return r * (de + (m(de) if lay else 0.0) + h * m(de * h) + 60 * U * sure)

    out = {}
    t, dt = (0.0, 0.0) if d["dy"] is None else (np.abs(d["dy"]), 0 * d["dy"])
    col = lambda terms, err: (rows + 40) * U * np.abs(terms).sum(0) + err.sum(0)  # noqa: E731
    if d["norm_y"] != "none":
        hy, ry = norm(d["y"], d["norm_y"], d["mean_y"], d["rstd_y"])
        e = np.abs(d["dn"]) * one(d["gamma_y"])
        b = back(e, 2 * U * e, hy, ry, d["norm_y"] == "layer")
        lay = d["norm_y"] == "layer"
        mag = ry * (e + (m(e) if lay else 0.0) + np.abs(hy) * m(e * np.abs(hy)))
        t, dt = t + mag, dt + b + 2 * U * (t + mag)
        out["dgamma_y"], out["dbeta_y"] = col(d["dn"] * hy, 3 * U * np.abs(d["dn"] * hy)), col(d["dn"], 0 * e)
    out["dx"] = abs(d["alpha"]) * dt + 2 * U * abs(d["alpha"]) * t
    if d["a"] is None:
        return out
    ha, ra = norm(d["a"], d["norm_a"], d["mean_a"], d["rstd_a"])
    gate = np.abs(of._per_row(d["gate"], d["gate_rows"], rows)) * np.ones_like(d["a"])
    ha, g = np.abs(ha), one(d["gamma_a"])
    e, de = t * gate * g, (dt + 3 * U * t) * gate * g
    out["da"] = back(e, de, ha, ra, d["norm_a"] == "layer")
    out["dgamma_a"] = col(t * gate * ha, (dt + 6 * U * t) * gate * ha)
    out["dbeta_a"] = col(t * gate, (dt + 6 * U * t) * gate)
    if d["gate"] is not None:
        p = ha * g + (0.0 if d["beta_a"] is None else np.abs(d["beta_a"].astype(np.float64)))
        share = d["gate_rows"] if 0 < d["gate_rows"] < rows else rows
        out["dgate"] = np.zeros(d["gate"].shape)
        np.add.at(out["dgate"], np.arange(rows) // share, ((min(share, rows) + 46) * U * t + dt) * p)
    return out


def _check_backward(d, name, **kw):
    got, want, tol = _run(d, name, **kw), _oracle_bwd(d), backward_bounds(d)
    for k, v in got.items():
        if v is not None:
            _close(v, want[k], tol[k], "f32" if k in SUMS else name, k)


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("name", list(TYPES))
def test_backward(rows, cols, name):
    for i, (ka, ky) in enumerate(KINDS):
        gate_rows = (0, None, 3, 1, rows)[i % 5]
        d = _errors(_case(rows, cols, name, ka, ky, gate_rows, alpha=(1.0, 0.5, -2.0)[i % 3]), name,
                    dy=ky == "none" or i % 2 == 0)
        _check_backward(d, name)


@pytest.mark.parametrize("rows,cols,gate_rows", SHORT)
@pytest.mark.parametrize("name", list(TYPES))
def test_backward_of_short_rows(rows, cols, gate_rows, name):
    for ka, ky in (("layer", "rms"), ("rms", "rms"), ("none", "layer")):
        _check_backward(_errors(_case(rows, cols, name, ka, ky, gate_rows or None, alpha=0.5), name), name)


# a gate for few rows: more gates than workgroups, whole ones in a row group each; many runs of a few gates
@pytest.mark.parametrize("rows,cols,gate_rows", [(1300, 100, 2), (1300, 1024, 1), (700, 600, 1), (2000, 2100, 3), (1100, 5000, 2),
                                                 (4000, 64, 1000), (513, 70, 1), (512, 70, 1), (5000, 300, 2500), (9000, 48, 600)])
@pytest.mark.parametrize("name", ["f32", "bf16"])
def test_backward_of_many_gates(rows, cols, gate_rows, name):
    for ka, ky in (("layer", "layer"), ("none", "rms"), ("rms", "none")):
        _check_backward(_errors(_case(rows, cols, name, ka, ky, gate_rows, alpha=0.5), name), name)


@pytest.mark.parametrize("name", list(TYPES))
def test_backward_of_the_first_norm(name):
    for kind in ("layer", "rms"):
        for rows, cols in ((1, 1), (7, 300), (400, 1024), (40, 4096)):
            _check_backward(_errors(_case(rows, cols, name, "none", kind, block=False), name), name)


def test_backward_in_place():
    for inplace in ((("dx", "dy"),), (("da", "dn"), ("dx", "dy")), (("da", "a"), ("dx", "y")), (("dx", "dn"),)):
        for rows, cols in ((300, 100), (600, 4096)):
            _check_backward(_errors(_case(rows, cols, "bf16", "rms", "layer", 7), "bf16"), "bf16", inplace=inplace)


def test_backward_outputs_are_optional():
    d = _errors(_case(40, 300, "f32", "layer", "layer", 3), "f32")
    whole = _run(d, "f32")
    for want in (["dx"], ["da"], ["dgate"], ["dgamma_a", "dbeta_y"], ["dbeta_a"], ["dgamma_y"]):
        part = _run(d, "f32", want=want)
        for k in want:
            assert torch.equal(part[k], whole[k]), k


def test_backward_of_no_rows():
    d = _errors(_case(0, 30, "f32", "layer", "rms"), "f32")
    got = _run(d, "f32")
    for k in ("dgamma_a", "dbeta_a", "dgamma_y"):
        assert not host(got[k]).any()


def test_backward_against_differences():
    """dx, da and the vectors' gradients of sum(dy y + dn n) against central
    differences of the float64 formula: h^2 times third derivatives (rows of unit
    scale: below 60 times the terms' sum) and 1e-16 / h of cancellation."""
    rows, cols, h = 4, 6, 2.0 ** -13
    for ka, ky in KINDS:
        d = _errors(_case(rows, cols, "f32", ka, ky, 3, alpha=0.5), "f32")
        # statistics and y of the formula itself
        got = {k: None if v is None else _np(v) for k, v in _run(d, "f32").items()}

        def loss(**change):
            w = _oracle({**d, **change})
            return (d["dy"] * w["y"]).sum() + (0.0 if d["dn"] is None else (d["dn"] * w["n"]).sum())
        scale = np.abs(d["dy"]).sum() + (0.0 if d["dn"] is None else np.abs(d["dn"]).sum())
        for k, g in (("x", "dx"), ("a", "da"), ("gate", "dgate"), ("gamma_a", "dgamma_a"), ("beta_a", "dbeta_a"),
                     ("gamma_y", "dgamma_y"), ("beta_y", "dbeta_y")):
            if got[g] is None:
                continue
            base = d[k].astype(np.float64)
            for at in np.ndindex(base.shape):
                step = np.zeros(base.shape)
                step[at] = h
                diff = (loss(**{k: base + step}) - loss(**{k: base - step})) / (2 * h)
                assert abs(diff - got[g][at]) <= scale * (60 * h * h + 2.0 ** -18), (ka, ky, k, at)


def test_repeatable_and_on_another_stream():
    d = _errors(_case(3000, 520, "bf16", "rms", "layer", 500), "bf16")
    a, b = _run(d, "bf16"), _run(d, "bf16")
    for k in a:
        assert a[k] is None or torch.equal(a[k], b[k])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        c, f = _run(d, "bf16"), _forward(d, "bf16")
    s.synchronize()
    for k in a:
        assert a[k] is None or torch.equal(a[k], c[k])
    g = _forward(d, "bf16")
    assert torch.equal(f["y"], g["y"]) and torch.equal(f["n"], g["n"])


@pytest.mark.parametrize("rows,cols,gate_rows", [(64, 4096, 0), (1500, 100, 2), (900, 256, 300)])
def test_captured_and_replayed(rows, cols, gate_rows):
    g = torch.Generator(device=dev()).manual_seed(5)
    rnd = lambda *s, t=torch.bfloat16: torch.randn(s, device=dev(), generator=g).to(t)  # noqa: E731
    f32 = torch.float32
    a, x, dy, dn = (rnd(rows, cols) for _ in range(4))
    y, n, da, dx = (torch.zeros_like(a) for _ in range(4))
    gates = -(-rows // gate_rows) if gate_rows else 1
    gate, ga, gy = rnd(gates, cols, t=f32), rnd(cols, t=f32), rnd(cols, t=f32)
    ra, ry, dgate, dga, dgy = (torch.zeros(s, device=dev()) for s in ((rows,), (rows,), (gates, cols), (cols,), (cols,)))
    ws = _ws(ops.ionn_residual_norm_bwd_workspace_bytes(rows, cols, gate_rows))

    def step():
        ops.ionn_residual_norm_fwd(a, x, y, n, gamma_a=ga, gate=gate, gate_rows=gate_rows, gamma_y=gy, rstd_a=ra, rstd_y=ry)
        ops.ionn_residual_norm_bwd(dy, dn, a, y, da, dx, gamma_a=ga, gate=gate, gate_rows=gate_rows, gamma_y=gy, rstd_a=ra,
                                   rstd_y=ry, dgamma_a=dga, dgate=dgate, dgamma_y=dgy, workspace=ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    outs = (y, n, ra, ry, da, dx, dgate, dga, dgy)
    for k in range(3):
        a.copy_(rnd(rows, cols))
        dn.copy_(rnd(rows, cols))
        graph.replay()
        got = [t.clone() for t in outs]
        torch.cuda.synchronize()
        step()
        assert all(torch.equal(p, q) for p, q in zip(got, outs))
