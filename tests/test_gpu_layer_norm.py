"""GPU: layer norm forward and backward against the oracle in float64.

Tolerances.  A row's sum has at most 32 terms in a thread and a tree of 10
levels after them for the rows held in registers (more terms for longer
rows): the mean, the variance and the two sums of the gradient are off by
less than 128 half steps of float32, 2^-17, of the mean magnitude of their
terms.  The store adds half a step of the output's type.  Column sums over R
rows: (R + 64) half steps of the sum of magnitudes."""
import numpy as np
import pytest
import torch

from gpu_helpers import dev, host, say, to_dev
from integer_only_nn_amd import ops
from oracle import floats as of

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SMALLEST = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}
S = 2.0 ** -17
# every way a row is held: part of a wavefront's vector, one, several, a
# workgroup, a large workgroup, a loop; and the sizes around their limits
COLS = [1, 2, 3, 7, 8, 63, 64, 100, 255, 256, 257, 512, 513, 1000, 1024, 1025, 2048, 2049, 4095, 4096, 4100, 8192, 8193,
        16385, 33000]


def _round(x, name):
    return torch.from_numpy(np.ascontiguousarray(x)).float().to(TYPES[name]).double().numpy()


def _typed(x, name):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).to(dev()).to(TYPES[name])


def _half(name):
    return torch.finfo(TYPES[name]).eps / 2


def _np(t):
    return host(t.double())


def _case(rows, cols, name, seed=0, affine=True):
    rng = np.random.default_rng(seed + 3 * rows + cols)
    return dict(x=_round(rng.standard_normal((rows, cols)) * 1.5 + rng.standard_normal((rows, 1)), name),
                dy=_round(0.1 * rng.standard_normal((rows, cols)), name),
                dres=_round(0.1 * rng.standard_normal((rows, cols)), name),
                gamma=(1 + 0.2 * rng.standard_normal(cols)).astype(np.float32) if affine else None,
                beta=rng.standard_normal(cols).astype(np.float32) if affine else None)


def _dev(a):
    return None if a is None else to_dev(a)


def _check_fwd(d, name, eps=1e-5, inplace=False, stats=True):
    rows, cols = d["x"].shape
    say("norm fwd", rows, cols, name)
    x = _typed(d["x"], name)
    y = x if inplace else torch.full_like(x, 7.0)
    mean, rstd = (torch.full((rows,), 7.0, device=dev()) if stats else None for _ in range(2))
    m = torch.zeros(1, dtype=torch.int32, device=dev())
    ops.ionn_layer_norm_fwd(x, y, gamma=_dev(d["gamma"]), beta=_dev(d["beta"]), eps=eps, mean=mean, rstd=rstd, absmax_y=m)
    want, mu, rs = of.layer_norm_fwd(d["x"], d["gamma"], d["beta"], eps)
    mag = np.abs(d["x"]).mean(1) if cols else np.zeros(rows)
    g = 1.0 if d["gamma"] is None else np.abs(d["gamma"])
    b = 0.0 if d["beta"] is None else np.abs(d["beta"])
    # the mean's error against the row's spread, and the relative one of the rest
    tol = S * (mag * rs)[:, None] * (1 + np.abs(want)) * g + S * (np.abs(want) + b)
    bad = np.abs(_np(y) - want) - tol - _half(name) * (np.abs(want) + tol) - SMALLEST[name]
    assert (bad <= 0).all(), f"y off by {bad.max()} beyond the tolerance"
    if stats:
        assert (np.abs(_np(mean) - mu) <= S * mag + 2.0 ** -149).all()
        assert (np.abs(_np(rstd) - rs) <= S * rs * (1 + mag * rs)).all()
    top = float(host(m).view(np.float32)[0])
    assert abs(top - np.abs(want).max(initial=0.0)) <= tol.max(initial=0.0)


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("name", list(TYPES))
def test_forward(cols, name):
    for rows in (1, 5, 37):
        _check_fwd(_case(rows, cols, name, affine=rows != 5), name, stats=rows != 37)


def test_forward_many_rows_and_in_place():
    _check_fwd(_case(5000, 96, "bf16"), "bf16")
    _check_fwd(_case(3000, 1000, "f16"), "f16", inplace=True)
    _check_fwd(_case(9, 40000, "bf16"), "bf16", inplace=True)
    _check_fwd(_case(70001, 8, "f32"), "f32")


def test_forward_constant_rows_and_far_means():
    x = np.full((4, 1000), 3.0)
    x[1] = 0.0
    x[2] = 1e4 + np.arange(1000) * 2.0 ** -9  # spread 2^-9 around 1e4: needs the squares around the mean
    x[3] = -1e-20
    d = dict(x=x, gamma=None, beta=None)
    y, rstd = torch.empty(4, 1000, device=dev()), torch.empty(4, device=dev())
    ops.ionn_layer_norm_fwd(_typed(x, "f32"), y, rstd=rstd, eps=1e-5)
    want = of.layer_norm_fwd(_round(x, "f32"), None, None, 1e-5)[0]
    assert (host(y)[[0, 1]] == 0).all()
    # the mean of row 2 is off by at most 2^-17 1e4 = 0.08 against a spread of
    # 0.56; what the float32 sums really lose is far less
    assert np.abs(host(y)[2] - want[2]).max() < 0.14
    assert np.isfinite(host(y)).all()
    del d


def test_forward_not_finite_rows_stay_apart():
    d = _case(6, 300, "f32")
    d["x"][1, 5], d["x"][3, 299], d["x"][4, 0] = np.nan, np.inf, -np.inf
    y = torch.empty(6, 300, device=dev())
    ops.ionn_layer_norm_fwd(_typed(d["x"], "f32"), y)
    y = host(y)
    assert np.isnan(y[[1, 3, 4]]).all() and np.isfinite(y[[0, 2, 5]]).all()


def test_empty():
    for rows, cols in ((0, 5), (5, 0)):
        x = torch.empty(rows, cols, device=dev())
        ops.ionn_layer_norm_fwd(x, torch.empty_like(x))
        dg, db = torch.full((cols,), 7.0, device=dev()), torch.full((cols,), 7.0, device=dev())
        ops.ionn_layer_norm_bwd(x, x, torch.empty(rows, device=dev()), torch.empty(rows, device=dev()),
                                torch.empty_like(x), dgamma=dg, dbeta=db)
        assert not host(dg).any() and not host(db).any()  # rows = 0: the sums are 0


def _check_bwd(d, name, sums=True, dres=True, inplace=None):
    rows, cols = d["x"].shape
    say("norm bwd", rows, cols, name)
    _, mean, rstd = of.layer_norm_fwd(d["x"], d["gamma"], d["beta"], 1e-5)
    mean, rstd = mean.astype(np.float32), rstd.astype(np.float32)
    x, dy, dr = _typed(d["x"], name), _typed(d["dy"], name), _typed(d["dres"], name) if dres else None
    dx = {"dy": dy, "dres": dr}.get(inplace)
    dx = torch.full_like(x, 7.0) if dx is None else dx
    dg, db = (torch.full((cols,), 7.0, device=dev()) if sums else None for _ in range(2))
    ws = torch.empty(ops.ionn_layer_norm_bwd_workspace_bytes(rows, cols), dtype=torch.uint8, device=dev())
    ops.ionn_layer_norm_bwd(dy, x, to_dev(mean), to_dev(rstd), dx, gamma=_dev(d["gamma"]), dres=dr, dgamma=dg, dbeta=db,
                            workspace=ws if sums else None)
    wx, wg, wb = of.layer_norm_bwd(d["dy"], d["x"], mean, rstd, d["gamma"], d["dres"] if dres else None)
    rs = rstd.astype(np.float64)[:, None]
    h = (d["x"] - mean.astype(np.float64)[:, None]) * rs
    # h itself: the subtraction's operands are exact, one half step of |x| + |mean|
    hm = np.abs(h) + (np.abs(d["x"]) + np.abs(mean)[:, None]) * rs
    dd = d["dy"] * (1.0 if d["gamma"] is None else d["gamma"].astype(np.float64))
    tol = S * rs * (np.abs(dd) + np.abs(dd).mean(1, keepdims=True) + hm * (np.abs(dd) * hm).mean(1, keepdims=True))
    if dres:
        tol = tol + 2.0 ** -23 * np.abs(d["dres"])
    bad = np.abs(_np(dx) - wx) - tol - _half(name) * (np.abs(wx) + tol) - SMALLEST[name]
    assert (bad <= 0).all(), f"dx off by {bad.max()} beyond the tolerance"
    if sums:
        k = (rows + 64) * 2.0 ** -24
        assert (np.abs(_np(dg) - wg) <= k * (np.abs(d["dy"]) * hm).sum(0)).all()
        assert (np.abs(_np(db) - wb) <= k * np.abs(d["dy"]).sum(0)).all()


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("name", list(TYPES))
def test_backward(cols, name):
    for rows in (1, 5, 37):
        _check_bwd(_case(rows, cols, name, affine=rows != 5), name, sums=rows != 1, dres=rows == 37)


def test_backward_many_rows():
    _check_bwd(_case(5000, 96, "bf16"), "bf16")
    _check_bwd(_case(3000, 1000, "f16"), "f16")
    _check_bwd(_case(70001, 8, "f32"), "f32")
    _check_bwd(_case(2100, 2048, "f32"), "f32", dres=False)


@pytest.mark.parametrize("cols", [64, 1000, 4096, 9000, 20000])
def test_backward_in_place(cols):
    for inplace in ("dy", "dres"):
        _check_bwd(_case(50, cols, "bf16"), "bf16", inplace=inplace)


def test_backward_matches_differences():
    """The kernels' gradient against central differences of the float64 forward."""
    d = _case(3, 40, "f32")
    _, mean, rstd = of.layer_norm_fwd(d["x"], d["gamma"], d["beta"], 1e-5)
    dx, dg, db = torch.empty(3, 40, device=dev()), torch.empty(40, device=dev()), torch.empty(40, device=dev())
    ws = torch.empty(ops.ionn_layer_norm_bwd_workspace_bytes(3, 40), dtype=torch.uint8, device=dev())
    ops.ionn_layer_norm_bwd(_typed(d["dy"], "f32"), _typed(d["x"], "f32"), to_dev(mean.astype(np.float32)),
                            to_dev(rstd.astype(np.float32)), dx, gamma=_dev(d["gamma"]), dgamma=dg, dbeta=db, workspace=ws)
    loss = lambda x, g: float((d["dy"] * of.layer_norm_fwd(x, g, None, 1e-5)[0]).sum())  # noqa: E731
    step = 1e-5
    for i in np.ndindex(3, 40):
        x = d["x"].copy()
        x[i] += step
        up = loss(x, d["gamma"])
        x[i] -= 2 * step
        # (the differences are good to 1e-8, the kernel to 2^-17 of terms below 1)
        assert float(dx[i]) == pytest.approx((up - loss(x, d["gamma"])) / (2 * step), abs=2e-5)
    g64 = d["gamma"].astype(np.float64)
    for c in range(40):
        g = g64.copy()
        g[c] += step
        up = loss(d["x"], g)
        g[c] -= 2 * step
        assert float(dg[c]) == pytest.approx((up - loss(d["x"], g)) / (2 * step), abs=2e-5)


def test_backward_repeatable():
    d = _case(4000, 500, "bf16")
    outs = []
    for _ in range(2):
        dx, dg, db = torch.empty(4000, 500, dtype=torch.bfloat16, device=dev()), torch.empty(500, device=dev()), torch.empty(500, device=dev())
        ws = torch.empty(ops.ionn_layer_norm_bwd_workspace_bytes(4000, 500), dtype=torch.uint8, device=dev())
        ops.ionn_layer_norm_bwd(_typed(d["dy"], "bf16"), _typed(d["x"], "bf16"), torch.zeros(4000, device=dev()),
                                torch.ones(4000, device=dev()), dx, gamma=_dev(d["gamma"]), dgamma=dg, dbeta=db, workspace=ws)
        outs.append((dx, dg, db))
    for a, b in zip(*outs):
        assert torch.equal(a, b)
