"""The residual norm's host-side checks (no GPU needed: none of these calls
reaches one), and the oracle's gradient against differences of its forward."""
import ctypes
import itertools

import numpy as np
import pytest

from integer_only_nn_amd import _lib, ops
from oracle import floats as of

lib = _lib.lib()
OK, ARG, SHAPE, RANGE, ALIGN, UNSUP, HIP, WS = range(8)
P = ctypes.c_void_p
A, X, Y, N, ODD = P(0x10000), P(0x20000), P(0x30000), P(0x40000), P(0x10001)  # never dereferenced
V = P(0x1000)
NONE, LAYER, RMS = range(3)
NAN, INF = float("nan"), float("inf")


def test_fwd():
    def f(a=A, x=X, na=RMS, ga=V, ba=None, gate=V, gr=2, al=1.0, ny=LAYER, gy=V, by=V, eps=1e-5, y=Y, n=N, ma=None, ra=V,
          my=V, ry=V, dt=0, rows=4, cols=8, m=None):
        return lib.ionn_residual_norm_fwd(a, x, na, ga, ba, gate, gr, al, ny, gy, by, eps, y, n, ma, ra, my, ry, dt, rows,
                                          cols, m, None)
    assert f(dt=3) == ARG and f(na=3) == ARG and f(ny=-1) == ARG
    assert f(rows=-1) == SHAPE and f(cols=16385) == SHAPE and f(rows=1 << 31) == SHAPE
    assert f(eps=-1.0) == RANGE and f(eps=NAN) == RANGE and f(al=INF) == RANGE and f(al=NAN) == RANGE and f(gr=-1) == RANGE
    assert f(a=None) == ARG and f(a=None, na=NONE, ga=None, ra=None) == ARG  # a norm, a gate of no block
    assert f(na=NONE) == ARG and f(ny=NONE) == ARG  # gains of no norm
    assert f(ny=NONE, gy=None, by=None, my=None, ry=None) == ARG  # n of no norm
    assert f(ba=V) == ARG and f(ma=V) == ARG and f(ny=RMS) == ARG  # a shift or a mean of an RMS norm
    assert f(x=None) == ARG and f(y=None, n=None) == ARG and f(n=None) == ARG  # (statistics of a norm that is not taken)
    assert f(x=ODD, dt=1) == ALIGN and f(gate=ODD) == ALIGN and f(ry=ODD) == ALIGN and f(m=ODD) == ALIGN
    assert f(n=Y) == ARG and f(y=P(0x20004)) == ARG and f(n=P(0x10004)) == ARG and f(n=P(0x30004)) == ARG
    assert f(rows=0, x=None) == OK and f(cols=0) == OK


def test_bwd():
    need = lib.ionn_residual_norm_bwd_workspace_bytes(4, 8, 2)
    assert need > 0 and lib.ionn_residual_norm_bwd_workspace_bytes(-1, 8, 2) == 0
    assert lib.ionn_residual_norm_bwd_workspace_bytes(4, 8, -2) == 0
    # a gate for every row costs no more than a workgroup's sums each
    assert lib.ionn_residual_norm_bwd_workspace_bytes(1 << 20, 4096, 1) <= 2 * 512 * 2 * 4096 * 4

    def f(dy=P(0x50000), dn=P(0x60000), a=A, y=Y, na=RMS, ga=V, ba=None, gate=V, gr=2, al=1.0, ny=LAYER, gy=V, ma=None, ra=V,
          my=V, ry=V, da=P(0x70000), dx=P(0x80000), dga=V, dba=None, dg=V, dgy=V, dby=V, dt=0, rows=4, cols=8, ws=V, wb=need):
        return lib.ionn_residual_norm_bwd(dy, dn, a, y, na, ga, ba, gate, gr, al, ny, gy, ma, ra, my, ry, da, dx, dga, dba, dg,
                                          dgy, dby, dt, rows, cols, ws, wb, None)
    assert f(dt=3) == ARG and f(na=5) == ARG and f(ny=5) == ARG
    assert f(rows=-1) == SHAPE and f(cols=16385) == SHAPE and f(al=NAN) == RANGE and f(gr=-1) == RANGE
    assert f(na=NONE) == ARG and f(ny=NONE) == ARG and f(dba=V) == ARG and f(ba=V) == ARG and f(ny=RMS) == ARG
    assert f(gate=None) == ARG  # dgate of no gate
    assert f(dn=None) == ARG and f(y=None) == ARG and f(ry=None) == ARG and f(my=None) == ARG and f(ra=None) == ARG
    assert f(a=None) == ARG
    nothing = dict(da=None, dx=None, dga=None, dg=None, dgy=None, dby=None)
    assert f(**nothing) == ARG
    assert f(dx=P(0x70000)) == ARG and f(dx=P(0x50004)) == ARG and f(da=P(0x10004)) == ARG and f(da=P(0x80004)) == ARG
    assert f(dx=P(0x80001), dt=1) == ALIGN and f(dg=ODD) == ALIGN and f(my=ODD) == ALIGN
    assert f(ws=None) == WS and f(wb=need - 1) == WS and f(ws=P(0x1008)) == WS


@pytest.mark.parametrize("ka,ky", list(itertools.product(("none", "layer", "rms"), repeat=2)))
def test_oracle_gradient_against_differences(ka, ky):
    rng = np.random.default_rng(3)
    rows, cols, h = 5, 4, 2.0 ** -14
    r = rng.standard_normal
    d = dict(a=r((rows, cols)), x=r((rows, cols)), gamma_a=r(cols), beta_a=r(cols), gate=r((3, cols)), gamma_y=r(cols),
             beta_y=r(cols))
    for k, kind in (("a", ka), ("y", ky)):
        d["gamma_" + k] = None if kind == "none" else d["gamma_" + k]
        d["beta_" + k] = d["beta_" + k] if kind == "layer" else None
    dy, dn = r((rows, cols)), r((rows, cols))
    fwd = lambda d: of.residual_norm_fwd(d["a"], d["x"], ka, d["gamma_a"], d["beta_a"], d["gate"], 2, 0.5, ky, d["gamma_y"], d["beta_y"], 1e-5)  # noqa: E731,E501
    w = fwd(d)
    loss = lambda d: (lambda o: (dy * o["y"]).sum() + (0.0 if ky == "none" else (dn * o["n"]).sum()))(fwd(d))  # noqa: E731
    g = of.residual_norm_bwd(dy, dn, d["a"], w["y"], ka, d["gamma_a"], d["beta_a"], d["gate"], 2, 0.5, ky, d["gamma_y"],
                             w["mean_a"], w["rstd_a"], w["mean_y"], w["rstd_y"])
    scale = np.abs(dy).sum() + np.abs(dn).sum()
    for k, name in (("x", "dx"), ("a", "da"), ("gate", "dgate"), ("gamma_a", "dgamma_a"), ("beta_a", "dbeta_a"),
                    ("gamma_y", "dgamma_y"), ("beta_y", "dbeta_y")):
        if d[k] is None:
            continue
        for at in np.ndindex(d[k].shape):
            lo, hi = d[k].copy(), d[k].copy()
            lo[at] -= h
            hi[at] += h
            diff = (loss({**d, k: hi}) - loss({**d, k: lo})) / (2 * h)
            # third derivatives of rows of deviation 0.3 and more: below 1000 times the terms
            assert abs(diff - g[name][at]) <= scale * 1000 * h * h, (k, at)


def test_workspace_serves_a_call_without_a_gate():
    """gate_rows does not count without a gate, whatever the workspace was asked for with."""
    for rows, cols in ((1, 5), (300, 64), (8192, 700), (40000, 24)):
        for gate_rows in (1, 3, 70, 299, 300, 8000, 50000):
            assert (ops.ionn_residual_norm_bwd_workspace_bytes(rows, cols, gate_rows)
                    >= ops.ionn_residual_norm_bwd_workspace_bytes(rows, cols))
