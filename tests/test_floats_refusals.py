"""The floating-point operations' host-side checks: bad calls are refused with
the documented status before anything is enqueued (no GPU needed: none of
these calls reaches one), and the binding's own checks."""
import ctypes

import pytest
import torch

from integer_only_nn_amd import _lib, ops

lib = _lib.lib()
OK, ARG, SHAPE, RANGE, ALIGN, UNSUP, HIP, WS = range(8)
P = ctypes.c_void_p
A, ODD = P(0x1000), P(0x1001)  # never dereferenced
NAN, INF = float("nan"), float("inf")


def test_from_float():
    f = lambda x=A, dt=0, n=8, m=None, out=A, e=A, st=None, ws=A, wb=1 << 20: lib.dfp8_from_float(  # noqa: E731
        x, dt, n, m, out, e, st, ws, wb, None)
    assert f(dt=3) == ARG and f(dt=-1) == ARG
    assert f(n=0) == SHAPE and f(n=-1) == SHAPE and f(n=(1 << 40) + 1) == SHAPE
    assert f(x=None) == ARG and f(out=None) == ARG and f(e=None) == ARG
    assert f(x=ODD, dt=1) == ALIGN and f(x=P(0x1002), dt=0) == ALIGN and f(e=ODD) == ALIGN and f(m=ODD) == ALIGN
    assert f(ws=None) == WS and f(wb=16) == WS and f(ws=ODD) == WS
    assert lib.dfp8_from_float_workspace_bytes() > 16


def test_linear_fwd():
    def f(X=A, eX=A, W=A, eW=A, bias=None, act=0, R=None, Z=None, Y=A, dt=0, B=4, IN=8, OUT=8, m=None, ws=A, wb=1 << 40):
        return lib.dfp8_linear_fwd(X, eX, W, eW, bias, act, R, Z, Y, dt, B, IN, OUT, m, ws, wb, None)
    assert f(dt=7) == ARG and f(act=5) == ARG and f(act=-1) == ARG
    assert f(B=-1) == SHAPE and f(IN=131072) == SHAPE and f(OUT=(1 << 30) + 1) == SHAPE and f(IN=-5) == SHAPE
    assert f(X=None) == ARG and f(W=None) == ARG and f(Y=None) == ARG and f(eX=None) == ARG and f(eW=None) == ARG
    assert f(Z=P(0x2000), Y=P(0x2000)) == ARG and f(Z=P(0x3000), R=P(0x3000)) == ARG
    assert f(Y=P(0x1002)) == ALIGN and f(bias=ODD) == ALIGN and f(eX=ODD) == ALIGN and f(R=ODD, dt=1) == ALIGN
    assert f(B=0) == OK and f(OUT=0, Y=None) == OK  # nothing to do
    assert lib.dfp8_linear_fwd_workspace_bytes(-1, 4, 4) == 0
    need = lib.dfp8_linear_fwd_workspace_bytes(64, 8192, 64)
    if need:
        assert f(B=64, IN=8192, OUT=64, ws=None) == WS and f(B=64, IN=8192, OUT=64, wb=need - 1) == WS


def test_linear_bwd():
    need = lib.dfp8_linear_bwd_workspace_bytes(4, 8, 8)
    assert need > 0 and lib.dfp8_linear_bwd_workspace_bytes(4, 8, -8) == 0

    def f(dY=A, Z=A, act=2, dt=0, X=A, eX=A, W=A, eW=A, q=A, e=A, dX=A, G=A, gb=A, B=4, IN=8, OUT=8, st=None, ws=A, wb=need):
        return lib.dfp8_linear_bwd(dY, Z, act, dt, X, eX, W, eW, q, e, dX, G, gb, B, IN, OUT, st, ws, wb, None)
    assert f(dt=3) == ARG and f(act=9) == ARG
    assert f(B=-1) == SHAPE and f(OUT=131072) == SHAPE and f(B=131072) == SHAPE and f(IN=(1 << 30) + 1) == SHAPE
    assert f(dY=None) == ARG and f(Z=None) == ARG and f(q=None) == ARG and f(e=None) == ARG
    assert f(W=None) == ARG and f(eW=None) == ARG and f(X=None) == ARG and f(eX=None) == ARG
    assert f(dY=P(0x1002)) == ALIGN and f(gb=ODD) == ALIGN and f(e=ODD) == ALIGN and f(st=ODD) == ALIGN
    assert f(ws=None) == WS and f(wb=need - 1) == WS and f(ws=P(0x1008)) == WS


def test_layer_norm():
    def fwd(x=A, g=A, b=A, eps=1e-5, y=P(0x9000), mu=A, rs=A, dt=0, rows=4, cols=8, m=None):
        return lib.ionn_layer_norm_fwd(x, g, b, eps, y, mu, rs, dt, rows, cols, m, None)
    assert fwd(dt=4) == ARG and fwd(rows=-1) == SHAPE and fwd(cols=1 << 31) == SHAPE
    assert fwd(eps=-1.0) == RANGE and fwd(eps=NAN) == RANGE and fwd(eps=INF) == RANGE
    assert fwd(x=None) == ARG and fwd(y=None) == ARG
    assert fwd(x=P(0x1002)) == ALIGN and fwd(g=ODD) == ALIGN and fwd(mu=ODD) == ALIGN and fwd(y=ODD, dt=1) == ALIGN
    assert fwd(y=P(0x1010)) == ARG  # overlaps x in part
    assert fwd(rows=0, x=None) == OK and fwd(cols=0, y=None) == OK
    need = lib.ionn_layer_norm_bwd_workspace_bytes(4, 8)
    assert need == 4 * 2 * 8 * 4 and lib.ionn_layer_norm_bwd_workspace_bytes(-1, 8) == 0

    def bwd(dy=A, x=P(0x2000), mu=A, rs=A, g=None, dr=None, dx=P(0x9000), dg=A, db=A, dt=0, rows=4, cols=8, ws=A, wb=need):
        return lib.ionn_layer_norm_bwd(dy, x, mu, rs, g, dr, dx, dg, db, dt, rows, cols, ws, wb, None)
    assert bwd(dt=-2) == ARG and bwd(cols=-1) == SHAPE
    assert bwd(dy=None) == ARG and bwd(x=None) == ARG and bwd(mu=None) == ARG and bwd(rs=None) == ARG and bwd(dx=None) == ARG
    assert bwd(dx=P(0x2000)) == ARG and bwd(dx=P(0x1010)) == ARG and bwd(dr=P(0x9010)) == ARG
    assert bwd(dy=P(0x1001)) == ALIGN and bwd(dg=ODD) == ALIGN
    assert bwd(ws=None) == WS and bwd(wb=need - 1) == WS and bwd(ws=P(0x1004)) == WS
    assert bwd(cols=0) == OK


def test_adamw():
    arr = lambda *ps: (ctypes.c_void_p * len(ps))(*ps)  # noqa: E731
    num = lambda *ns: (ctypes.c_int64 * len(ns))(*ns)  # noqa: E731
    T = arr(0x1000, 0x2000)

    def f(L=2, p=T, g=T, gd=0, m=T, v=T, s=None, bits=32, n=num(8, 300), t=1, lr=1e-3, b1=0.9, b2=0.99, eps=1e-8, wd=0.0,
          step=None, lrd=None, gs=None, mx=None):
        return lib.ionn_adamw_step(L, p, g, gd, m, v, s, bits, n, t, lr, b1, b2, eps, wd, step, lrd, gs, mx, None)
    assert f(L=0) == SHAPE and f(n=num(8, 0)) == SHAPE and f(n=num(8, (1 << 40) + 1)) == SHAPE
    assert f(gd=3) == ARG and f(bits=16) == ARG and f(p=None) == ARG and f(n=None) == ARG and f(bits=8) == ARG
    assert f(g=arr(0x1000, None)) == ARG and f(bits=8, s=arr(0x1000, None)) == ARG
    assert f(p=arr(0x1000, 0x2002)) == ALIGN and f(g=arr(0x1001, 0x2000), gd=1) == ALIGN and f(m=arr(0x1002, 0x2000)) == ALIGN
    assert f(step=ODD) == ALIGN and f(mx=ODD) == ALIGN and f(gs=ODD) == ALIGN
    assert f(b1=1.0) == RANGE and f(b1=-0.1) == RANGE and f(b2=1.0) == RANGE and f(b2=NAN) == RANGE
    assert f(eps=-1e-8) == RANGE and f(lr=NAN) == RANGE and f(wd=INF) == RANGE and f(t=0) == RANGE
    assert b"t = 0" in lib.ionn_last_error()


def test_binding_refuses_host_tensors_and_shapes():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="device tensor"):
        ops.ionn_layer_norm_fwd(x, torch.empty_like(x))
    for shape in ((4, 7), (8, 4)):
        with pytest.raises(ValueError, match="shape mismatch: y has"):
            ops._m(torch.empty(shape), torch.float32, x.shape, "y")
    with pytest.raises(ValueError, match="shape mismatch: gamma has 7, needs 8"):
        ops._v(torch.empty(7), torch.float32, 8, "gamma")
    with pytest.raises(ValueError, match="device tensor"):
        ops._v(torch.empty(8), torch.float32, 8, "gamma")
    for get in (lambda t: ops._m(t, torch.float32, (8,), "y"), lambda t: ops._v(t, torch.float32, 8, "y"),
                lambda t: ops._s(t, torch.float32, "y")):
        assert get(None) is None
        with pytest.raises(TypeError):
            get([1.0] * 8)
    with pytest.raises(TypeError):
        ops._dtype(torch.zeros(3, dtype=torch.float64), "x")
    with pytest.raises(ValueError, match="shape mismatch"):
        ops.ionn_adamw_step([x], [x], [x], [x[:2]], 1, 1e-3)
    with pytest.raises(TypeError, match="one byte"):
        ops._state_ptrs([x], 8, "M")
