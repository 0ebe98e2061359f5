"""The gated layer's host-side checks (no GPU needed: none of these calls
reaches one), and that its GPU tests' sizes take every way of cutting a product."""
import ctypes

import pytest
import torch

from integer_only_nn_amd import _lib, ops
from test_gpu_dfp8_gated import COPIES, WAYS

lib = _lib.lib()
OK, ARG, SHAPE, RANGE, ALIGN, UNSUP, HIP, WS = range(8)
P = ctypes.c_void_p
A, ODD, FAR = P(0x1000), P(0x1001), P(0x900000)  # never dereferenced


@pytest.mark.parametrize("B,IN,H", list(WAYS))
def test_sizes_take_their_ways(B, IN, H):
    assert ops.dfp8_linear_path("fwd", B, IN, 2 * H) == WAYS[B, IN, H]


def test_every_way_is_taken():
    assert set(WAYS.values()) == {"rows", "tiles 256", "tiles 128", "tiles", "narrow"}
    assert ops.dfp8_gated_fwd_workspace_bytes(300, 9001, 300) > 0  # ranges of the reduction


@pytest.mark.parametrize("B,IN,H", list(COPIES))
def test_sizes_whose_rows_are_copied(B, IN, H):
    whole = lambda n: (n + 15) // 16 * 16  # noqa: E731
    size = {"Z": B * whole(2 * H), "X": B * whole(IN), "W": 2 * H * whole(IN)}
    fwd, bwd = COPIES[B, IN, H]
    assert ops.dfp8_gated_fwd_workspace_bytes(B, IN, H) == sum(size[t] for t in fwd)
    errors = ops.dfp8_gated_bwd_workspace_bytes(B, 0, H)
    assert ops.dfp8_gated_bwd_workspace_bytes(B, IN, H) - errors == sum(size[t] for t in bwd)


def test_fwd():
    def f(X=A, eX=A, W=A, eW=A, bias=None, act=4, Z=None, Y=FAR, dt=0, B=4, IN=8, H=8, m=None, ws=A, wb=1 << 40):
        return lib.dfp8_gated_fwd(X, eX, W, eW, bias, act, Z, Y, dt, B, IN, H, m, ws, wb, None)
    assert f(dt=7) == ARG and f(act=5) == ARG and f(act=-1) == ARG
    assert f(B=-1) == SHAPE and f(IN=131072) == SHAPE and f(H=(1 << 29) + 1) == SHAPE and f(IN=-5) == SHAPE and f(H=-1) == SHAPE
    assert f(X=None) == ARG and f(W=None) == ARG and f(Y=None) == ARG and f(eX=None) == ARG and f(eW=None) == ARG
    assert f(Z=FAR) == ARG and f(Z=P(0x900000 + 4 * 8 * 4 - 4)) == ARG and f(Z=P(0x900000 - 2 * 4 * 8 * 4 + 4)) == ARG
    assert f(Y=P(0x1002)) == ALIGN and f(bias=ODD) == ALIGN and f(eX=ODD) == ALIGN and f(Z=ODD, dt=1) == ALIGN and f(m=ODD) == ALIGN
    assert f(B=0) == OK and f(H=0, Y=None) == OK  # nothing to do
    assert lib.dfp8_gated_fwd_workspace_bytes(-1, 4, 4) == 0
    need = lib.dfp8_gated_fwd_workspace_bytes(300, 9001, 300)
    assert f(B=300, IN=9001, H=300, ws=None) == WS and f(B=300, IN=9001, H=300, wb=need - 1) == WS
    assert f(B=300, IN=9001, H=300, ws=P(0x1008)) == WS
    assert f(B=1 << 26, IN=64, H=1 << 26) == SHAPE  # more tiles than a grid takes


def test_bwd():
    need = lib.dfp8_gated_bwd_workspace_bytes(4, 8, 8)
    assert need > 0 and lib.dfp8_gated_bwd_workspace_bytes(4, 8, -8) == 0

    def f(dY=A, Z=A, act=2, dt=0, X=A, eX=A, W=A, eW=A, q=A, e=A, dX=A, G=A, gb=A, B=4, IN=8, H=8, st=None, ws=A, wb=need):
        return lib.dfp8_gated_bwd(dY, Z, act, dt, X, eX, W, eW, q, e, dX, G, gb, B, IN, H, st, ws, wb, None)
    assert f(dt=3) == ARG and f(act=9) == ARG
    assert f(B=-1) == SHAPE and f(H=65536) == SHAPE and f(B=131072) == SHAPE and f(IN=(1 << 30) + 1) == SHAPE
    assert f(dY=None) == ARG and f(Z=None) == ARG and f(Z=None, act=0) == ARG and f(q=None) == ARG and f(e=None) == ARG
    assert f(W=None) == ARG and f(eW=None) == ARG and f(X=None) == ARG and f(eX=None) == ARG
    assert f(dY=P(0x1002)) == ALIGN and f(gb=ODD) == ALIGN and f(e=ODD) == ALIGN and f(st=ODD) == ALIGN
    assert f(ws=None) == WS and f(wb=need - 1) == WS and f(ws=P(0x1008)) == WS


def test_the_binding_refuses_before_the_library():
    t = lambda *s, dt=torch.int8: torch.zeros(s, dtype=dt)  # noqa: E731
    one = t(1, dt=torch.int32)
    with pytest.raises(ValueError):  # an odd number of weight rows
        ops.dfp8_gated_fwd(t(3, 4), one, t(5, 4), one, t(3, 2, dt=torch.float32))
    with pytest.raises(ValueError):  # Z of one half
        ops.dfp8_gated_fwd(t(3, 4), one, t(4, 4), one, t(3, 2, dt=torch.float32), Z=t(3, 2, dt=torch.float32))
    with pytest.raises((ValueError, TypeError)):  # not on a device
        ops.dfp8_gated_fwd(t(3, 4), one, t(4, 4), one, t(3, 2, dt=torch.float32))
