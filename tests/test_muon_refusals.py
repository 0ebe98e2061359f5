"""The Muon step's host-side checks (no GPU needed: none of these calls reaches
one), and the oracle's orthogonalisation against singular values."""
import ctypes

import numpy as np
import pytest
import torch

from integer_only_nn_amd import _lib, ops, steps
from oracle import floats as of
from test_gpu_muon import TILES

lib = _lib.lib()
OK, ARG, SHAPE, RANGE, ALIGN, UNSUP, HIP, WS = range(8)
P = ctypes.c_void_p
NAN, INF = float("nan"), float("inf")


def test_step():
    arr = lambda v: (ctypes.c_void_p * 1)(v)  # noqa: E731
    i64 = lambda v: (ctypes.c_int64 * 1)(v)  # noqa: E731
    need = lib.ionn_muon_workspace_bytes(1, i64(8), i64(8))
    assert need > 0

    def f(L=1, p=arr(0x1000), g=arr(0x3000), dt=0, m=arr(0x2000), r=i64(8), c=i64(8), lr=0.1, mu=0.9, nes=1, eps=1e-7, wd=0.0,
          k=5, sc=None, lrd=None, gs=None, top=None, ws=P(0x10000), wb=need):
        return lib.ionn_muon_step(L, p, g, dt, m, r, c, lr, mu, nes, eps, wd, k, sc, lrd, gs, top, ws, wb, None)
    assert f(L=0) == SHAPE and f(r=i64(0)) == SHAPE and f(c=i64(-1)) == SHAPE and f(r=i64(1 << 15), c=i64(1 << 14)) == SHAPE
    assert f(dt=3) == ARG and f(p=None) == ARG and f(g=None) == ARG and f(m=None) == ARG and f(r=None) == ARG
    assert f(p=arr(0)) == ARG and f(g=arr(0)) == ARG and f(m=arr(0)) == ARG
    assert f(p=arr(0x1002)) == ALIGN and f(m=arr(0x1001)) == ALIGN and f(g=arr(0x1001), dt=1) == ALIGN
    assert f(lrd=P(0x1001)) == ALIGN and f(gs=P(0x1002)) == ALIGN and f(top=P(0x1001)) == ALIGN
    assert f(mu=1.0) == RANGE and f(mu=-0.1) == RANGE and f(mu=NAN) == RANGE and f(eps=-1.0) == RANGE and f(lr=INF) == RANGE
    assert f(wd=NAN) == RANGE and f(k=0) == RANGE and f(k=33) == RANGE and f(sc=(ctypes.c_double * 1)(NAN)) == RANGE
    assert f(ws=None) == WS and f(wb=need - 1) == WS and f(ws=P(0x10080)) == WS
    assert f(m=arr(0x1000)) == ARG and f(m=arr(0x10fc)) == ARG and f(g=arr(0x20fc)) == ARG and f(g=arr(0x1f82), dt=1) == ARG
    assert f(m=arr(0x1100), ws=None) == WS and f(g=arr(0x1f80), dt=1, ws=None) == WS  # next to each other
    two = lambda a, b: (ctypes.c_void_p * 2)(a, b)  # noqa: E731
    twice = dict(L=2, g=two(0x8000, 0x9000), r=(ctypes.c_int64 * 2)(8, 8), c=(ctypes.c_int64 * 2)(8, 8), ws=None)
    assert f(p=two(0x1000, 0x1000), m=two(0x2000, 0x3000), **twice) == ARG
    assert f(p=two(0x1000, 0x10f0), m=two(0x2000, 0x3000), **twice) == ARG
    assert f(p=two(0x1000, 0x4000), m=two(0x2000, 0x2000), **twice) == ARG
    assert f(p=two(0x1000, 0x2000), m=two(0x2000, 0x3000), **twice) == ARG
    assert f(p=two(0x1000, 0x1100), m=two(0x2000, 0x2100), **twice) == WS


def test_gradients_apart_from_what_the_step_writes():
    def f(p, m, g, dt=0):
        two = lambda v: (ctypes.c_void_p * 2)(*v)  # noqa: E731
        s = (ctypes.c_int64 * 2)(8, 8)
        return lib.ionn_muon_step(2, two(p), two(g), dt, two(m), s, s, 0.1, 0.9, 1, 1e-7, 0.0, 5, None, None, None, None, None, 0, None)
    p, m = (0x1000, 0x1100), (0x2000, 0x2100)
    for g in ((0x1000, 0x8000), (0x8000, 0x10fc), (0x8000, 0x2000), (0x21fc, 0x8000), (0x0f04, 0x8000)):
        assert f(p, m, g) == ARG
    assert f(p, m, (0x0f82, 0x8000), 1) == ARG
    for g in ((0x8000, 0x8000), (0x0f00, 0x1200), (0x1f00, 0x2200)):  # a shared gradient; next to each other
        assert f(p, m, g) == WS
    assert f(p, m, (0x0f80, 0x2200), 1) == WS


def test_workspace_of_a_list_is_that_of_its_largest_part():
    one = ops.ionn_muon_workspace_bytes([(4096, 4096)])
    assert one > 4096 * 4096 * 16
    assert ops.ionn_muon_workspace_bytes([(4096, 4096)] * 5 + [(10, 10)]) == one
    assert ops.ionn_muon_workspace_bytes([(4096, 4096), (0, 4)]) == 0


@pytest.mark.parametrize("side", list(TILES))
def test_sizes_take_their_tiles(side):
    for shape in TILES[side]:
        assert ops.ionn_muon_tile([shape]) == side, shape


def test_tiles_of_a_list():
    shapes = [(10, 10)] * 3 + [(4096, 4096)] + [(1000, 1000)] * 9
    assert [ops.ionn_muon_tile(shapes, l) for l in (0, 2, 3, 4, 11, 12)] == [32, 32, 256, 128, 128, 64]
    for bad in (([(0, 4)], 0), ([(4, 4)], 1), ([(4, 4)], -1)):
        with pytest.raises(ValueError):
            ops.ionn_muon_tile(*bad)


def test_the_binding_refuses_before_the_library():
    w = torch.zeros(4, 5)
    with pytest.raises(ValueError):
        steps.Muon([w], [torch.zeros(5, 4)])
    with pytest.raises(ValueError):
        steps.Muon([torch.zeros(4)], [torch.zeros(4)])
    with pytest.raises(ValueError):
        steps.Muon([w], [w], scale=[1.0, 2.0])
    with pytest.raises(ValueError):
        ops.ionn_muon_step([w], [torch.zeros(5, 4)], [w], 0.1, None)
    steps.Muon([], []).step()  # nothing to do


def test_oracle_orthogonalises():
    """The matrix's singular vectors with the polynomial's values of its singular values."""
    rng = np.random.default_rng(0)
    for shape in ((5, 9), (9, 5), (6, 6), (1, 4)):
        x = rng.standard_normal(shape)
        x /= np.linalg.norm(x)
        u, s, v = np.linalg.svd(x, full_matrices=False)
        for _ in range(5):
            s = 3.4445 * s - 4.7750 * s ** 3 + 2.0315 * s ** 5
        np.testing.assert_allclose(of.newton_schulz(x, 5), (u * s) @ v, atol=1e-10)
