"""GPU: silu's derivative at gates far below 0, where it is small but not 0
(float32 holds exp(z) down to z = -87), in the gated layer's and the Linear
layer's backward pass.

Tolerance.  For z in [-85, -28] the value is z p and the derivative p (1 + z (1 -
p)), p = 1 / (1 + e), e = 2^x, x = -z log2(e).  With u = 2^-24: log2(e) is held to
0.7 u of itself and the product rounds once, so x is off by 1.7 u |z| 1.443 and e
by ln 2 of that, 1.7 u |z| of itself; the exponential and the reciprocal are off by
2 u each, 1 + e, the three products that follow, 1 - p and the last sum by u each,
and 1 + z (1 - p), whose terms are |z| and 1, makes |z| / (|z| - 1) < 1.04 of it.
The products with dY and u round once each.  1.8 |z| + 24 half steps cover it."""
import numpy as np
import pytest
import torch

from gpu_helpers import dev, host, say
from integer_only_nn_amd import ops
from oracle import floats as of
from test_gpu_dfp8_linear import TYPES, _e, _np, _round, _typed, _ws

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DEEPEST = (28.5, 30.5, 31.0, 40.0, 60.0, 84.0)


def _tail(z):
    return (1.8 * np.abs(z) + 24) * U


def _check(dz, rel, q, e, gb):
    """The mantissas and the column sums of an error that is known to rel of itself."""
    top = np.abs(dz).max()
    assert 64 * 2.0 ** e <= top * (1 + rel.max()) and top * (1 - rel.max()) < 128 * 2.0 ** e
    t = np.ldexp(dz, -e)
    assert (np.abs(q - t) <= 0.5 + np.abs(t) * rel).all(), f"mantissas off by {np.abs(q - t).max()}"
    tol = (np.abs(dz) * rel).sum(0) + (len(dz) + 8) * U * np.abs(dz).sum(0) + 2.0 ** -149 * len(dz)
    assert (np.abs(gb - dz.sum(0)) <= tol).all(), f"column sums off by {(np.abs(gb - dz.sum(0)) / np.abs(dz).sum(0)).max()} of themselves"


@pytest.mark.parametrize("deepest", DEEPEST)
@pytest.mark.parametrize("name", list(TYPES))
def test_gated_layer(deepest, name):
    rng = np.random.default_rng(int(deepest))
    for B, H in ((1, 9), (40, 70), (300, 260)):
        g = _round(-deepest - 0.9 * rng.random((B, H)), name)
        up = _round(1 + rng.random((B, H)), name)
        dY = _round(rng.standard_normal((B, H)), name)
        Z = np.concatenate([g, up], 1)
        q, e, st = torch.empty(B, 2 * H, dtype=torch.int8, device=dev()), _e(99), _e(99)
        gb = torch.full((2 * H,), 7.0, device=dev())
        say("gated bwd, silu", B, H, -deepest, name)
        ops.dfp8_gated_bwd(_typed(dY, name), _typed(Z, name), "silu", torch.empty(B, 0, dtype=torch.int8, device=dev()), None,
                           None, None, q, e, gb=gb, status_out=st, workspace=_ws(ops.dfp8_gated_bwd_workspace_bytes(B, 0, H)))
        assert int(host(st)[0]) == 0
        rel = np.concatenate([_tail(g), _tail(g)], 1)
        _check(of.gated_error(dY, Z, "silu"), rel, host(q), int(host(e)[0]), _np(gb))


@pytest.mark.parametrize("deepest", DEEPEST)
@pytest.mark.parametrize("name", list(TYPES))
def test_linear_layer(deepest, name):
    rng = np.random.default_rng(int(deepest))
    for B, OUT in ((1, 9), (40, 70), (300, 520), (2100, 260)):
        Z = _round(-deepest - 0.9 * rng.random((B, OUT)), name)
        dY = _round(rng.standard_normal((B, OUT)), name)
        q, e, st = torch.empty(B, OUT, dtype=torch.int8, device=dev()), _e(99), _e(99)
        gb = torch.full((OUT,), 7.0, device=dev())
        say("linear bwd, silu", B, OUT, -deepest, name)
        ops.dfp8_linear_bwd(_typed(dY, name), _typed(Z, name), "silu", torch.empty(B, 0, dtype=torch.int8, device=dev()), None,
                            None, None, q, e, gb=gb, status_out=st, workspace=_ws(ops.dfp8_linear_bwd_workspace_bytes(B, 0, OUT)))
        assert int(host(st)[0]) == 0
        _check(dY * of.act_grad(Z, "silu"), _tail(Z), host(q), int(host(e)[0]), _np(gb))


def test_infinite_gates():
    """The limits: value and derivative 0 at -inf, derivative 1 at +inf."""
    Z = np.tile([[-np.inf, np.inf, -100.0, -1e30, 1e30, 2.0, 3.0, 0.5, 1.0, 1.0]], (3, 1))
    dY = np.ones((3, 5))
    q, e, gb = torch.empty(3, 10, dtype=torch.int8, device=dev()), _e(99), torch.empty(10, device=dev())
    x = torch.empty(3, 0, dtype=torch.int8, device=dev())
    ops.dfp8_gated_bwd(_typed(dY, "f32"), _typed(Z, "f32"), "silu", x, None, None, None, q, e, gb=gb,
                       workspace=_ws(ops.dfp8_gated_bwd_workspace_bytes(3, 0, 5)))
    assert _np(gb).tolist() == [0.0, 9.0, 0.0, 0.0, 3.0] + [0.0, np.inf, 0.0, 0.0, float(np.float32(3 * float(np.float32(1e30))))]
