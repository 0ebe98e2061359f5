"""GPU: gelu and its derivative against the definition, relative to the value,
far into the negative tail.

An IN = 0 layer's z is its bias, and a single row's bias gradient is dY act'(Z)
in float32, so both are seen alone.  gelu(z) = max(z, 0) - |z| Phi(-|z|).
Tolerance: the fit of Phi's tail (relative: 2^-14.9 for 16-bit results, 2^-23
otherwise), z^2 half steps of float32 from the exponent's argument and 16 from
the rest of the arithmetic, of the terms' magnitudes; then half a step of the
output's type."""
import numpy as np
import pytest
import torch

from gpu_helpers import dev, host, say, to_dev
from integer_only_nn_amd import ops
from oracle import floats as of

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SMALLEST = {"f32": 2.0 ** -126, "bf16": 2.0 ** -126, "f16": 2.0 ** -24}


def _e(v):
    return torch.tensor([v], dtype=torch.int32, device=dev())


def _points():
    z = np.concatenate([np.linspace(-13, 6, 60001), -np.geomspace(1e-30, 13, 4000), np.geomspace(1e-30, 6, 4000)])
    return z.astype(np.float32)


@pytest.mark.parametrize("name", list(TYPES))
def test_value(name):
    z = _points()
    n = z.size
    say("gelu", name, n)
    Y = torch.empty(1, n, dtype=TYPES[name], device=dev())
    i8 = lambda *s: torch.empty(*s, dtype=torch.int8, device=dev())  # noqa: E731
    ops.dfp8_linear_fwd(i8(1, 0), _e(0), i8(n, 0), _e(0), Y, bias=to_dev(z), act="gelu")
    y, z = host(Y.double())[0], z.astype(np.float64)
    want = of.act(z, "gelu")
    fit = 2.0 ** -23 if name == "f32" else 2.0 ** -14.9
    tail = np.abs(of.act(-np.abs(z), "gelu"))  # |z| Phi(-|z|)
    arith = (fit + (16 + z * z) * 2.0 ** -24) * tail + 2.0 ** -24 * np.abs(want)
    half = torch.finfo(TYPES[name]).eps / 2
    off = np.abs(y - want)
    bad = off - arith - half * (np.abs(want) + arith) - SMALLEST[name]
    i = int(np.argmax(off / (np.abs(want) + SMALLEST[name])))
    say("largest relative error", off[i] / np.abs(want[i]), "at", z[i])
    assert (bad <= 0).all(), f"gelu({z[bad.argmax()]}) = {y[bad.argmax()]}, not {want[bad.argmax()]}"


@pytest.mark.parametrize("name", list(TYPES))
def test_derivative(name):
    z = torch.from_numpy(_points()).to(dev()).to(TYPES[name]).view(1, -1)
    n = z.numel()
    say("gelu derivative", name, n)
    gb, dZ8 = torch.empty(n, device=dev()), torch.empty(1, n, dtype=torch.int8, device=dev())
    W = torch.zeros(n, 1, dtype=torch.int8, device=dev())
    ops.dfp8_linear_bwd(torch.ones_like(z), z, "gelu", None, None, W, _e(0), dZ8, _e(0), gb=gb,
                        workspace=torch.empty(ops.dfp8_linear_bwd_workspace_bytes(1, 1, n), dtype=torch.uint8, device=dev()))
    z = host(z.double())[0]
    want = of.act_grad(z, "gelu")
    density = np.abs(z) * np.exp(-0.5 * z * z) / np.sqrt(2 * np.pi)
    tol = (2.0 ** -23 + (16 + z * z) * 2.0 ** -24) * (np.abs(want - np.sign(z) * density) + density) + 2.0 ** -126
    bad = np.abs(host(gb) - want) - tol
    assert (bad <= 0).all(), f"gelu'({z[bad.argmax()]}) = {host(gb)[bad.argmax()]}, not {want[bad.argmax()]}"
