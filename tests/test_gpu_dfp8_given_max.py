"""GPU: DFP-8 conversion with the maximum that a producer left, which is taken
before the producer rounds its values to their type.  The result has to be
the conversion that takes the maximum itself (exact)."""
import numpy as np
import pytest
import torch

from gpu_helpers import dev, host, say, to_dev
from integer_only_nn_amd import ops

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _convert(x, absmax=None):
    out, e, st = torch.full(x.shape, 9, dtype=torch.int8, device=dev()), *(torch.full((1,), 99, dtype=torch.int32, device=dev()) for _ in range(2))
    ws = None if absmax is not None else torch.empty(ops.dfp8_from_float_workspace_bytes(), dtype=torch.uint8, device=dev())
    ops.dfp8_from_float(x, out, e, absmax=absmax, workspace=ws, status_out=st)
    return host(out), int(host(e)[0]), int(host(st)[0])


def _bits(v):
    return to_dev(np.array([v], np.float32).view(np.int32))


@pytest.mark.parametrize("name", list(TYPES))
def test_maximum_that_rounds(name):
    t = TYPES[name]
    # values just below a power of two round up to it in 16 bits, others down or not at all
    for top in (1.99999, 0.999999, 511.95, 1.5, 1.501, 3.7251, 2.0 ** -20 * 1.99999):
        x = (torch.linspace(-1, 1, 1001, dtype=torch.float64) * top).float().to(dev())
        say("given max", name, top)
        got, want = _convert(x.to(t), _bits(top)), _convert(x.to(t))
        assert got[1:] == want[1:]
        np.testing.assert_array_equal(got[0], want[0])


def test_stored_infinity_is_reported():
    x = torch.tensor([1.0, 70000.0, -3.0], device=dev())
    assert _convert(x.half(), _bits(70000.0))[2] == 2  # finite before it became float16
    assert _convert(x.half(), _bits(65519.0))[2] == 0  # the largest that does not overflow
    assert _convert(x.bfloat16(), _bits(70000.0))[2] == 0
    assert _convert(x.bfloat16(), _bits(3.4028235e38))[2] == 2
    for bad in (np.nan, np.inf):
        for t in TYPES.values():
            assert _convert(x.to(t), _bits(bad))[2] == 2


@pytest.mark.parametrize("name", ["bf16", "f16"])
def test_after_a_linear_layer(name):
    """The layer's output and the maximum it left."""
    B, IN, OUT = 40, 64, 70
    rng = np.random.default_rng(0)
    X, W = (to_dev(rng.integers(-128, 128, s).astype(np.int8)) for s in ((B, IN), (OUT, IN)))
    for bias, eW in ((1.99999, -40), (70000.0, -20)):
        b = torch.zeros(OUT, device=dev())
        b[3] = bias
        Y, m = torch.empty(B, OUT, dtype=TYPES[name], device=dev()), torch.zeros(1, dtype=torch.int32, device=dev())
        ops.dfp8_linear_fwd(X, torch.tensor([-6], dtype=torch.int32, device=dev()), W,
                            torch.tensor([eW], dtype=torch.int32, device=dev()), Y, bias=b, absmax_Y=m)
        got, want = _convert(Y, m), _convert(Y)
        assert got[1:] == want[1:] and want[2] == (2 if name == "f16" and bias > 65520 else 0)
        if want[2] == 0:
            np.testing.assert_array_equal(got[0], want[0])
