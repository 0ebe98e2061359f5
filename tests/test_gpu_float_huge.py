"""GPU: sizes whose grids, one workgroup for each piece of the output, would
have more threads than the runtime takes, and sizes next to them."""
import numpy as np
import pytest
import torch

from gpu_helpers import dev, say
from integer_only_nn_amd import ops

pytestmark = pytest.mark.gpu


def _e(v):
    return torch.tensor([v], dtype=torch.int32, device=dev())


@pytest.mark.parametrize("OUT", [(1 << 27) + 3, 1 << 28])
def test_forward_of_one_row(OUT):
    IN = 16
    say("fwd", 1, IN, OUT)
    g = torch.Generator(device=dev()).manual_seed(1)
    X = torch.randint(-128, 128, (1, IN), dtype=torch.int8, device=dev(), generator=g)
    W = torch.randint(-128, 128, (OUT, IN), dtype=torch.int8, device=dev(), generator=g)
    Y = torch.full((1, OUT), 7.0, dtype=torch.bfloat16, device=dev())
    assert ops.dfp8_linear_fwd_workspace_bytes(1, IN, OUT) == 0
    ops.dfp8_linear_fwd(X, _e(-3), W, _e(-4), Y)
    for a in range(0, OUT, 1 << 25):
        s = (W[a:a + (1 << 25)].int() * X.int()).sum(1, dtype=torch.int32)
        assert torch.equal(Y[0, a:a + (1 << 25)], torch.ldexp(s.float(), _e(-7)).bfloat16()), a


def test_bias_gradient_of_many_columns():
    OUT = 1 << 30
    say("gb", OUT)
    dY = torch.empty(1, OUT, dtype=torch.bfloat16, device=dev()).normal_()
    gb, dZ8 = torch.full((OUT,), 7.0, device=dev()), torch.empty(1, OUT, dtype=torch.int8, device=dev())
    ops.dfp8_linear_bwd(dY, None, "none", None, None, torch.empty(OUT, 0, dtype=torch.int8, device=dev()), None, dZ8, _e(0),
                        gb=gb, workspace=torch.empty(ops.dfp8_linear_bwd_workspace_bytes(1, 0, OUT), dtype=torch.uint8,
                                                     device=dev()))
    for a in range(0, OUT, 1 << 27):
        assert torch.equal(gb[a:a + (1 << 27)], dY[0, a:a + (1 << 27)].float()), a


def test_norm_gradient_of_many_columns():
    cols = (1 << 27) + 1
    say("norm bwd", 1, cols)
    x, dy = (torch.empty(1, cols, device=dev()).normal_() for _ in range(2))
    mean, rstd = torch.zeros(1, device=dev()), torch.ones(1, device=dev())
    dx, dg, db = torch.empty_like(x), torch.full((cols,), 7.0, device=dev()), torch.full((cols,), 7.0, device=dev())
    ws = torch.empty(ops.ionn_layer_norm_bwd_workspace_bytes(1, cols), dtype=torch.uint8, device=dev())
    ops.ionn_layer_norm_bwd(dy, x, mean, rstd, dx, dgamma=dg, dbeta=db, workspace=ws)
    # one row: the column sums are single terms
    assert torch.equal(db, dy[0]) and torch.equal(dg, dy[0] * x[0])
    # dx = dy - mean(dy) - x mean(dy x), both means below 6 / sqrt(cols) = 5e-4
    assert float((dx - dy).abs().max()) < 5e-4 * (1 + 7) and np.isfinite(float(dx.double().sum()))
