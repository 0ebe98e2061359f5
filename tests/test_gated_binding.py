"""The bindings of the DFP-8 layers' backward passes without X and W: what they
refuse, they refuse as they refuse other tensors (no GPU needed)."""
import pytest
import torch

from integer_only_nn_amd import ops


@pytest.mark.parametrize("call,half", [(ops.dfp8_gated_bwd, 2), (ops.dfp8_linear_bwd, 1)])
def test_neither_x_nor_w(call, half):
    t = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt)  # noqa: E731
    q, e = t(3, 4 * half, dt=torch.int8), t(1, dt=torch.int32)
    for kw in (dict(gb=t(4 * half)), dict(dX=t(3, 5)), dict(G=t(4 * half, 5))):
        with pytest.raises((ValueError, TypeError)):  # not on a device, or of no layer
            call(t(3, 4), t(3, 4 * half), "none", None, None, None, None, q, e, **kw)
