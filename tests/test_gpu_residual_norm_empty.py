"""GPU: the gradients of the vectors of ionn_residual_norm_bwd for a batch of no
rows: zeros, whatever the vectors hold."""
import itertools

import pytest
import torch

from gpu_helpers import dev, host, say
from integer_only_nn_amd import ops

pytestmark = pytest.mark.gpu

KINDS = list(itertools.product(("none", "layer", "rms"), repeat=2))


@pytest.mark.parametrize("norm_a,norm_y", KINDS)
@pytest.mark.parametrize("gate_rows", [0, 1, 3])
@pytest.mark.parametrize("cols", [1, 30, 4100])
def test_gradients_of_no_rows(norm_a, norm_y, gate_rows, cols):
    """A gate that all rows share is there without rows too, [1][cols]."""
    say("no rows", norm_a, norm_y, gate_rows, cols)
    rows = lambda: torch.empty(0, cols, dtype=torch.bfloat16, device=dev())  # noqa: E731
    vec = lambda v=7.0: torch.full((cols,), v, device=dev())  # noqa: E731
    none = torch.empty(0, device=dev())
    for v in (1.5, float("inf"), float("nan")):
        out = {"dgate": vec()}
        kw = dict(gate=vec(v), gate_rows=gate_rows)
        for k, kind in (("a", norm_a), ("y", norm_y)):
            if kind != "none":
                kw["gamma_" + k], kw["rstd_" + k], out["dgamma_" + k] = vec(v), none, vec()
            if kind == "layer":
                kw["mean_" + k], out["dbeta_" + k] = none, vec()
        if norm_a == "layer":
            kw["beta_a"] = vec(v)
        ops.ionn_residual_norm_bwd(rows(), rows() if norm_y != "none" else None, rows(), rows(), rows(), rows(), norm_a=norm_a,
                                   norm_y=norm_y, **kw, **out)
        for k, t in out.items():
            assert not host(t).any(), (k, v)


def test_gradients_that_are_not_asked_for():
    rows = torch.empty(0, 40, dtype=torch.float32, device=dev())
    gate, dgate = torch.ones(40, device=dev()), torch.full((40,), 7.0, device=dev())
    ops.ionn_residual_norm_bwd(rows, None, rows, None, rows, rows, norm_a="none", norm_y="none", gate=gate, dgate=dgate)
    assert not host(dgate).any()
    ops.ionn_residual_norm_bwd(rows, None, rows, None, rows, rows, norm_a="none", norm_y="none", gate=gate)
