"""GPU: the Muon step where |u| is far below eps.

X = u / (|u| + eps) is then small and stays in the polynomial's linear part, and
its elements, pairs of float16 terms scaled by 2^12, are held to half a step of
float16's subnormals, 2^-25 / 2^12 = 2^-37 each, wherever that is more than their
relative error: in the root of the sum of squares sqrt(m n) 2^-37 of the first
form, and after each product again; what comes later has grown by a = 3.4445 less
each time, so all of it is below 1.41 times the first.  It grows as X itself does.
Beside it X is right to 2e-6 of its size, as elsewhere."""
import numpy as np
import pytest
import torch

from gpu_helpers import dev, host, say
from integer_only_nn_amd import ops
from oracle import floats as of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,cols", [(64, 64), (300, 70), (512, 700), (2048, 2048), (2304, 2400)])
def test_updates_far_below_eps(rows, cols):
    g = np.random.default_rng(rows).standard_normal((rows, cols))
    g /= np.linalg.norm(g)
    ws = torch.empty(ops.ionn_muon_workspace_bytes([(rows, cols)]), dtype=torch.uint8, device=dev())
    for size in (1e-2, 1e-4, 1e-6, 1e-8, 1e-12):
        G = (size * g).astype(np.float32)
        P, M = (torch.zeros(rows, cols, device=dev()) for _ in range(2))
        ops.ionn_muon_step([P], [torch.from_numpy(G).to(dev())], [M], 1.0, ws, momentum=0.0, nesterov=False, eps=1.0, scale=[1.0])
        first = G.astype(np.float64) / (np.linalg.norm(G.astype(np.float64)) + 1.0)
        x = of.newton_schulz(first, 5)
        off, grown = np.linalg.norm(host(P) + x), np.linalg.norm(x) / np.linalg.norm(first)
        tol = 2e-6 * np.linalg.norm(x) + 1.41 * np.sqrt(rows * cols) * 2.0 ** -37 * grown
        say(rows, cols, size, "off", off, "tolerance", tol)
        assert off <= tol
