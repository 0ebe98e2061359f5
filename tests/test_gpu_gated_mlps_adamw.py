"""GPU: steps.GatedMlps with AdamW for the matrices: every weight after two updates
by the optimiser's definition, from the blocks' own gradients, bit for bit."""
import numpy as np
import pytest
import torch

from gpu_helpers import dev, host
from oracle import floats as of
from test_gpu_gated_mlps import _make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("state_bits", [32, 8])
def test_every_weight_by_its_own_gradient(state_bits):
    m, x, dn, dy = _make(50, 64, 96, matrices="adamw", state_bits=state_bits, lr=0.01, weight_decay=0.1, dtype=torch.bfloat16)
    x, dn, dy = (t.to(dev()).bfloat16() for t in (x, dn, dy))
    names = [("W1", "gW1", 0.01, 0.1), ("W2", "gW2", 0.01, 0.1)] + [(k, "g" + k, 1e-3, 0.0) for k in ("b1", "b2", "gamma", "gate")]
    place = [(b, t, n) for b, t in zip(m.blocks, m.bufs) for n in names]
    states = {}
    for step in (1, 2):
        old = [host(b[n[0]]).copy() for b, _, n in place]
        m.forward(x)
        m.backward(x, dn, dy)
        grads = [host(t[n[1]].float()).copy() for _, t, n in place]
        m.update()
        for i, ((b, _, (k, _, lr, decay)), p, g) in enumerate(zip(place, old, grads)):
            p, g = p.reshape(-1), g.reshape(-1)
            if i not in states:
                states[i] = [np.zeros(p.size, np.float32 if state_bits == 32 else np.uint8)] * 2
                if state_bits == 8:
                    states[i] += [np.zeros((-(-p.size // of.ADAMW_BLOCK), 2), np.int8), np.zeros(p.size, np.int8)]
            mean, square, *coded = states[i]
            kw = dict(zip(("exps", "rest"), coded))
            new, *states[i] = of.adamw_step(p, g, mean, square, step, lr, 0.9, 0.999, 1e-8, decay, **kw)
            np.testing.assert_array_equal(host(b[k]).reshape(-1), new, err_msg=f"{k}, step {step}")
        for b, t in zip(m.blocks, m.bufs):
            for k in ("W1", "W2"):
                np.testing.assert_array_equal(host(t[k + "_8"]), of.dfp8(host(b[k]))[0])
