"""GPU: 8-bit states with a first moment of long memory (beta1 above 15/16),
whose steps are smaller than the distance of two codes: bit for bit the
oracle's, and over many steps, with gradients that vanish and come back, the
32-bit state's mean.

Tolerance.  The codes keep m's expectation, so the mean of n independent
elements is off by its scatter over sqrt(n).  An element goes to one of two
codes at most w = m / 8 apart, a variance of at most w^2 / 4 a step, pulled back
by 1 - beta1: w^2 / (8 (1 - beta1)) = m^2 / (512 (1 - beta1)), and while m falls by its
gradients' absence a step of d m adds d w m: to m^2 / 8 for each factor e.  With m =
0.3 +- 0.07 (beta1 = 0.99) the first is 0.44 m; six e-folds later the second 0.87
of what is left: below m each; n = 16384: 1 / 128 of the mean magnitude, five of
which are 4%."""
import numpy as np
import pytest
import torch

from gpu_helpers import dev, host, say
from integer_only_nn_amd import steps
from oracle import floats as of
from test_gpu_adamw import _compare, _run, _tensor, _want

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1, 3, 255, 257, 70001])
@pytest.mark.parametrize("beta1", [0.9375, 0.95, 0.999])
def test_one_step(n, beta1):
    d = _tensor(n, 8, "bf16", spread=3.0)
    d["g"][: n // 3] = 0
    for t in (1, 77):
        _compare(_run([d], t, 8, beta1=beta1), [_want(d, t, beta1=beta1)])


def test_not_finite_means():
    d = _tensor(700, 8, "f32")
    d["g"][10], d["g"][300], d["g"][699] = float("nan"), float("inf"), -float("inf")
    _compare(_run([d], 2, 8, beta1=0.99), [_want(d, 2, beta1=0.99)])


@pytest.mark.parametrize("beta1", [0.95, 0.99])
@pytest.mark.parametrize("rests", [None, False])
def test_mean_follows_its_definition(beta1, rests):
    n = 16384
    new = lambda: [torch.zeros(n, device=dev())]  # noqa: E731
    kw = dict(betas=(beta1, 0.999), weight_decay=0.0)
    words, codes = steps.AdamW.make(new(), bits=32, **kw), steps.AdamW.make(new(), bits=8, Rs=rests, **kw)
    gen = torch.Generator(device=dev()).manual_seed(3)
    folds = round(6 / (1 - beta1))
    say("adamw mean", beta1, rests)
    for t in range(1, 1401 + folds):
        g = torch.randn(n, generator=gen, device=dev()) + 0.3
        g = g if t <= 400 else 0 * g if t <= 400 + folds else 0.1 * g
        words.step([g])
        codes.step([g])
        if t in (50, 400, 400 + folds // 3, 400 + folds, 1400 + folds):
            m = host(words.M[0]).astype(np.float64)
            c = of.state_decode(host(codes.M[0]), host(codes.S[0])[:, 0]).astype(np.float64)
            say(t, c.mean(), m.mean(), np.abs(m).mean())
            assert abs(c.mean() - m.mean()) < 0.04 * np.abs(m).mean()
