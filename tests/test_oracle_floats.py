"""CPU pins of the oracle's floating-point operations (oracle/floats.py):
activations and gradients against central differences, the DFP-8 and E4M3
conversions against exact arithmetic and torch's cast, AdamW against its
formula in float64."""
import math

import numpy as np
import pytest
import torch

from oracle import floats as of


@pytest.mark.parametrize("kind", of.ACTIVATIONS)
def test_activation_gradient_matches_differences(kind):
    z = np.concatenate([np.linspace(-6, 6, 241) + 0.013, [-40.0, 40.0]])
    h = 1e-5
    want = (of.act(z + h, kind) - of.act(z - h, kind)) / (2 * h)
    # the central difference is off by h^2 / 6 |f'''| (< 1e-10) and the
    # values' rounding over 2 h (|f| 2^-53 / h < 1e-9)
    np.testing.assert_allclose(of.act_grad(z, kind), want, atol=2e-9, rtol=0)


def test_activation_values():
    assert of.act([1.0], "gelu")[0] == pytest.approx(0.8413447460685429, rel=1e-14)
    assert of.act([-1.0], "silu")[0] == pytest.approx(-1 / (1 + math.e), rel=1e-14)
    assert of.act([1.0], "gelu_tanh")[0] == pytest.approx(0.8411919906082768, rel=1e-12)


def test_layer_norm_gradient_matches_differences():
    rng = np.random.default_rng(0)
    x, dy = rng.standard_normal((3, 7)) + 2.0, rng.standard_normal((3, 7))
    gamma, beta = rng.standard_normal(7), rng.standard_normal(7)
    loss = lambda x, g, b: float((dy * of.layer_norm_fwd(x, g, b, 1e-5)[0]).sum())  # noqa: E731
    _, mean, rstd = of.layer_norm_fwd(x, gamma, beta, 1e-5)
    dx, dg, db = of.layer_norm_bwd(dy, x, mean, rstd, gamma, None)
    h = 1e-6
    for got, at, put in ((dx, x, 0), (dg, gamma, 1), (db, beta, 2)):
        for i in np.ndindex(at.shape):
            args = [x, gamma, beta]
            hi, lo = at.copy(), at.copy()
            hi[i] += h
            lo[i] -= h
            args[put] = hi
            up = loss(*args)
            args[put] = lo
            # rounding of the losses (|loss| < 30) over 2 h: below 1e-8
            assert got[i] == pytest.approx((up - loss(*args)) / (2 * h), abs=1e-7)


def test_dfp8_hand_cases():
    for x, want, e in (([1.0, -1.0, 0.5], [64, -64, 32], -6), ([1.999, 0.0], [127, 0], -6), ([0.0, 0.0], [0, 0], 0),
                       ([-4.0, 0.09375, 0.03125], [-64, 2, 0], -4), ([2.0 ** -140], [64], -146)):
        I, got = of.dfp8(np.array(x))
        assert got == e and I.tolist() == want, x


def test_e4m3_codes():
    t = of.e4m3_table()
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(t, want)
    rng = np.random.default_rng(1)
    mid = (t[:0x7e] + t[1:0x7f]) / 2  # every tie
    x = np.concatenate([t[:0x7f], -t[:0x7f], mid, -mid, mid * (1 + 1e-6), mid * (1 - 1e-6),
                        rng.standard_normal(5000) * 40]).astype(np.float32)
    x = x[np.abs(x) <= 448]
    got = of.e4m3_encode(x)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(got, want)
    assert of.e4m3_encode(np.array([np.nan, np.inf, -np.inf])).tolist() == [0x7f] * 3


def test_state_exponents_keep_every_block_in_range():
    for top in (1.75, 1.7500001, 1.0, 1.9999999, 2.0 ** -120, 2.0 ** -149, 3e38, 0.0):
        x = np.zeros(300, np.float32)
        x[7], x[270] = top, -top / 2
        c, e = of.state_encode(x, False)
        v = of.state_decode(c, e)
        assert np.all(np.abs(v - x) <= np.abs(x) * 2.0 ** -4 + 2.0 ** -135), top
        assert e.tolist()[0] == (0 if top == 0 else max(-126, math.frexp(np.float32(top))[1] - 9 +
                                                       (math.frexp(np.float32(top))[0] > 0.875)))
    # a positive root never vanishes, a zero stays zero
    c, e = of.state_encode(np.array([1.0, 1e-30, 0.0], np.float32), True)
    assert c[1] == 1 and c[2] == 0


def test_adamw_follows_its_formula():
    rng = np.random.default_rng(2)
    n, t = 5000, 7
    p, g, m = (rng.standard_normal(n).astype(np.float32) for _ in range(3))
    v = np.square(rng.standard_normal(n)).astype(np.float32)
    a = dict(t=t, lr=1e-2, beta1=0.9, beta2=0.99, eps=1e-6, weight_decay=0.1)
    P, M, V = of.adamw_step(p, g, m, v, grad_scale=0.5, **a)
    G = 0.5 * g.astype(np.float64)
    m64 = 0.9 * m + 0.1 * G
    v64 = 0.99 * v + 0.01 * G * G
    u = m64 / (1 - 0.9 ** t) / (np.sqrt(v64 / (1 - 0.99 ** t)) + 1e-6)
    want = p * (1 - 1e-3) - 1e-2 * u
    # at most 4 roundings of each term, and 8 on the way to the update
    np.testing.assert_allclose(M, m64, atol=4 * 2.0 ** -24 * (np.abs(m) + np.abs(g)).max(), rtol=0)
    np.testing.assert_allclose(V, v64, rtol=6 * 2.0 ** -24)
    tol = 2.0 ** -24 * (2 * np.abs(p) + 1e-2 * 8 * (np.abs(m) + np.abs(g)) / np.sqrt(v64))
    assert np.all(np.abs(P - want) <= tol * 2)
