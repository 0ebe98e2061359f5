"""CPU: the oracle's 8-bit optimiser states over many steps against its
32-bit ones, with gradients that grow and shrink: the rule itself follows
AdamW's second moment.  Tolerances: see test_gpu_adamw_long.py."""
import numpy as np
import pytest

from oracle import floats as of


def test_draws_are_uniform_and_unrelated():
    n, steps = 1 << 14, 64
    u = np.stack([of.draws(n, t).astype(np.float64) for t in range(1, steps + 1)])
    assert u.min() >= 0 and u.max() < 1
    # n * steps = 2^20 numbers: each of 256 cells has 4096 +- 64; six of those
    cells = np.histogram(u, 256, (0, 1))[0]
    assert np.abs(cells - u.size / 256).max() < 6 * 64
    c = u - 0.5
    for a, b in ((c[:, 1:], c[:, :-1]), (c[:, 4:], c[:, :-4]), (c[:, 256:], c[:, :-256]), (c[1:], c[:-1]), (c[1:, 1:], c[:-1, :-1])):
        r = 12 * (a * b).mean()  # correlation, +- 2^-10
        assert abs(r) < 6 * 2.0 ** -10
    # a weight's numbers over the steps: their means scatter by 1 / sqrt(12 steps)
    assert abs(c.mean(0).std() * np.sqrt(12 * steps) - 1) < 0.05


def test_root_rounding_keeps_the_expectation_of_the_square():
    r = np.concatenate([np.full(1, 448.0), np.full(1 << 16, 3.3), np.full(1 << 16, 0.0301)]).astype(np.float32)
    c, e = of.root_encode(r, of.draws(r.size, 7))
    v = of.state_decode(c, e).astype(np.float64) ** 2
    for lo in (1, 1 + (1 << 16)):
        x = float(r[lo]) ** 2
        part = v[lo:lo + (1 << 16)]
        assert len(np.unique(part)) == 2
        # two values at most 0.27 of the value apart: half of that over 256 (2^16 of them), six times
        assert abs(part.mean() / x - 1) < 6 * 0.135 / 256


def test_carried_root_is_exact_to_its_step():
    rng = np.random.default_rng(1)
    r = np.abs(rng.standard_normal(4096) * np.exp(2 * rng.standard_normal(4096))).astype(np.float32)
    r[:3] = 0.0, np.inf, np.nan
    c, rest, e = of.root_encode_carried(r, of.draws(r.size, 3))
    back = of.root_decode_carried(c, rest, e)
    near, _ = of.state_encode(r, True)
    np.testing.assert_array_equal(c, near)  # the nearest codes
    assert back[0] == 0 and np.isnan(back[1:3]).all() and rest[1] == rest[2] == 0
    step = np.maximum(np.exp2(np.floor(np.log2(np.maximum(of._TABLE[c[3:]], 2.0 ** -9))) - 3), 2.0 ** -9)
    step = np.ldexp(step, e.astype(int).repeat(256)[3:4096])
    ok = r[3:] >= step / 2  # (below: held at the smallest code's lower end)
    assert (np.abs(back[3:] - r[3:])[ok] <= step[ok] / 254 * 1.001).all()


@pytest.mark.parametrize("beta2", [0.95, 0.999])
def test_second_moment_follows_its_definition(beta2):
    n, rng = 4096, np.random.default_rng(0)
    z = np.zeros(n, np.float32)
    c = np.zeros(n, np.uint8)
    a, q, k = [z, z, z], [z, c, c, np.zeros((n // 256, 2), np.int8)], [z, c, c, np.zeros((n // 256, 2), np.int8), np.zeros(n, np.int8)]
    for t in range(1, 1201):
        g = (rng.standard_normal(n) * (1.0 if t < 500 else 0.1 if t < 1000 else 3.0)).astype(np.float32)
        hyper = (t, 1e-3, 0.9, beta2, 1e-8, 0.0)
        a = list(of.adamw_step(a[0], g, a[1], a[2], *hyper))
        q = list(of.adamw_step(q[0], g, q[1], q[2], *hyper, exps=q[3]))
        k = list(of.adamw_step(k[0], g, k[1], k[2], *hyper, exps=k[3], rest=k[4]))
        if t in (10, 200, 499, 600, 999, 1200):
            v = a[2].astype(np.float64)
            vq = of.state_decode(q[2], q[3][:, 1]).astype(np.float64) ** 2
            vk = of.root_decode_carried(k[2], k[4], k[3][:, 1]).astype(np.float64) ** 2
            assert abs(vq.mean() / v.mean() - 1) < 0.09, t
            ratio = np.sqrt(vk / v)
            assert abs(np.median(ratio) - 1) < 0.004 and np.sqrt(np.mean((ratio - 1) ** 2)) < 0.034, t
