"""GPU: 8-bit optimiser states over many steps.

The codes and remainders of one step are bit for bit the oracle's.  Over
thousands of steps, with gradients that grow and shrink, the second moment is
compared with the 32-bit state's.

Tolerances.  Between two of its roundings a root r changes by d r, and goes to
one of two values w r apart with its expectation (or that of v = r^2) kept, so
the relative variance grows by |d| w a step and is pulled back by 1 - beta2.
Codes: w <= 1/8 of r, 0.27 of v.  Unit gradients, E|g^2 - 1| = 0.97: a variance
of v of 0.97 * 0.27 / 2 = 0.13; while v falls to a hundredth, (1 - beta2) steps =
4.6, nothing pulls back and it grows to 4.6 * 0.27 = 1.24.  The mean of n
elements' v is off by sqrt(1.24 / n), five of which are 4.4% for 16384 (8.7% for
4096).  Remainders: w <= 1 / (8 * 254): at most 0.5 * 4.6 * w = 0.0011 of r, 3.4% in
the root mean square; the median of 4096 by 1.25 * 3.4% / 64 = 0.07%, four of
which and the 0.11% between r and the root of r^2's mean are 0.4%."""
import numpy as np
import pytest
import torch

from gpu_helpers import dev, host, say, to_dev
from integer_only_nn_amd import ops, steps
from oracle import floats as of
from test_gpu_adamw import HYPER, TYPES, _bits, _tensor

pytestmark = pytest.mark.gpu


def _rests(n, seed=0):
    return np.random.default_rng(seed).integers(-127, 128, n).astype(np.int8)


@pytest.mark.parametrize("n", [1, 3, 4, 255, 256, 257, 4095, 4097, 70001])
@pytest.mark.parametrize("grad", list(TYPES))
def test_step_with_remainders(n, grad):
    d, q = _tensor(n, 8, grad, spread=2.0), _rests(n)
    q[d["v"] == 0] = 0
    for off in (0, 3):
        for t in (1, 1000):
            put = lambda a: torch.cat([torch.zeros(off, dtype=a.dtype), a]).to(dev())[off:]  # noqa: E731
            P, G, M, V, R = (put(torch.from_numpy(d["p"])), put(d["g"]), put(torch.from_numpy(d["m"])),
                             put(torch.from_numpy(d["v"])), put(torch.from_numpy(q)))
            S = to_dev(d["s"])
            say("adamw carried", n, grad, off, t)
            ops.ionn_adamw_step([P], [G], [M], [V], t, Ss=[S], Rs=[R], **HYPER)
            want = of.adamw_step(d["p"], d["g"].float().numpy(), d["m"], d["v"], t, exps=d["s"], rest=q, **HYPER)
            for x, y, k in zip((P, M, V, S, R), want, "PMVSR"):
                _bits(host(x), y, f"n {n} t {t} {k}")


def test_not_finite_roots_have_no_remainder():
    d, q = _tensor(1000, 8, "f32"), _rests(1000)
    d["g"][10], d["g"][300], d["g"][999] = float("nan"), float("inf"), -float("inf")
    P, M, V, S, R = (to_dev(x) for x in (d["p"], d["m"], d["v"], d["s"], q))
    ops.ionn_adamw_step([P], [d["g"].to(dev())], [M], [V], 5, Ss=[S], Rs=[R], **HYPER)
    want = of.adamw_step(d["p"], d["g"].numpy(), d["m"], d["v"], 5, exps=d["s"], rest=q, **HYPER)
    for x, y, k in zip((P, M, V, S, R), want, "PMVSR"):
        _bits(host(x), y, k)
    assert not host(R)[[10, 300, 999]].any()


def test_class_carries_remainders():
    """Twenty steps of the optimiser class, bit for bit, and resumed from its states."""
    n = 3000
    P = torch.zeros(n, device=dev())
    opt = steps.AdamW.make([P], bits=8, Rs=None, lr=1e-2, weight_decay=0.1)
    ref = [np.zeros(n, np.float32), np.zeros(n, np.uint8), np.zeros(n, np.uint8), np.zeros((-(-n // 256), 2), np.int8),
           np.zeros(n, np.int8)]
    for t in range(1, 21):
        g = np.random.default_rng(t).standard_normal(n).astype(np.float32)
        if t == 11:
            opt = steps.AdamW(opt.P, opt.M, opt.V, opt.S, lr=1e-2, weight_decay=0.1, t=opt.t, Rs=opt.R)
        opt.step([to_dev(g)])
        ref = list(of.adamw_step(ref[0], g, ref[1], ref[2], t, 1e-2, 0.9, 0.999, 1e-8, 0.1, exps=ref[3], rest=ref[4]))
        for x, y, k in zip((P, opt.M[0], opt.V[0], opt.S[0], opt.R[0]), ref, "PMVSR"):
            _bits(host(x).reshape(y.shape), y, f"step {t} {k}")


@pytest.mark.parametrize("beta2", [0.95, 0.999])
def test_second_moment_follows_its_definition(beta2):
    n = 16384
    new = lambda dt: torch.zeros(n, dtype=dt, device=dev())  # noqa: E731
    say("adamw long", beta2)
    words, carried, codes = (steps.AdamW.make([new(torch.float32)], bits=b, betas=(0.9, beta2), weight_decay=0.0, Rs=rs)
                             for b, rs in ((32, None), (8, None), (8, False)))
    gen = torch.Generator(device=dev()).manual_seed(5)
    for t in range(1, 3001):
        g = torch.randn(n, generator=gen, device=dev()) * (1.0 if t < 1000 else 0.1 if t < 2000 else 3.0)
        words.step([g])
        carried.step([g])
        codes.step([g])
        if t in (10, 200, 999, 1100, 1999, 2100, 3000):
            v = host(words.V[0]).astype(np.float64)
            vc = of.state_decode(host(codes.V[0]), host(codes.S[0])[:, 1]).astype(np.float64) ** 2
            root = of.root_decode_carried(host(carried.V[0]), host(carried.R[0]), host(carried.S[0])[:, 1])
            ratio = root / np.sqrt(v)
            say(t, "codes %.4f" % (vc.mean() / v.mean()), "carried %.4f %.4f" % (np.median(ratio), np.sqrt(np.mean((ratio - 1) ** 2))))
            assert abs(vc.mean() / v.mean() - 1) < 0.044
            assert abs(np.median(ratio) - 1) < 0.004 and np.sqrt(np.mean((ratio - 1) ** 2)) < 0.034


def test_refuses_remainders_that_do_not_fit():
    z = lambda n, dt=torch.float32: torch.zeros(n, dtype=dt, device=dev())  # noqa: E731
    u8, i8 = torch.uint8, torch.int8
    S = [torch.zeros(1, 2, dtype=i8, device=dev())]
    with pytest.raises(ValueError, match="R of a tensor"):
        ops.ionn_adamw_step([z(4)], [z(4)], [z(4, u8)], [z(4, u8)], 1, 1e-3, Ss=S, Rs=[z(3, i8)])
    with pytest.raises(ValueError, match="R of a tensor"):
        ops.ionn_adamw_step([z(4)], [z(4)], [z(4)], [z(4)], 1, 1e-3, Rs=[z(4, i8)])
    with pytest.raises(TypeError, match="R"):
        ops.ionn_adamw_step([z(4)], [z(4)], [z(4, u8)], [z(4, u8)], 1, 1e-3, Ss=S, Rs=[z(4, u8)])
    with pytest.raises(ValueError, match="remainders"):
        steps.AdamW([z(4)], [z(4)], [z(4)], Rs=[z(4, i8)])
    with pytest.raises(ValueError, match="remainders"):
        steps.AdamW([z(4)], [z(4, u8)], [z(4, u8)], S, Rs=[z(5, i8)])
