"""GPU: the AdamW step over many tensors against the oracle, bit for bit: the
definition rounds every operation to float32 on its own, so weights, moments,
8-bit codes and block exponents all have one right value."""
import numpy as np
import pytest
import torch

from gpu_helpers import dev, host, say, to_dev
from integer_only_nn_amd import ops, steps
from oracle import floats as of

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HYPER = dict(lr=1e-2, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1)


def _bits(a, b, what):
    a, b = np.ascontiguousarray(a), np.ascontiguousarray(b)
    if a.dtype == np.float32:
        nan = np.isnan(a) & np.isnan(b)
        a, b = np.where(nan, 0, a.view(np.uint32)), np.where(nan, 0, b.view(np.uint32))
    bad = np.flatnonzero(a.reshape(-1) != b.reshape(-1))
    assert bad.size == 0, f"{what}: {bad.size} of {a.size} differ, first at {bad[:5]}"


def _tensor(n, bits, grad, seed=0, spread=1.0):
    rng = np.random.default_rng(seed + n)
    d = dict(p=rng.standard_normal(n).astype(np.float32),
             g=torch.from_numpy(rng.standard_normal(n) * np.exp(spread * rng.standard_normal(n)) * 1e-2).float().to(TYPES[grad]),
             m=(rng.standard_normal(n) * np.exp(spread * rng.standard_normal(n)) * 1e-2).astype(np.float32),
             v=np.square(rng.standard_normal(n) * 1e-2).astype(np.float32), s=None)
    if bits == 8:
        (m, em), (r, er) = of.state_encode(d["m"], False), of.state_encode(np.sqrt(d["v"]), True)
        d.update(m=m, v=r, s=np.stack([em, er], 1))
    return d


def _want(d, t, scale=1.0, **kw):
    return of.adamw_step(d["p"], d["g"].float().numpy(), d["m"], d["v"], t, grad_scale=scale, exps=d["s"],
                         **{**HYPER, **kw})


def _run(ds, t, bits, grad_scale=None, off=0, absmax=None, **kw):
    """The library's step of these tensors (each `off` elements into its storage)."""
    put = lambda a: torch.cat([torch.zeros(off, dtype=a.dtype), a]).to(dev())[off:]  # noqa: E731
    of_np = lambda a: put(torch.from_numpy(a))  # noqa: E731
    P, G, M, V = [of_np(d["p"]) for d in ds], [put(d["g"]) for d in ds], [of_np(d["m"]) for d in ds], [of_np(d["v"]) for d in ds]
    S = None if bits == 32 else [to_dev(d["s"]) for d in ds]
    say("adamw", bits, len(ds), [d["p"].size for d in ds][:8])
    ops.ionn_adamw_step(P, G, M, V, t, Ss=S, grad_scale=grad_scale, absmax_P=absmax, **{**HYPER, **kw})
    return [tuple(host(x) for x in ((p, m, v) if S is None else (p, m, v, S[i]))) for i, (p, m, v) in enumerate(zip(P, M, V))]


def _compare(got, want, what=""):
    for i, (a, b) in enumerate(zip(got, want)):
        for x, y, k in zip(a, b, ("P", "M", "V", "S")):
            _bits(x, y, f"{what} tensor {i} {k}")


@pytest.mark.parametrize("n", [1, 3, 4, 63, 255, 256, 257, 1023, 1025, 4095, 4096, 4097, 70001])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("grad", list(TYPES))
def test_one_tensor(n, bits, grad):
    d = _tensor(n, bits, grad)
    for t in (1, 2, 1000):
        _compare(_run([d], t, bits), [_want(d, t)])


@pytest.mark.parametrize("bits", [32, 8])
def test_many_tensors_in_several_launches(bits):
    sizes = [1 + (37 * i * i) % 5000 for i in range(150)]
    ds = [_tensor(n, bits, "bf16", seed=i) for i, n in enumerate(sizes)]
    top = torch.zeros(150, dtype=torch.int32, device=dev())
    got = _run(ds, 5, bits, absmax=top)
    _compare(got, [_want(d, 5) for d in ds])
    want = np.array([np.abs(g[0]).max() for g in got], np.float32)
    _bits(host(top).view(np.float32), want, "absmax")


@pytest.mark.parametrize("bits", [32, 8])
def test_tensors_that_start_anywhere(bits):
    for off in (1, 2, 3):
        ds = [_tensor(n, bits, "f16") for n in (5, 300, 5000)]
        _compare(_run(ds, 3, bits, off=off), [_want(d, 3) for d in ds])


@pytest.mark.parametrize("bits", [32, 8])
def test_wide_ranges_within_a_block(bits):
    d = _tensor(3000, bits, "f32", spread=6.0)
    _compare(_run([d], 4, bits), [_want(d, 4)])


def test_hyperparameters():
    for kw in (dict(beta1=0.0), dict(beta2=0.0), dict(weight_decay=0.0), dict(lr=0.0), dict(eps=0.0), dict(eps=1.0)):
        for bits in (32, 8):
            d = _tensor(700, bits, "f32")
            _compare(_run([d], 2, bits, **kw), [_want(d, 2, **kw)], str(kw))


@pytest.mark.parametrize("bits", [32, 8])
def test_zero_states_and_gradients(bits):
    d = _tensor(600, bits, "f32")
    d["m"][:], d["v"][:] = 0, 0
    if bits == 8:
        d["s"][:] = 0
    got = _run([d], 1, bits)
    _compare(got, [_want(d, 1)])
    d["g"] = torch.zeros(600)
    d["g"][300:] = 1e-3  # the first block stays zero, the others do not
    got = _run([d], 1, bits)
    _compare(got, [_want(d, 1)])
    assert (got[0][0][:300] == d["p"][:300] * np.float32(1 - 1e-3)).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_not_finite_gradients_stay_in_their_element(bits):
    d = _tensor(1000, bits, "f32")
    d["g"][10], d["g"][300], d["g"][999] = float("nan"), float("inf"), -float("inf")
    got, want = _run([d], 2, bits), [_want(d, 2)]
    _compare(got, want)
    good = np.ones(1000, bool)
    good[[10, 300, 999]] = False
    assert np.isfinite(got[0][0][good]).all() and not np.isfinite(got[0][0][~good]).any()
    if bits == 8:
        assert (got[0][1][~good] & 0x7f == 0x7f).all() and not (got[0][1][good] & 0x7f == 0x7f).any()


@pytest.mark.parametrize("bits", [32, 8])
def test_gradient_scale(bits):
    d = _tensor(900, bits, "bf16")
    s = torch.tensor([0.37], device=dev())
    _compare(_run([d], 2, bits, grad_scale=s), [_want(d, 2, scale=float(s.cpu()[0]))])


@pytest.mark.parametrize("bits", [32, 8])
def test_consecutive_steps(bits):
    """Ten steps of the optimiser class, each state feeding the next."""
    ds = [_tensor(n, bits, "f32", seed=n) for n in (33, 4000)]
    P = [to_dev(d["p"]) for d in ds]
    opt = steps.AdamW.make(P, bits=bits, **{"lr": 1e-2, "betas": (0.9, 0.999), "eps": 1e-8, "weight_decay": 0.1})
    ref = [dict(d, m=np.zeros(d["p"].size, d["m"].dtype), v=np.zeros(d["p"].size, d["v"].dtype),
                s=None if bits == 32 else np.zeros_like(d["s"])) for d in ds]
    for t in range(1, 11):
        rng = np.random.default_rng(t)
        for r in ref:
            r["g"] = torch.from_numpy(rng.standard_normal(r["p"].size)).float()
        opt.step([r["g"].to(dev()) for r in ref])
        for i, r in enumerate(ref):
            out = _want(r, t)
            r.update(p=out[0], m=out[1], v=out[2], s=None if bits == 32 else out[3])
            _bits(host(P[i]), r["p"], f"step {t} tensor {i}")
    assert opt.t == 10


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_steps_replay(bits):
    """Steps in a graph, with the count and the learning rate on the device,
    replayed with eager work in between."""
    d = _tensor(5000, bits, "f32")
    ref = dict(d, m=np.zeros(5000, d["m"].dtype), v=np.zeros(5000, d["v"].dtype),
               s=None if bits == 32 else np.zeros_like(d["s"]))
    P, G = to_dev(d["p"]), torch.zeros(5000, device=dev())
    opt = steps.AdamW.make([P], bits=bits, lr=1e-2, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.1, on_device=True)
    opt.bind_grads([G])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step()
    for t in range(1, 5):
        lr = 1e-2 / t
        G.copy_(torch.from_numpy(np.random.default_rng(t).standard_normal(5000)).float())
        opt.lr_dev.fill_(lr)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        ref["g"] = G.cpu()
        out = _want(ref, t, lr=float(np.float32(lr)))
        ref.update(p=out[0], m=out[1], v=out[2], s=None if bits == 32 else out[3])
        _bits(host(P), ref["p"], f"replay {t}")
