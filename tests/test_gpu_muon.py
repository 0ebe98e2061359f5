"""GPU: the Muon step (ionn_muon_step, steps.Muon) against the oracle in 64 bits.

Tolerances.  M is one fused operation: half a step of float32, and half a step
of the momentum's factor.  Of X: the products' operands are pairs of float16 terms, off by
2^-23 of themselves at most (half a step of the low term, whose own leading bit
is 2^-12 of the value or less), lo lo is left out (2^-24), and a sum of K terms
in float32 rounds K times, to half a step of a partial sum each, which add up as
independent errors do (sqrt(K) 2^-24 of the terms' root sum of squares).  How
far such errors move X depends on its singular values, so the oracle runs the
same steps with errors of those sizes drawn at random, and X may be off by four
times what that moves it (in the root of the sum of squares; a single element by
that spread over all, times 12, which a normal variable exceeds once in 10^32)."""
import numpy as np
import pytest
import torch

from gpu_helpers import dev, host, say, to_dev
from integer_only_nn_amd import ops, steps
from oracle import floats as of
from test_gpu_dfp8_linear import TYPES, _np, _round, _typed, _ws

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _model(rng):
    """A product with its operands' and its sums' roundings, drawn at random."""
    def rounded(p, q):
        noisy = lambda t: t * (1 + 2.0 ** -22 * rng.uniform(-1, 1, t.shape))  # noqa: E731
        size = np.sqrt((p * p) @ (q * q))
        return noisy(p) @ noisy(q) + np.sqrt(p.shape[1]) * U * size * rng.standard_normal(size.shape)
    return rounded


def _case(rows, cols, kind="gauss", seed=0):
    rng = np.random.default_rng(seed + 100 * rows + cols)
    f = lambda *s: rng.standard_normal(s)  # noqa: E731
    k = min(4, rows, cols)
    m = 1e-3 * f(rows, cols) + (2e-3 * f(rows, k) @ f(k, cols) if kind == "strong" else 0.0)
    return dict(P=(f(rows, cols) / np.sqrt(cols)).astype(np.float32), G=1e-3 * f(rows, cols), M=m.astype(np.float32))


def _check(P, M, d, name, lr=0.5, momentum=0.95, nesterov=True, eps=1e-7, weight_decay=0.1, ns_steps=5, scale=None, gs=1.0):
    G = _round(d["G"], name) * gs
    args = (d["P"], G, d["M"], lr, np.float32(momentum), nesterov, eps, weight_decay, ns_steps, scale)
    p, m, x = of.muon_step(*args)
    assert (np.abs(_np(M) - m) <= 3 * U * (np.abs(momentum * d["M"]) + np.abs(G)) + 2.0 ** -149).all()
    moved = max(np.linalg.norm(of.muon_step(*args, rounded=_model(np.random.default_rng(s)))[2] - x) for s in range(2))
    s = np.sqrt(max(1.0, p.shape[0] / p.shape[1])) if scale is None else abs(scale)
    # X itself is rounded once more to a pair (2^-22), its first form and P in float32
    tol = abs(lr * s) * (4 * moved + 2.0 ** -21 * np.linalg.norm(x))
    own = 3 * U * (np.abs(d["P"]) + abs(lr * s) * np.abs(x))
    off = np.maximum(np.abs(_np(P) - p) - own, 0.0)
    say("off", np.linalg.norm(off), "tolerance", tol)
    assert np.linalg.norm(off) <= tol
    assert off.max() <= 12 * tol / np.sqrt(p.size) + 3 * U


def _step(ds, name, absmax=True, lr=0.5, weight_decay=0.1, **kw):
    P, M = [to_dev(d["P"]) for d in ds], [to_dev(d["M"]) for d in ds]
    G = [_typed(d["G"], name) for d in ds]
    top = torch.zeros(len(ds), dtype=torch.int32, device=dev()) if absmax else None
    say("muon", [d["P"].shape for d in ds], name)
    ops.ionn_muon_step(P, G, M, lr, _ws(ops.ionn_muon_workspace_bytes([p.shape for p in P])), weight_decay=weight_decay,
                       absmax_P=top, **kw)
    if absmax:
        assert host(top).view(np.float32).tolist() == [float(p.abs().max()) for p in P]
    return P, M


SHAPES = [(1, 1), (1, 5), (7, 1), (3, 3), (33, 2), (10, 128), (64, 64), (128, 256), (100, 30), (129, 127), (256, 784),
          (784, 256), (300, 513), (128, 3000), (700, 1000)]
LARGE = [(2048, 2048), (2000, 2100), (2100, 1990), (1024, 4096), (1030, 4500), (4100, 1300), (2304, 2304), (2250, 2500),
         (2500, 2300), (1300, 8000), (20000, 40), (1100, 1000)]
# tiles by sizes, as the CPU test holds them to
TILES = {32: [(1, 1), (256, 784), (512, 512), (30, 8192)], 64: [(700, 1000), (1100, 1000)],
         128: [(2048, 2048), (2100, 1990), (1024, 4096), (20000, 40)], 256: [(2304, 2304), (2500, 2300), (1300, 8000)]}


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("name", list(TYPES))
def test_step(rows, cols, name):
    for nesterov in (True, False):
        d = _case(rows, cols)
        P, M = _step([d], name, nesterov=nesterov)
        _check(P[0], M[0], d, name, nesterov=nesterov)


@pytest.mark.parametrize("rows,cols", LARGE)
def test_step_of_a_large_matrix(rows, cols):
    d = _case(rows, cols)
    P, M = _step([d], "bf16")
    _check(P[0], M[0], d, "bf16")


@pytest.mark.parametrize("rows,cols", [(30, 8192), (512, 512)])
def test_step_of_a_long_reduction(rows, cols):
    d = _case(rows, cols)
    P, M = _step([d], "f16")
    _check(P[0], M[0], d, "f16")


@pytest.mark.parametrize("rows,cols", [(64, 64), (200, 300), (400, 100), (2048, 2048)])
def test_step_of_few_strong_directions(rows, cols):
    d = _case(rows, cols, "strong")
    P, M = _step([d], "f32")
    _check(P[0], M[0], d, "f32")


def test_many_matrices_at_once():
    """More than a launch takes, small and large ones in any order, each as it is by itself."""
    shapes = [(10, 128), (300, 200), (2048, 2050), (1, 9), (128, 256), (5, 5), (256, 784), (64, 1), (90, 90), (33, 70), (70, 33),
              (2, 2), (2400, 2300), (3, 4), (600, 800), (900, 700)]
    ds = [_case(*s, seed=i) for i, s in enumerate(shapes)]
    P, M = _step(ds, "bf16")
    for p, m, d in zip(P, M, ds):
        _check(p, m, d, "bf16")


def test_settings():
    d = _case(60, 90)
    gs, lr = torch.tensor([0.25], device=dev()), torch.tensor([0.125], device=dev())
    P, M = _step([d], "f32", lr=99.0, lr_dev=lr, grad_scale=gs, momentum=0.5, ns_steps=3, scale=[2.5], eps=0.0)
    _check(P[0], M[0], d, "f32", lr=0.125, gs=0.25, momentum=0.5, ns_steps=3, scale=2.5, eps=0.0)
    P, M = _step([d], "f32", momentum=0.0, weight_decay=0.0, ns_steps=1)
    _check(P[0], M[0], d, "f32", momentum=0.0, weight_decay=0.0, ns_steps=1)


def test_updates_of_any_size():
    """Squares that leave float32's range; eps where it counts; an update of zeros."""
    for scale, eps in ((1e30, 1e-7), (1e-30, 0.0), (1e-5, 1e-3)):
        d = _case(40, 50)
        d["G"], d["M"] = d["G"] * scale, (d["M"] * scale).astype(np.float32)
        P, M = _step([d], "f32", eps=eps)
        _check(P[0], M[0], d, "f32", eps=eps)
    for eps in (0.0, 1e-7):
        d = _case(40, 50)
        d["G"], d["M"] = 0 * d["G"], 0 * d["M"]
        P, M = _step([d], "f32", lr=0.5, weight_decay=0.1, eps=eps)
        assert (host(P[0]) == d["P"] * np.float32(1 - 0.05)).all() and not host(M[0]).any()


def test_what_is_not_finite_stays_in_its_matrix():
    for bad in (np.nan, np.inf):
        for shape in ((40, 50), (2048, 2048), (2304, 2304)):
            ds = [_case(20, 30), _case(*shape), _case(30, 20)]
            ds[1]["G"][3, 4] = bad
            P, M = _step(ds, "f32", absmax=False)
            assert torch.isnan(P[1]).all() and int((~torch.isfinite(M[1])).sum()) == 1
            for i in (0, 2):
                _check(P[i], M[i], ds[i], "f32")


def test_nothing_else_is_written():
    """Weights and momenta inside larger storage, at addresses of one element."""
    rows, cols = 37, 41
    d = _case(rows, cols)
    n = rows * cols
    P, M = (torch.full((n + 64,), 5.0, device=dev()) for _ in range(2))
    G = torch.zeros(n + 1, dtype=torch.bfloat16, device=dev())
    P[1:n + 1], M[3:n + 3], G[1:] = to_dev(d["P"]).view(-1), to_dev(d["M"]).view(-1), _typed(d["G"], "bf16").view(-1)
    need = ops.ionn_muon_workspace_bytes([(rows, cols)])
    ws = torch.full((need + 256,), 77, dtype=torch.uint8, device=dev())
    ops.ionn_muon_step([P[1:n + 1].view(rows, cols)], [G[1:].view(rows, cols)], [M[3:n + 3].view(rows, cols)], 0.5, ws[:need],
                       weight_decay=0.1)
    _check(P[1:n + 1].view(rows, cols), M[3:n + 3].view(rows, cols), d, "bf16")
    assert (P[n + 1:] == 5).all() and P[0] == 5 and (M[n + 3:] == 5).all() and (M[:3] == 5).all() and (ws[need:] == 77).all()


@pytest.mark.parametrize("rows,cols", [(300, 500), (33, 65), (900, 1000), (2048, 2048), (2304, 2310)])
def test_the_result_does_not_depend_on_the_workspace(rows, cols):
    d = _case(rows, cols)
    out = []
    for fill in (0, 0xff):
        P, M = to_dev(d["P"]), to_dev(d["M"])
        ws = torch.full((ops.ionn_muon_workspace_bytes([P.shape]),), fill, dtype=torch.uint8, device=dev())
        ops.ionn_muon_step([P], [_typed(d["G"], "f32")], [M], 0.5, ws)
        out.append(P)
    assert torch.equal(*out)


def test_orthogonal_after_many_steps_of_the_polynomial():
    """Singular values of X lie where the polynomial keeps them, 0.68 to 1.21."""
    for rows, cols in ((100, 300), (300, 100)):
        d = _case(rows, cols)
        d["P"][:] = 0
        P, _ = _step([d], "f32", lr=1.0, weight_decay=0.0, scale=[1.0], ns_steps=8)
        s = np.linalg.svd(_np(P[0]), compute_uv=False)
        assert 0.67 < s.min() and s.max() < 1.22


def test_optimiser_over_several_steps_and_on_another_stream():
    ds = [_case(40, 70), _case(2304, 2304), _case(90, 33)]
    Ps, Ms = [d["P"].astype(np.float64) for d in ds], [0 * d["M"].astype(np.float64) for d in ds]
    P = [to_dev(d["P"]) for d in ds]
    opt = steps.Muon.make(P, lr=0.01, weight_decay=0.1)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    rng = np.random.default_rng(1)
    for k in range(3):
        Gs = [_round(1e-3 * rng.standard_normal(p.shape), "bf16") for p in Ps]
        opt.step([_typed(g, "bf16") for g in Gs], stream=s if k == 1 else None)
        torch.cuda.synchronize()
        for i, g in enumerate(Gs):
            Ps[i], Ms[i], _ = of.muon_step(Ps[i], g, Ms[i], 0.01, np.float32(0.95), True, 1e-7, 0.1, 5)
    for i in range(3):
        # three steps of 0.01 sqrt(max(1, rows / cols)) X, each X off by less than 2e-5 of its size, P by 3 half steps a step
        x = 0.01 * max(1.0, np.sqrt(P[i].shape[0] / P[i].shape[1])) * 1.22 * np.sqrt(min(P[i].shape))
        assert np.linalg.norm(_np(P[i]) - Ps[i]) <= 3 * (2e-5 * x + 3 * U * np.linalg.norm(Ps[i]))
        assert np.linalg.norm(_np(opt.M[i]) - Ms[i]) <= 9 * U * np.linalg.norm(Ms[i])


def test_repeatable_and_captured():
    ds = [_case(40, 70), _case(300, 200), _case(2350, 2304), _case(900, 1000), _case(33, 10)]
    a, b = _step(ds, "bf16"), _step(ds, "bf16")
    assert all(torch.equal(p, q) for p, q in zip(a[0] + a[1], b[0] + b[1]))
    P, Q = ([to_dev(d["P"]) for d in ds] for _ in range(2))
    G = [_typed(d["G"], "bf16") for d in ds]
    opt, eager = (steps.Muon.make(w, lr=0.02, weight_decay=0.1, on_device=True) for w in (P, Q))
    opt.bind_grads(G)
    eager.bind_grads(G)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        opt.step()
    torch.cuda.current_stream().wait_stream(s)
    eager.step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step()
    for k in range(3):
        for g, d in zip(G, ds):
            g.copy_(torch.randn(g.shape, device=dev()) * 1e-3)
        opt.lr_dev.fill_(0.01 / (k + 1))
        eager.lr_dev.fill_(0.01 / (k + 1))
        graph.replay()
        torch.cuda.synchronize()
        eager.step()
        assert all(torch.equal(p, q) for p, q in zip(P + opt.M, Q + eager.M))
