"""GPU: gated feed-forward blocks on a residual stream (steps.GatedMlps), which
run the gated layer, the norms around a block, the Linear layer, the DFP-8
conversion, Muon and AdamW together as a training step: against the blocks in
float64, their gradients against differences, and step by step from a graph."""
import numpy as np
import pytest
import torch

from gpu_helpers import dev, host, say
from integer_only_nn_amd import steps
from oracle import floats as of

pytestmark = pytest.mark.gpu


def _make(B, D, H, L=2, norm="rms", full=True, seed=0, **kw):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    blocks = []
    for _ in range(L):
        b = dict(W1=r(2 * H, D) / D ** 0.5, W2=r(D, H) / H ** 0.5)
        if full:
            b.update(b1=0.1 * r(2 * H), b2=0.1 * r(D), gamma=1 + 0.1 * r(D), gate=0.5 + 0.1 * r(D))
            if norm == "layer":
                b["beta"] = 0.1 * r(D)
        blocks.append({k: v.to(dev()) for k, v in b.items()})
    gamma = [(1 + 0.1 * r(D)).to(dev()) for _ in range(L + 1)]
    beta = [(0.1 * r(D)).to(dev()) for _ in range(L + 1)] if norm == "layer" else None
    x, dn, dy = r(B, D), 0.1 * r(B, D), 0.1 * r(B, D)
    return steps.GatedMlps(blocks, gamma, B, norm=norm, beta=beta, **kw), x, dn, dy


class Reference:
    """The blocks in float64, without any rounding to 8 bits."""

    def __init__(self, m):
        f = lambda t: None if t is None else host(t).astype(np.float64)  # noqa: E731
        self.blocks = [{k: f(v) for k, v in b.items()} for b in m.blocks]
        self.gamma, self.beta = [f(v) for v in m.gamma], [f(v) for v in m.beta]
        self.norm, self.act, self.alpha, self.eps = m.norm, m.act, m.alpha, m.eps

    def _pass(self, l, a, y, blk):
        post = "none" if blk is None or blk["gamma"] is None else self.norm
        gate = None if blk is None or blk["gate"] is None else blk["gate"][None]
        vec = (None, None) if blk is None else (blk["gamma"], blk["beta"])
        args = (post, *vec, gate, 0, 1.0 if blk is None else self.alpha, self.norm, self.gamma[l])
        return args, of.residual_norm_fwd(a, y, *args, self.beta[l], self.eps)

    def forward(self, x):
        self.kept = [(None, x, *self._pass(0, None, x, None))]
        y, n = x, self.kept[0][3]["n"]
        for l, b in enumerate(self.blocks):
            H = b["W2"].shape[1]
            z = n @ b["W1"].T + (0 if b["b1"] is None else b["b1"])
            h = of.act(z[:, :H], self.act) * z[:, H:]
            a = h @ b["W2"].T + (0 if b["b2"] is None else b["b2"])
            args, w = self._pass(l + 1, a, y, b)
            self.kept.append((a, y, args, w, z, h, n))
            y, n = w["y"], w["n"]
        return y, n

    def backward(self, dn, dy):
        out = {}
        for l in reversed(range(len(self.blocks) + 1)):
            a, y, args, w = self.kept[l][:4]
            stream = w["y"] if l else y
            g = of.residual_norm_bwd(dy, dn, a, stream, *args, *(w[k] for k in ("mean_a", "rstd_a", "mean_y", "rstd_y")))
            out[f"ggamma {l}"], out[f"gbeta {l}"] = g["dgamma_y"], g["dbeta_y"]
            if l == 0:
                out["dx"] = g["dx"]
                return out
            z, h, n = self.kept[l][4:]
            b = self.blocks[l - 1]
            da, dy = g["da"], g["dx"]
            dz = of.gated_error(da @ b["W2"], z, self.act)
            dn = dz @ b["W1"]
            out.update({f"{k} of {l - 1}": v for k, v in dict(
                gW2=da.T @ h, gb2=da.sum(0), gW1=dz.T @ n, gb1=dz.sum(0), ggamma=g["dgamma_a"], gbeta=g["dbeta_a"],
                ggate=g.get("dgate")).items()})


def _got(m, key):
    if key == "dx":
        return m.dx
    k, l = key.rsplit(" ", 1)
    return m.bufs[int(l)][k[:-3]] if k.endswith(" of") else getattr(m, k)[int(l)]


@pytest.mark.parametrize("B,D,H,norm,full", [(1, 64, 256, "rms", True), (37, 100, 333, "layer", True), (300, 256, 512, "rms", False),
                                             (512, 256, 700, "layer", True)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_against_float64(B, D, H, norm, full, dtype):
    """Each value that becomes 8 bits is off by at most half a step of the
    tensor's largest: a relative error of 0.03 each at the most (as in the residual
    MLP block's test).  An output's error of each block has n, W1, the hidden
    activation (a product of two such sums: n and W1 twice) and W2: six in
    quadrature, 0.073, and of two blocks 0.104; a gradient has as many again behind
    it and its own error's rounding, and a norm's gradient subtracts what of it
    lies along the row: below 0.2 for one block's products in quadrature with the
    other's."""
    m, x, dn, dy = _make(B, D, H, norm=norm, full=full, dtype=dtype)
    x, dn, dy = (t.to(dtype).to(dev()) for t in (x, dn, dy))
    m.forward(x)
    m.backward(x, dn, dy)
    assert not host(m.status).any()
    ref = Reference(m)
    y, n = ref.forward(host(x.double()))
    rel = lambda got, want: np.linalg.norm(host(got.double()).reshape(want.shape) - want) / np.linalg.norm(want)  # noqa: E731
    assert rel(m.n, n) < 0.104 and rel(m.bufs[-1]["y"], y) < 0.104
    for k, w in ref.backward(host(dn.double()), host(dy.double())).items():
        got = _got(m, k) if w is not None else None
        if got is None:
            assert w is None or "gbeta" in k or not full or k.startswith("gbeta"), k
            continue
        say(k, "%.4f" % rel(got, w))
        assert rel(got, w) < 0.2, k


def test_reference_gradient_against_differences():
    """The float64 blocks' own gradient (the one above is held to) against central differences of their forward pass."""
    m, x, dn, dy = _make(5, 12, 10, norm="layer")
    ref = Reference(m)
    x, dn, dy = (t.double().numpy() for t in (x, dn, dy))

    def loss():
        y, n = ref.forward(x)
        return (dn * n).sum() + (dy * y).sum()
    loss()
    want = ref.backward(dn, dy)
    rng, h = np.random.default_rng(0), 2.0 ** -16
    places = [(x, "dx")] + [(ref.gamma[i], f"ggamma {i}") for i in range(3)] + [(ref.beta[i], f"gbeta {i}") for i in range(3)]
    places += [(ref.blocks[l][p], f"g{p} of {l}") for l in range(2) for p in ("W1", "W2", "b1", "b2", "gamma", "beta", "gate")]
    scale = np.abs(dn).sum() + np.abs(dy).sum()
    for t, k in places:
        for _ in range(4):
            at = tuple(rng.integers(s) for s in t.shape)
            old = t[at]
            t[at] = old + h
            hi = loss()
            t[at] = old - h
            lo = loss()
            t[at] = old
            # third derivatives below 10^4 times the errors' sum; 1e-16 / h of cancellation
            assert abs((hi - lo) / (2 * h) - want[k].reshape(t.shape)[at]) <= scale * (1e4 * h * h + 1e-10), (k, at)


@pytest.mark.parametrize("B,D,H,kw", [(65, 96, 200, dict(norm="layer")), (300, 256, 512, dict(matrices="adamw", full=False)),
                                      (40, 128, 130, dict(alpha=0.5, L=3))])
def test_captured_step_replays(B, D, H, kw):
    """Forward, backward and update in one graph, replayed with other inputs
    and eager work in between, bit for bit what eager steps give."""
    say("graph", B, D, H, kw)
    eager, x, dn, dy = _make(B, D, H, on_device=True, **kw)
    m = _make(B, D, H, on_device=True, **kw)[0]
    x, dn, dy = (t.to(dev()).bfloat16() for t in (x, dn, dy))

    def step(k):
        k.forward(x)
        k.backward(x, dn, dy)
        k.update()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(m)
    for k in range(3):
        g = torch.Generator().manual_seed(10 + k)
        x.copy_(torch.randn(B, D, generator=g).bfloat16())
        dn.copy_((0.1 * torch.randn(B, D, generator=g)).bfloat16())
        step(eager)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        same = [(m.n, eager.n), (m.dx, eager.dx), (m.e, eager.e), (m.top, eager.top)] + list(zip(m.gamma, eager.gamma))
        for a, b, p, q in zip(m.blocks, eager.blocks, m.bufs, eager.bufs):
            same += [(a[i], b[i]) for i in a if a[i] is not None] + [(p[i], q[i]) for i in ("W1_8", "gW1", "gW2", "y")]
        assert all(torch.equal(a, b) for a, b in same), f"replay {k}"


@pytest.mark.parametrize("matrices", ["muon", "adamw"])
def test_an_update_moves_what_it_should(matrices):
    """The weights by the optimiser's definition from the block's own gradients, and their 8-bit copies by the new weights."""
    m, x, dn, dy = _make(50, 64, 96, matrices=matrices, lr=0.01, weight_decay=0.1, dtype=torch.float32)
    x, dn, dy = (t.to(dev()) for t in (x, dn, dy))
    before = [{k: host(v).copy() for k, v in b.items() if v is not None} for b in m.blocks]
    m.forward(x)
    m.backward(x, dn, dy)
    m.update()
    for b, old, t in zip(m.blocks, before, m.bufs):
        if matrices == "muon":
            H, gW1 = 96, host(t["gW1"])
            parts = [(old["W1"][:H], gW1[:H], host(b["W1"])[:H]), (old["W1"][H:], gW1[H:], host(b["W1"])[H:]),
                     (old["W2"], host(t["gW2"]), host(b["W2"]))]
            for P, G, new in parts:
                want, _, X = of.muon_step(P, G, 0 * P, 0.01, np.float32(0.95), True, 1e-7, 0.1, 5)
                step = 0.01 * np.sqrt(max(1.0, P.shape[0] / P.shape[1])) * np.linalg.norm(X)
                # X off by less than 2e-5 of its size, P by three half steps
                assert np.linalg.norm(new - want) <= 2e-5 * step + 3 * 2.0 ** -24 * np.linalg.norm(want)
        else:
            assert not np.array_equal(old["W1"], host(b["W1"]))
        for k in ("W1", "W2"):
            np.testing.assert_array_equal(host(t[k + "_8"]), of.dfp8(host(b[k]))[0])
        for k in ("b1", "b2", "gamma", "gate"):
            # AdamW's first step: 1e-3 against the gradient's sign, where it is not near 0
            g = host(t["g" + k]).reshape(-1)
            far = np.abs(g) > 1e-5
            moved = host(b[k]).reshape(-1) - old[k].reshape(-1)
            assert (np.abs(moved[far] + 1e-3 * np.sign(g[far])) < 1e-3 * 0.2).all(), k


def test_reports_what_is_not_finite():
    m, x, dn, _ = _make(20, 64, 96)
    x, dn = x.to(dev()).bfloat16(), dn.to(dev()).bfloat16()
    m.forward(x)
    assert not host(m.status).any()
    m.blocks[1]["b1"][5] = float("inf")
    m.forward(x)
    assert host(m.status).tolist() == [0] * 7 + [2] + [0] * 4  # the second block's hidden activation
    m.blocks[1]["b1"][5] = 0.0
    m.forward(x)
    m.backward(x, dn)
    assert not host(m.status).any()


def test_refuses_what_does_not_fit():
    z = lambda *s: torch.zeros(*s, device=dev())  # noqa: E731
    ok = dict(W1=z(12, 4), W2=z(4, 6))
    gains = [z(4), z(4)]
    steps.GatedMlps([ok], gains, 2)
    for bad in (dict(ok, W1=z(6, 4)), dict(ok, b1=z(6)), dict(ok, gate=z(5)), dict(ok, beta=z(4)), dict(ok, gamma=z(3))):
        with pytest.raises(ValueError, match="shape mismatch"):
            steps.GatedMlps([bad], gains, 2)
    with pytest.raises(ValueError, match="gains"):
        steps.GatedMlps([ok], gains[:1], 2)
    with pytest.raises(ValueError, match="shifts"):
        steps.GatedMlps([ok], gains, 2, beta=gains)
    with pytest.raises(ValueError, match="norm"):
        steps.GatedMlps([ok], gains, 2, norm="none")
    with pytest.raises(ValueError, match="matrices"):
        steps.GatedMlps([ok], gains, 2, matrices="sgd")
