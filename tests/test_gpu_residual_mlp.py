"""GPU: the residual MLP block (steps.ResidualMlp), which runs the DFP-8
Linear layer, its conversion, layer norm and AdamW together as a training
step: against the block in float64, step by step from a graph, and trained."""
import numpy as np
import pytest
import torch

from gpu_helpers import dev, host, say
from integer_only_nn_amd import ops, steps
from oracle import floats as of

pytestmark = pytest.mark.gpu


def _block(B, D, H, seed=0, **kw):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    p = [(r(H, D) / D ** 0.5), 0.1 * r(H), (r(D, H) / H ** 0.5), 0.1 * r(D), 1 + 0.1 * r(D), 0.1 * r(D)]
    x, dy = r(B, D), 0.1 * r(B, D)
    p = [t.to(dev()) for t in p]
    return steps.ResidualMlp(*p, B=B, **kw), x, dy


def _reference(blk, x, dy):
    """y, dx and the parameters' gradients of the block in float64, without any rounding to 8 bits."""
    W1, b1, W2, b2, g, b = (host(t).astype(np.float64) for t in (blk.W1, blk.b1, blk.W2, blk.b2, blk.gamma, blk.beta))
    x, dy = x.double().numpy(), dy.double().numpy()
    h, mean, rstd = of.layer_norm_fwd(x, g, b, blk.eps)
    z = h @ W1.T + b1
    a = of.act(z, blk.act)
    y = x + a @ W2.T + b2
    dz = (dy @ W2) * of.act_grad(z, blk.act)
    dx, dg, db = of.layer_norm_bwd(dz @ W1, x, mean, rstd, g, dy)
    return dict(y=y, dx=dx, gW1=dz.T @ h, gb1=dz.sum(0), gW2=dy.T @ a, gb2=dy.sum(0), ggamma=dg, gbeta=db)


@pytest.mark.parametrize("B,D,H", [(1, 64, 256), (37, 100, 333), (512, 256, 1024)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_against_float64(B, D, H, dtype):
    """Each value that becomes 8 bits is off by at most half a step of the
    tensor's largest, 2^-7 of it: for values of normal spread, whose largest
    is at most about six times their root mean square, a relative error of
    6 * 2^-7 / sqrt(3) = 0.03 each.  Three such factors meet in y's sum (norm
    output and W1 in z, then activation and W2) and five in the first layer's
    gradients, in quadrature below 0.03 * sqrt(5) = 0.07."""
    say("residual mlp", B, D, H, dtype)
    blk, x, dy = _block(B, D, H, dtype=dtype)
    x, dy = x.to(dtype).float(), dy.to(dtype).float()
    want = _reference(blk, x, dy)
    xd, dyd = x.to(dev()).to(dtype), dy.to(dev()).to(dtype)
    blk.forward(xd)
    blk.backward(xd, dyd)
    assert host(blk.status).tolist() == [0, 0]
    for k, w in want.items():
        got = host(getattr(blk, k).double())
        err = np.linalg.norm(got - w) / np.linalg.norm(w)
        say(k, "%.4f" % err)
        assert err < 0.07, k


@pytest.mark.parametrize("state_bits", [32, 8])
def test_training_reaches_its_target(state_bits):
    """The block learns another block's outputs: the squared error falls to a
    small part of what it was, with 32- and with 8-bit states."""
    B, D, H = 256, 64, 256
    teacher, x, _ = _block(B, D, H, seed=1)
    blk, _, _ = _block(B, D, H, seed=2, state_bits=state_bits, lr=3e-3, weight_decay=0.0)
    x = x.to(dev()).bfloat16()
    target = teacher.forward(x).float().clone()
    first = last = None
    for _ in range(200):
        err = blk.forward(x).float() - target
        last = float(err.square().mean())
        first = first if first is not None else last
        blk.backward(x, (err / D).bfloat16())
        blk.update()
    say("loss", first, last)
    assert last < 0.05 * first


@pytest.mark.parametrize("B,D,H", [(65, 96, 200), (512, 256, 512)])
def test_captured_step_replays(B, D, H):
    """Forward, backward and update in one graph, replayed with other inputs
    and eager work in between, bit for bit what eager steps give."""
    say("graph", B, D, H)
    kw = dict(on_device=True, state_bits=8)
    eager, x, dy = _block(B, D, H, **kw)
    blk, _, _ = _block(B, D, H, **kw)
    xd, dyd = x.to(dev()).bfloat16(), dy.to(dev()).bfloat16()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        blk.forward(xd)
        blk.backward(xd, dyd)
        blk.update()
    for k in range(4):
        g = torch.Generator().manual_seed(10 + k)
        xd.copy_(torch.randn(B, D, generator=g).bfloat16())
        dyd.copy_((0.1 * torch.randn(B, D, generator=g)).bfloat16())
        eager.forward(xd)
        eager.backward(xd, dyd)
        eager.update()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for n in ("y", "dx", "gW1", "gW2", "ggamma", "W1", "W2", "b1", "gamma", "W1_8", "e", "top"):
            assert torch.equal(getattr(blk, n), getattr(eager, n)), f"replay {k}: {n}"


def test_refuses_weights_that_do_not_fit():
    z = lambda *s: torch.zeros(*s, device=dev())  # noqa: E731
    with pytest.raises(ValueError, match="shape mismatch"):
        steps.ResidualMlp(z(8, 4), z(8), z(4, 7), z(4), z(4), z(4), B=2)
    with pytest.raises(ValueError, match="bits"):
        steps.AdamW.make([z(4)], bits=16)
    opt = steps.AdamW.make([z(4)])
    with pytest.raises(ValueError, match="gradient"):
        opt.step()
    with pytest.raises(ValueError, match="gradient"):
        opt.bind_grads([z(5)])
    with pytest.raises(TypeError):
        ops.ionn_adamw_step([z(4)], [z(4).double()], [z(4)], [z(4)], 1, 1e-3)


def test_binding_refuses_wrong_tensors():
    x = torch.zeros(4, 8, device=dev())
    for y, error in ((torch.empty(4, 7, device=dev()), "shape mismatch"), (torch.empty(8, 4, device=dev()), "shape"),
                     (torch.empty(4, 8), "device tensor"), (torch.empty(8, 4, device=dev()).t(), "contiguous")):
        with pytest.raises(ValueError, match=error):
            ops.ionn_layer_norm_fwd(x, y)
    with pytest.raises(TypeError, match="bfloat16"):
        ops.ionn_layer_norm_fwd(x, torch.empty(4, 8, dtype=torch.bfloat16, device=dev()))
    i8 = lambda *s: torch.zeros(*s, dtype=torch.int8, device=dev())  # noqa: E731
    e = torch.zeros(1, dtype=torch.int32, device=dev())
    with pytest.raises(ValueError, match="W has"):
        ops.dfp8_linear_fwd(i8(4, 8), e, i8(3, 7), e, torch.empty(4, 3, device=dev()))
    with pytest.raises(TypeError, match="eX"):
        ops.dfp8_linear_fwd(i8(4, 8), e.float(), i8(3, 8), e, torch.empty(4, 3, device=dev()))
    with pytest.raises(ValueError, match="bias has"):
        ops.dfp8_linear_fwd(i8(4, 8), e, i8(3, 8), e, torch.empty(4, 3, device=dev()), bias=torch.zeros(4, device=dev()))
