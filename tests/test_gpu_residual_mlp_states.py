"""GPU: what the residual MLP block and the optimiser report and keep: the
status of every 8-bit operand, updates without a forward pass between them,
and refused optimiser steps."""
import pytest
import torch

from gpu_helpers import dev, host, say
from integer_only_nn_amd import ops, steps
from test_gpu_residual_mlp import _block

pytestmark = pytest.mark.gpu


def _forward(blk, x, dtype):
    blk.forward(x.to(dev()).to(dtype))
    return host(blk.operand_status).tolist()


def test_operands_report_what_is_not_finite():
    """operand_status: norm output, hidden activation, W1, W2."""
    blk, x, dy = _block(20, 64, 96, dtype=torch.float16)
    assert _forward(blk, x, torch.float16) == [0, 0, 0, 0]
    # an activation that float16 cannot hold
    blk.b1[5] = 1e5
    assert _forward(blk, x, torch.float16) == [0, 2, 0, 0]
    blk.b1[5] = 0.0
    blk.gamma[3] = float("nan")
    assert _forward(blk, x, torch.float16)[0] == 2
    blk.gamma[3] = 1.0
    assert _forward(blk, x, torch.float16) == [0, 0, 0, 0]  # no state is left over


def test_updated_weights_report_what_is_not_finite():
    blk, x, dy = _block(20, 64, 96, lr=1e-3)
    x, dy = x.to(dev()).bfloat16(), dy.to(dev()).bfloat16()
    blk.forward(x)
    blk.backward(x, dy)
    blk.update()
    assert host(blk.operand_status).tolist() == [0, 0, 0, 0]
    blk.gW2[7, 9] = float("inf")
    blk.update()
    assert host(blk.operand_status).tolist()[2:] == [0, 2]


def test_first_weights_report_what_is_not_finite():
    p = [torch.ones(s, device=dev()) for s in ((96, 64), (96,), (64, 96), (64,), (64,), (64,))]
    p[0][2, 3] = float("inf")
    blk = steps.ResidualMlp(*p, B=4)
    assert host(blk.operand_status).tolist()[2:] == [2, 0]


def test_updates_without_a_forward_pass_between_them():
    """Each update's 8-bit weights go by the weights' own maximum, not by an earlier one."""
    blk, x, dy = _block(20, 64, 96, lr=1e-3)
    x, dy = x.to(dev()).bfloat16(), dy.to(dev()).bfloat16()
    blk.forward(x)
    blk.backward(x, dy)
    ws = torch.empty(ops.dfp8_from_float_workspace_bytes(), dtype=torch.uint8, device=dev())
    for scale in (1.0, 2.0 ** -6, 2.0 ** -3):
        blk.W1.mul_(scale)
        blk.W2.mul_(scale)
        blk.update()
        for W, q, e in ((blk.W1, blk.W1_8, blk.e[2]), (blk.W2, blk.W2_8, blk.e[3])):
            out, eo = torch.empty_like(q), torch.zeros(1, dtype=torch.int32, device=dev())
            ops.dfp8_from_float(W, out, eo, workspace=ws)
            assert int(e) == int(eo) and torch.equal(q, out), scale
    blk.forward(x)  # (clears its own maxima only)
    top = host(blk.top).view("float32")
    assert abs(top[2] / float(blk.W1.abs().max()) - 1) < 1e-6 and top[0] > 0 and top[1] > 0


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("on_device", [False, True])
def test_refused_steps_are_not_counted(bits, on_device):
    z = lambda n: torch.zeros(n, device=dev())  # noqa: E731
    P = torch.ones(300, device=dev())
    opt = steps.AdamW.make([P], bits=bits, on_device=on_device)
    g = torch.full((300,), 0.5, device=dev())
    opt.step([g])
    w = P.clone()

    def counts():
        return opt.t, int(opt.step_dev) if on_device else None

    assert counts() == (1, 1 if on_device else None)
    eps, opt.eps = opt.eps, -1.0
    say("refused", bits, on_device)
    for stream in (None, torch.cuda.current_stream()):
        with pytest.raises(RuntimeError, match="eps"):
            opt.step([g], stream=stream)  # refused by the library
    opt.eps = eps
    with pytest.raises(ValueError):
        opt.step([z(299)])  # refused by the class
    with pytest.raises(TypeError):
        opt.step([g], grad_scale=torch.ones(1, device=dev(), dtype=torch.float64))  # and by the binding
    with pytest.raises(ValueError):
        opt.step([g], absmax_P=torch.zeros(2, dtype=torch.int32, device=dev()))
    assert counts() == (1, 1 if on_device else None) and torch.equal(P, w)
    opt.step([g])
    assert counts() == (2, 2 if on_device else None)
