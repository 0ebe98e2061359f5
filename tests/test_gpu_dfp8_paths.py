"""GPU: every way of cutting a DFP-8 product, by sizes that test_dfp8_paths.py
holds to it, so that a change of the rule cannot leave one of them untested.
Against the oracle with the tolerances of test_gpu_dfp8_linear.py; operands at
other addresses bit for bit against aligned ones (the sums are exact)."""
import pytest
import torch

from gpu_helpers import dev, say, to_dev
from integer_only_nn_amd import ops
from test_gpu_dfp8_linear import (_backward, _case, _check_backward, _check_forward, _e, _typed, _ws)

pytestmark = pytest.mark.gpu

# (B, IN, OUT) -> the ways of the forward product, dX and G
SIZES = {
    # tiles of 256: whole ones, cut rows and columns, reductions that end inside a step or are an odd number of them
    (4096, 4096, 4096): ("tiles 256", "tiles 256", "tiles 256"),
    (4090, 2064, 4080): ("tiles 256", "tiles 256", "tiles 256"),
    (3900, 3856, 4080): ("tiles 256", "tiles 256", "tiles 256"),
    (3901, 4096, 3856): ("tiles 256", "tiles 256", "tiles 256"),
    # tiles of 128, in one product or in all
    (2041, 2032, 2032): ("tiles 128", "tiles 128", "tiles 128"),
    (2040, 1040, 2032): ("tiles 128", "tiles", "tiles"),
    (2040, 2032, 1040): ("tiles", "tiles 128", "tiles"),
    (1040, 2032, 2032): ("tiles", "tiles", "tiles 128"),
    # tiles of 64, whole reductions and cut ones
    (1001, 1023, 2049): ("tiles", "tiles", "tiles"),
    (300, 9001, 600): ("tiles", "tiles", "tiles"),
    # a head of few outputs, few inputs: several tiles and steps
    (256, 128, 10): ("rows", "narrow", "narrow"),
    (300, 10, 200): ("narrow", "narrow", "narrow"),
    (1030, 784, 10): ("rows", "narrow", "narrow"),
    (515, 15, 15): ("narrow", "narrow", "narrow"),
    (15, 700, 333): ("rows", "tiles", "tiles"),
    (700, 7, 1): ("narrow", "narrow", "narrow"),
}


@pytest.mark.parametrize("B,IN,OUT", list(SIZES))
@pytest.mark.parametrize("name,kind", [("f32", "relu"), ("bf16", "gelu"), ("f16", "none")])
def test_forward(B, IN, OUT, name, kind):
    _check_forward(_case(B, IN, OUT, name, bias=name != "f16", residual=name != "f32"), kind, name, save_z=name != "bf16")


@pytest.mark.parametrize("B,IN,OUT", list(SIZES))
@pytest.mark.parametrize("name,kind", [("f32", "none"), ("bf16", "silu"), ("f16", "relu")])
def test_backward(B, IN, OUT, name, kind):
    _check_backward(_backward(B, IN, OUT, kind, name), kind, name)


def _at(a, off):
    """The int8 array `off` bytes into its storage."""
    flat = torch.zeros(a.numel() + off, dtype=torch.int8, device=dev())
    flat[off:] = a.reshape(-1)
    return flat[off:].view(a.shape)


# X, W, dZ8 off 16 bytes, in turn and together: each gradient takes its own way
OFFSETS = [(1, 0, 0), (0, 3, 0), (0, 0, 8), (5, 7, 9)]


@pytest.mark.parametrize("B,IN,OUT", [(2041, 2032, 2032), (2040, 2032, 1040), (4090, 2064, 4080), (1001, 1023, 2049), (1030, 784, 10)])
def test_operands_that_start_anywhere(B, IN, OUT):
    d = _case(B, IN, OUT, "bf16")
    X, W, b, R = to_dev(d["X"]), to_dev(d["W"]), to_dev(d["bias"]), _typed(d["R"], "bf16")
    g = torch.Generator(device=dev()).manual_seed(2)
    dY = torch.randn(B, OUT, device=dev(), generator=g).bfloat16()
    ex, ew = _e(d["eX"]), _e(d["eW"])

    def fwd(x, w):
        Y = torch.full((B, OUT), 7.0, dtype=torch.bfloat16, device=dev())
        ops.dfp8_linear_fwd(x, ex, w, ew, Y, bias=b, residual=R, workspace=_ws(ops.dfp8_linear_fwd_workspace_bytes(B, IN, OUT)))
        return Y

    def bwd(x, w, q):
        dX, G, gb = (torch.full(s, 7.0, dtype=t, device=dev()) for s, t in
                     (((B, IN), torch.bfloat16), ((OUT, IN), torch.bfloat16), ((OUT,), torch.float32)))
        ops.dfp8_linear_bwd(dY, None, "none", x, ex, w, ew, q, _e(0), dX=dX, G=G, gb=gb,
                            workspace=_ws(ops.dfp8_linear_bwd_workspace_bytes(B, IN, OUT)))
        return [q, dX, G, gb]

    q = torch.empty(B, OUT, dtype=torch.int8, device=dev())
    y, want = fwd(X, W), bwd(X, W, q)
    for ox, ow, oq in OFFSETS:
        say("offsets", ox, ow, oq)
        x, w = _at(X, ox), _at(W, ow)
        assert torch.equal(fwd(x, w), y)
        for a, c in zip(bwd(x, w, _at(torch.zeros_like(q), oq)), want):
            assert torch.equal(a, c)
