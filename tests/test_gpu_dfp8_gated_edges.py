"""GPU: the gated layer where a call's edges lie: errors next to a power of two,
outputs of more tiles of 64 than a grid has, calls for the error alone, and what
lies behind a backward pass's workspace."""
import numpy as np
import pytest
import torch

from gpu_helpers import dev, host, say
from integer_only_nn_amd import ops
from oracle import floats as of
from test_gpu_dfp8_gated import COPIES, _backward
from test_gpu_dfp8_linear import TYPES, _e, _np, _typed, _ws

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["none", "relu"])
@pytest.mark.parametrize("scale", [1.0, 2.0 ** -20, 2.0 ** 60, 2.0 ** -100])
@pytest.mark.parametrize("half", ["gate", "up"])
def test_largest_error_next_to_a_power_of_two(kind, scale, half):
    """(1 + 2^-23) (2 - 2^-22) = 2 - 2^-45, which float32 rounds to 2: the exponent
    is that of the product itself (errors behind none and relu are float64)."""
    rng = np.random.default_rng(3)
    for B, H, sign in ((1, 1, 1.0), (7, 33, -1.0), (70, 1030, 1.0)):
        dY, Z = scale * rng.uniform(-1, 1, (B, H)), rng.uniform(0.1, 1, (B, 2 * H))
        dY, Z = dY.astype(np.float32).astype(np.float64), Z.astype(np.float32).astype(np.float64)
        r, c = B // 2, H // 3
        dY[r, c] = sign * scale * (1 + 2.0 ** -23)
        # u behind the gate's error, g behind the up half's
        Z[r, c], Z[r, H + c] = (1.0, 2 - 2.0 ** -22) if half == "gate" else (2 - 2.0 ** -22, 1.0)
        dz = of.gated_error(dY, Z, kind)
        assert np.abs(dz).max() == scale * (2 - 2.0 ** -45)
        q, e, st = torch.empty(B, 2 * H, dtype=torch.int8, device=dev()), _e(99), _e(99)
        say("gated bwd next to a power of two", B, H, kind, scale, half)
        ops.dfp8_gated_bwd(_typed(dY, "f32"), _typed(Z, "f32"), kind, torch.empty(B, 0, dtype=torch.int8, device=dev()), None,
                           None, None, q, e, status_out=st, workspace=_ws(ops.dfp8_gated_bwd_workspace_bytes(B, 0, H)))
        want, exponent = of.dfp8(dz)
        assert int(host(e)[0]) == exponent and int(host(st)[0]) == 0
        np.testing.assert_array_equal(host(q), want)


def test_forward_of_more_outputs_than_tiles_of_64():
    """2^24 tiles of 64 x 32 outputs and more, which larger tiles take."""
    B, IN, H = (1 << 20) + 70, 512, 1 << 15
    assert ops.dfp8_linear_path("fwd", B, IN, 2 * H) == "tiles 128"
    say("gated fwd", B, IN, H)
    g = torch.Generator(device=dev()).manual_seed(2)
    X = torch.randint(-128, 128, (B, IN), dtype=torch.int8, device=dev(), generator=g)
    W = torch.randint(-128, 128, (2 * H, IN), dtype=torch.int8, device=dev(), generator=g)
    Y = torch.empty(B, H, dtype=torch.bfloat16, device=dev())
    ops.dfp8_gated_fwd(X, _e(-6), W, _e(-11), Y, act="silu", workspace=_ws(ops.dfp8_gated_fwd_workspace_bytes(B, IN, H)))
    for first in (0, 12345, B // 2, B - 64):
        rows = slice(first, first + 64)
        y = torch.empty(64, H, dtype=torch.bfloat16, device=dev())
        ops.dfp8_gated_fwd(X[rows], _e(-6), W, _e(-11), y, act="silu", workspace=_ws(ops.dfp8_gated_fwd_workspace_bytes(64, IN, H)))
        assert torch.equal(Y[rows], y), first


@pytest.mark.parametrize("name,kind", [("f32", "relu"), ("bf16", "silu")])
def test_the_error_alone(name, kind):
    """Without dX and G neither X nor W is read, in the gated layer and in the Linear layer."""
    B, H = 70, 50
    whole = _backward(B, 40, H, kind, name)
    dY, Z = _typed(whole["dY"], name), _typed(whole["Z"], name)
    q, e, gb = torch.empty(B, 2 * H, dtype=torch.int8, device=dev()), _e(99), torch.empty(2 * H, device=dev())
    ops.dfp8_gated_bwd(dY, Z, kind, None, None, None, None, q, e, gb=gb, workspace=_ws(ops.dfp8_gated_bwd_workspace_bytes(B, 0, H)))
    np.testing.assert_array_equal(host(q), whole["dZ8"])
    np.testing.assert_array_equal(_np(gb), whole["gb"])
    assert int(host(e)[0]) == whole["e"]
    z = Z[:, :H].contiguous()
    ws = _ws(ops.dfp8_linear_bwd_workspace_bytes(B, 40, H))
    got = []
    for X in (None, torch.ones(B, 40, dtype=torch.int8, device=dev())):
        q, e, gb = torch.empty(B, H, dtype=torch.int8, device=dev()), _e(99), torch.empty(H, device=dev())
        ops.dfp8_linear_bwd(dY, z, kind, X, _e(0), None, None, q, e, gb=gb, workspace=ws)
        got.append((q, e, gb))
    assert all(torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("B,IN,H", [s for s, c in COPIES.items() if c[1]] + [(513, 1281, 769), (4000, 70, 130), (40, 9001, 300)])
def test_backward_keeps_to_its_workspace(B, IN, H):
    g = torch.Generator(device=dev()).manual_seed(5)
    ints = lambda *s: torch.randint(-128, 128, s, dtype=torch.int8, device=dev(), generator=g)  # noqa: E731
    X, W = ints(B, IN), ints(2 * H, IN)
    need = ops.dfp8_gated_bwd_workspace_bytes(B, IN, H)
    ws = torch.full((need + (1 << 20),), 0x5a, dtype=torch.uint8, device=dev())
    for name, kind in (("f32", "none"), ("bf16", "silu")):
        dY, Z = (torch.randn(B, n, device=dev(), generator=g).to(TYPES[name]) for n in (H, 2 * H))
        new = lambda *s, t=TYPES[name]: torch.empty(s, dtype=t, device=dev())  # noqa: E731
        say("gated bwd", B, IN, H, name)
        ops.dfp8_gated_bwd(dY, Z, kind, X, _e(-6), W, _e(-12), new(B, 2 * H, t=torch.int8), _e(0), dX=new(B, IN), G=new(2 * H, IN),
                           gb=new(2 * H, t=torch.float32), workspace=ws[:need])
        assert (ws[need:] == 0x5a).all()
