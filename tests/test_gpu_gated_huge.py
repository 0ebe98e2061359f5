"""GPU: the gated layer and the norms around a block at sizes whose offsets pass
32 bits, or whose grids, one workgroup for each piece, would be too many."""
import pytest
import torch

from gpu_helpers import dev, say
from integer_only_nn_amd import ops

pytestmark = pytest.mark.gpu


def _e(v):
    return torch.tensor([v], dtype=torch.int32, device=dev())


def _ws(n):
    return torch.empty(n, dtype=torch.uint8, device=dev())


@pytest.mark.parametrize("H", [(1 << 26) + 3, 1 << 27])
def test_forward_of_one_row(H):
    IN = 16
    say("gated fwd", 1, IN, H)
    g = torch.Generator(device=dev()).manual_seed(1)
    X = torch.randint(-128, 128, (1, IN), dtype=torch.int8, device=dev(), generator=g)
    W = torch.randint(-128, 128, (2 * H, IN), dtype=torch.int8, device=dev(), generator=g)
    Y, Z = torch.full((1, H), 7.0, dtype=torch.bfloat16, device=dev()), torch.full((1, 2 * H), 7.0, dtype=torch.bfloat16, device=dev())
    assert ops.dfp8_gated_fwd_workspace_bytes(1, IN, H) == 0
    ops.dfp8_gated_fwd(X, _e(-3), W, _e(-4), Y, act="none", Z=Z)
    part = lambda a, b: torch.ldexp((W[a:b].int() * X.int()).sum(1, dtype=torch.int32).float(), _e(-7))  # noqa: E731
    for a in range(0, H, 1 << 25):
        b = min(H, a + (1 << 25))
        gate, up = part(a, b), part(H + a, H + b)
        assert torch.equal(Y[0, a:b], (gate * up).bfloat16()), a
        assert torch.equal(Z[0, a:b], gate.bfloat16()) and torch.equal(Z[0, H + a:H + b], up.bfloat16()), a


def test_layer_of_more_than_2_to_the_32_outputs():
    B, IN, H = (1 << 20) + 70, 16, 4112
    say("gated fwd, bwd", B, IN, H)
    g = torch.Generator(device=dev()).manual_seed(2)
    X = torch.randint(-128, 128, (B, IN), dtype=torch.int8, device=dev(), generator=g)
    W = torch.randint(-128, 128, (2 * H, IN), dtype=torch.int8, device=dev(), generator=g)
    Y, Z = torch.empty(B, H, dtype=torch.bfloat16, device=dev()), torch.empty(B, 2 * H, dtype=torch.bfloat16, device=dev())
    ops.dfp8_gated_fwd(X, _e(-6), W, _e(-9), Y, act="silu", Z=Z, workspace=_ws(ops.dfp8_gated_fwd_workspace_bytes(B, IN, H)))
    n, tail = 64, slice(B - 64, B)
    for rows in (slice(0, 64), tail):
        y, z = torch.empty(n, H, dtype=torch.bfloat16, device=dev()), torch.empty(n, 2 * H, dtype=torch.bfloat16, device=dev())
        ops.dfp8_gated_fwd(X[rows], _e(-6), W, _e(-9), y, act="silu", Z=z, workspace=_ws(ops.dfp8_gated_fwd_workspace_bytes(n, IN, H)))
        assert torch.equal(Y[rows], y) and torch.equal(Z[rows], z)
    # the errors of the last rows alone: everything else is 0
    Y.zero_()
    Y[tail] = torch.randn(n, H, device=dev(), generator=g).bfloat16()
    q, e, dX, gb = torch.empty(B, 2 * H, dtype=torch.int8, device=dev()), _e(9), torch.empty(B, IN, dtype=torch.bfloat16, device=dev()), torch.empty(2 * H, device=dev())
    ops.dfp8_gated_bwd(Y, Z, "silu", X, _e(-6), W, _e(-9), q, e, dX=dX, gb=gb, workspace=_ws(ops.dfp8_gated_bwd_workspace_bytes(B, IN, H)))
    q1, e1, dX1, gb1 = torch.empty(n, 2 * H, dtype=torch.int8, device=dev()), _e(9), torch.empty(n, IN, dtype=torch.bfloat16, device=dev()), torch.empty(2 * H, device=dev())
    ops.dfp8_gated_bwd(Y[tail], Z[tail], "silu", X[tail], _e(-6), W, _e(-9), q1, e1, dX=dX1, gb=gb1,
                       workspace=_ws(ops.dfp8_gated_bwd_workspace_bytes(n, IN, H)))
    assert torch.equal(e, e1) and torch.equal(q[tail], q1) and torch.equal(dX[tail], dX1)
    assert not q[:B - n].any() and not dX[:B - n].any()
    # the same 64 terms a column, summed in another order: 64 half steps of float32 of their magnitudes (below 6 each)
    assert float((gb - gb1).abs().max()) <= 64 * 2.0 ** -24 * 64 * 6 * 8


def test_errors_of_many_columns():
    H = 1 << 29
    say("gated bwd", 1, H)
    dY = torch.empty(1, H, dtype=torch.bfloat16, device=dev()).normal_()
    Z = torch.empty(1, 2 * H, dtype=torch.bfloat16, device=dev()).normal_()
    gb, q, e = torch.full((2 * H,), 7.0, device=dev()), torch.empty(1, 2 * H, dtype=torch.int8, device=dev()), _e(99)
    ops.dfp8_gated_bwd(dY, Z, "none", None, None, torch.empty(2 * H, 0, dtype=torch.int8, device=dev()), None, q, e, gb=gb,
                       workspace=_ws(ops.dfp8_gated_bwd_workspace_bytes(1, 0, H)))
    scale = torch.ldexp(torch.ones(1, device=dev()), -e)
    for a in range(0, H, 1 << 27):
        b = a + (1 << 27)
        for to, by in ((a, Z[0, H + a:H + b]), (H + a, Z[0, a:b])):
            want = dY[0, a:b].float() * by.float()
            assert torch.equal(gb[to:to + (1 << 27)], want), a
            assert torch.equal(q[0, to:to + (1 << 27)], (want * scale).round().clamp(-128, 127).to(torch.int8)), a


def test_norms_of_more_than_2_to_the_32_values():
    rows, cols, gate_rows = (1 << 19) + 65, 8200, 1 << 18
    say("residual norm", rows, cols)
    g = torch.Generator(device=dev()).manual_seed(3)
    new = lambda *s, t=torch.bfloat16: torch.empty(s, dtype=t, device=dev()).normal_(generator=g)  # noqa: E731
    a, x = new(rows, cols), new(rows, cols)
    ga, gy, gate = new(cols, t=torch.float32), new(cols, t=torch.float32), new(3, cols, t=torch.float32)
    y, n = torch.empty_like(a), torch.empty_like(a)
    ra, ry = torch.empty(rows, device=dev()), torch.empty(rows, device=dev())
    ops.ionn_residual_norm_fwd(a, x, y, n, gamma_a=ga, gate=gate, gate_rows=gate_rows, gamma_y=gy, rstd_a=ra, rstd_y=ry)
    tail = slice(2 * gate_rows, rows)  # the last gate's 65 rows
    k = rows - 2 * gate_rows
    y1, n1, ra1, ry1 = (torch.empty(s, dtype=t, device=dev()) for s, t in (((k, cols), torch.bfloat16),) * 2 + (((k,), torch.float32),) * 2)
    ops.ionn_residual_norm_fwd(a[tail], x[tail], y1, n1, gamma_a=ga, gate=gate[2], gamma_y=gy, rstd_a=ra1, rstd_y=ry1)
    assert torch.equal(y[tail], y1) and torch.equal(n[tail], n1) and torch.equal(ra[tail], ra1) and torch.equal(ry[tail], ry1)
    da, dx, dgate, dga = x, n, torch.empty_like(gate), torch.empty_like(ga)  # (their values are not needed any more)
    dy, dn = a.clone(), y.clone()
    ops.ionn_residual_norm_bwd(dy, dn, a, y, da, dx, gamma_a=ga, gate=gate, gate_rows=gate_rows, gamma_y=gy, rstd_a=ra, rstd_y=ry,
                               dgate=dgate, dgamma_a=dga, workspace=_ws(ops.ionn_residual_norm_bwd_workspace_bytes(rows, cols, gate_rows)))
    da1, dx1, dg1 = torch.empty_like(y1), torch.empty_like(y1), torch.empty_like(ga)
    ops.ionn_residual_norm_bwd(dy[tail], dn[tail], a[tail], y[tail], da1, dx1, gamma_a=ga, gate=gate[2], gamma_y=gy, rstd_a=ra1, rstd_y=ry1,
                               dgate=dg1, workspace=_ws(ops.ionn_residual_norm_bwd_workspace_bytes(k, cols)))
    assert torch.equal(da[tail], da1) and torch.equal(dx[tail], dx1)
    # the last gate's 65 terms a column, in another order (each below 6^3 times a gain of 6)
    assert float((dgate[2] - dg1).abs().max()) <= 65 * 2.0 ** -24 * 65 * 6 ** 4
    assert torch.isfinite(dga).all()
