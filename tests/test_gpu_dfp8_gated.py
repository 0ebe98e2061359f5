"""GPU: the gated layer on DFP-8 operands (dfp8_gated_fwd / _bwd) against the
oracle.

Tolerances.  The int32 sums are exact.  g and u carry half a step of float32
(2^-24) each for their conversion and the bias; 2^-20 of the magnitudes that
enter covers the activation's arithmetic as well (as in a Linear layer's
epilogue), and activations of 16-bit outputs may be evaluated to 2^-16 of their
argument.  With mg, mu the magnitudes behind g and u, and |act(g)| <= |g|, an
activation of slope at most 1.13 (gelu's largest) is off by at most slack * mg
in 16 half steps' room, so Y by slack * (mg |u| + |act(g)| mu) + the second
order slack^2 mg mu, and half a step of its type.  The gradients' products are
exact functions of the stored dZ8 and are compared bit for bit."""
import math

import numpy as np
import pytest
import torch

from gpu_helpers import dev, host, say, to_dev
from integer_only_nn_amd import ops
from oracle import floats as of
from test_gpu_dfp8_linear import SMALLEST, TYPES, _e, _half, _np, _round, _scaled, _slack, _typed, _ws

pytestmark = pytest.mark.gpu

# (B, IN, H): the way of the Linear layer's product of 2 H outputs, which is the gated one's
WAYS = {
    (1, 16, 1): "rows", (1, 4096, 300): "rows", (9, 129, 77): "rows", (33, 1000, 260): "rows", (64, 512, 130): "rows",
    (250, 784, 256): "rows", (200, 130, 40): "rows",
    (8, 17, 5000): "rows",
    (5, 8, 33): "narrow", (70, 3, 65): "narrow", (300, 15, 200): "narrow", (3, 1, 1): "narrow",
    (1001, 1023, 1025): "tiles", (700, 300, 500): "tiles", (300, 9001, 300): "tiles", (129, 20000, 40): "tiles",
    (2041, 2032, 1016): "tiles 128", (2048, 2048, 1024): "tiles 128", (2033, 2064, 1001): "tiles 128",
    (4096, 4096, 2048): "tiles 256", (4090, 2064, 2041): "tiles 256", (3901, 4080, 1929): "tiles 256",
}

# (B, IN, H) whose rows are not whole 16-byte pieces -> the tensors copied for larger tiles: forward, backward
COPIES = {
    (2043, 2027, 1011): ("XW", "ZXW"), (4090, 2063, 2041): ("XW", "ZXW"), (700, 4001, 2000): ("XW", "XW"),
    (1222, 2803, 533): ("", "ZXW"), (2048, 2032, 1017): ("", "Z"), (1470, 1249, 1592): ("", "X"), (4335, 823, 952): ("XW", "W"),
    (300, 4095, 8192): ("XW", ""), (8192, 1000, 2000): ("XW", "XW"), (2048, 1000, 1020): ("", ""), (1024, 2050, 2050): ("", ""),
}


def _case(B, IN, H, bias=True, seed=0):
    rng = np.random.default_rng(seed + 7 * B + 3 * IN + H)
    return dict(X=rng.integers(-128, 128, (B, IN)).astype(np.int8), W=rng.integers(-128, 128, (2 * H, IN)).astype(np.int8),
                eX=-6, eW=-round(math.log2(74 * math.sqrt(max(IN, 1)))),
                bias=rng.standard_normal(2 * H).astype(np.float32) if bias else None)


def _forward(d, kind, name, save_z=True, absmax=True, stream=None):
    (B, IN), H = d["X"].shape, d["W"].shape[0] // 2
    Y = torch.full((B, H), 3.0, dtype=TYPES[name], device=dev())
    Z = torch.full((B, 2 * H), 3.0, dtype=TYPES[name], device=dev()) if save_z else None
    m = torch.zeros(1, dtype=torch.int32, device=dev()) if absmax else None
    say("gated fwd", B, IN, H, kind, name)
    ops.dfp8_gated_fwd(to_dev(d["X"]), _e(d["eX"]), to_dev(d["W"]), _e(d["eW"]), Y,
                       bias=None if d["bias"] is None else to_dev(d["bias"]), act=kind, Z=Z, absmax_Y=m,
                       workspace=_ws(ops.dfp8_gated_fwd_workspace_bytes(B, IN, H)), stream=stream)
    return Y, Z, m


def _check_forward(d, kind, name, **kw):
    Y, Z, m = _forward(d, kind, name, **kw)
    H = d["W"].shape[0] // 2
    y, z = of.gated_fwd(d["X"], d["eX"], d["W"], d["eW"], d["bias"], kind)
    mag = np.abs(z if d["bias"] is None else z - d["bias"]) + (0 if d["bias"] is None else np.abs(d["bias"]))
    mg, mu = mag[:, :H], mag[:, H:]
    s = _slack(name)
    tol_y = s * (mg * np.abs(z[:, H:]) + np.abs(of.act(z[:, :H], kind)) * mu) + s * s * mg * mu
    bad = np.abs(_np(Y) - y) - tol_y - _half(name) * (np.abs(y) + tol_y) - SMALLEST[name]
    assert (bad <= 0).all(), f"Y off by {bad.max()} beyond the tolerance"
    if Z is not None:
        tol_z = 2.0 ** -20 * mag
        assert (np.abs(_np(Z) - z) <= tol_z + _half(name) * (np.abs(z) + tol_z) + SMALLEST[name]).all()
    if m is not None:
        got, top = float(host(m).view(np.float32)[0]), np.abs(y).max(initial=0.0)
        assert abs(got - top) <= tol_y.max(initial=0.0) + 2.0 ** -20 * top


@pytest.mark.parametrize("B,IN,H", list(WAYS))
@pytest.mark.parametrize("name", list(TYPES))
def test_forward(B, IN, H, name):
    small = B * IN * H < 1 << 25
    kinds = of.ACTIVATIONS if small else {"f32": ("relu",), "bf16": ("silu",), "f16": ("gelu_tanh",)}[name]
    for i, kind in enumerate(kinds):
        _check_forward(_case(B, IN, H, bias=i != 1), kind, name, save_z=i != 2, absmax=i != 3)


@pytest.mark.parametrize("B,IN,H", [s for s, c in COPIES.items() if c[0] and s[0] < 4096])
@pytest.mark.parametrize("name,kind", [("f32", "relu"), ("bf16", "silu"), ("f16", "gelu")])
def test_forward_of_copied_rows(B, IN, H, name, kind):
    _check_forward(_case(B, IN, H, bias=name != "f16"), kind, name, save_z=name != "bf16")


def test_forward_empty_sizes():
    _check_forward(_case(4, 0, 6), "gelu", "f32")  # IN = 0: z = bias
    for B, H in ((0, 6), (4, 0)):
        assert tuple(_forward(_case(B, 8, H), "silu", "f32")[0].shape) == (B, H)


def test_forward_of_the_largest_sums():
    IN = 131071
    d = dict(X=np.full((2, IN), -128, np.int8), W=np.full((6, IN), -128, np.int8), eX=-20, eW=-11, bias=None)
    v = np.float32(float(IN * 16384)) * np.float32(2.0 ** -31)
    assert (host(_forward(d, "none", "f32")[0]) == v * v).all()


def test_forward_not_finite_values_stay_in_their_place():
    d = _case(4, 32, 8)
    d["bias"][1], d["bias"][2], d["bias"][8 + 5] = np.inf, np.nan, np.nan
    for kind in of.ACTIVATIONS:
        Y = host(_forward(d, kind, "f32")[0])
        assert np.isinf(Y[:, 1]).all() and np.isnan(Y[:, [2, 5]]).all() and np.isfinite(np.delete(Y, (1, 2, 5), 1)).all()
        top = _forward(d, kind, "f32")[2]
        assert int(host(top)[0]) & 0x7fffffff > 0x7f800000  # a NaN counts above every number


@pytest.mark.parametrize("B,IN,H", [(70, 256, 256), (2041, 2032, 1016), (4090, 2064, 2041), (1001, 1023, 1025), (300, 9001, 300),
                                    (2043, 2027, 1011)])
def test_operands_that_start_anywhere(B, IN, H):
    d = _case(B, IN, H)
    want = _forward(d, "silu", "f16")[0]
    at = lambda a, off: torch.cat([torch.zeros(off, dtype=torch.int8), torch.from_numpy(a.reshape(-1))]).to(dev())[off:].view(a.shape)  # noqa: E731
    for ox, ow in ((1, 0), (0, 3), (8, 5)):
        say("offsets", ox, ow)
        Y = torch.zeros(B * H + 1, dtype=torch.float16, device=dev())[1:].view(B, H)
        ops.dfp8_gated_fwd(at(d["X"], ox), _e(d["eX"]), at(d["W"], ow), _e(d["eW"]), Y, bias=to_dev(d["bias"]), act="silu",
                           workspace=_ws(ops.dfp8_gated_fwd_workspace_bytes(B, IN, H)))
        assert torch.equal(Y, want)


def test_what_lies_behind_the_outputs_is_left():
    for B, IN, H in ((3, 64, 5), (65, 70, 33), (130, 2048, 70), (1030, 2048, 1029)):
        d = _case(B, IN, H)
        Y = torch.full((B * H + 64,), 5.0, dtype=torch.bfloat16, device=dev())
        Z = torch.full((2 * B * H + 64,), 5.0, dtype=torch.bfloat16, device=dev())
        ops.dfp8_gated_fwd(to_dev(d["X"]), _e(d["eX"]), to_dev(d["W"]), _e(d["eW"]), Y[:B * H].view(B, H), act="silu",
                           Z=Z[:2 * B * H].view(B, 2 * H), workspace=_ws(ops.dfp8_gated_fwd_workspace_bytes(B, IN, H)))
        assert (Y[B * H:] == 5).all() and (Z[2 * B * H:] == 5).all()


# ---- backward ----------------------------------------------------------------

def _backward(B, IN, H, kind, name, dY=None, Z=None, want=("dX", "G", "gb"), seed=0):
    rng = np.random.default_rng(seed + B + 5 * IN + 11 * H)
    d = _case(B, IN, H, seed=seed)
    dY = _round(0.1 * rng.standard_normal((B, H)) if dY is None else dY, name)
    Z = _round(2.0 * rng.standard_normal((B, 2 * H)) if Z is None else Z, name)
    full = lambda shape, t: torch.full(shape, 7.0, dtype=t, device=dev())  # noqa: E731
    out = {"dX": full((B, IN), TYPES[name]), "G": full((2 * H, IN), TYPES[name]), "gb": full((2 * H,), torch.float32)}
    out = {k: v if k in want else None for k, v in out.items()}
    dZ8, edZ, st = torch.full((B, 2 * H), 9, dtype=torch.int8, device=dev()), _e(99), _e(99)
    say("gated bwd", B, IN, H, kind, name)
    ops.dfp8_gated_bwd(_typed(dY, name), _typed(Z, name), kind, to_dev(d["X"]), _e(d["eX"]), to_dev(d["W"]), _e(d["eW"]),
                       dZ8, edZ, **out, status_out=st, workspace=_ws(ops.dfp8_gated_bwd_workspace_bytes(B, IN, H)))
    d.update(dY=dY, Z=Z, dZ8=host(dZ8), e=int(host(edZ)[0]), status=int(host(st)[0]),
             **{k: None if v is None else _np(v) for k, v in out.items()})
    return d


def _check_backward(d, kind, name):
    """err: float32's roundings of dY u act'(g) and dY act(g), the activation off
    by 2^-20 of its argument (its derivative by 2^-20), as in the forward; nothing
    where the error is exact before it is rounded."""
    H = d["dY"].shape[1]
    dz = of.gated_error(d["dY"], d["Z"], kind)
    dy, g, u = np.abs(d["dY"]), np.abs(d["Z"][:, :H]), np.abs(d["Z"][:, H:])
    exact = kind in ("none", "relu")
    err = 0.0 * dz if exact else 2.0 ** -20 * np.concatenate([dy * u, dy * g], 1)
    e = d["e"]
    assert d["status"] == 0
    top, slack = np.abs(dz).max(initial=0.0), err.max(initial=0.0)
    if top == 0:
        assert e == 0
    else:
        assert 64 * 2.0 ** e <= top + slack and top - slack < 128 * 2.0 ** e
    t = np.clip(np.ldexp(dz, -e), -128, 127)
    assert (np.abs(d["dZ8"] - t) <= 0.5 + np.ldexp(err, -e)).all()
    if exact:
        np.testing.assert_array_equal(d["dZ8"], of.dfp8(dz)[0])
    if d["dX"] is not None:
        np.testing.assert_array_equal(d["dX"], _scaled(of.product(d["dZ8"], d["W"].T), e + d["eW"], name))
    if d["G"] is not None:
        np.testing.assert_array_equal(d["G"], _scaled(of.product(d["dZ8"].T, d["X"].T), e + d["eX"], name))
    if d["gb"] is not None:
        tol = (dz.shape[0] + 8) * 2.0 ** -24 * np.abs(dz).sum(0) + err.sum(0) + 2.0 ** -149
        assert (np.abs(d["gb"] - dz.sum(0)) <= tol).all()


@pytest.mark.parametrize("B,IN,H", [(1, 1, 1), (1, 100, 64), (3, 5, 7), (1, 129, 300), (17, 300, 50), (64, 128, 32),
                                    (65, 127, 255), (130, 513, 129), (256, 784, 256), (9, 70, 9)])
@pytest.mark.parametrize("name", list(TYPES))
def test_backward(B, IN, H, name):
    for kind in of.ACTIVATIONS:
        _check_backward(_backward(B, IN, H, kind, name), kind, name)


@pytest.mark.parametrize("B,IN,H", [(513, 1281, 769), (4000, 70, 130), (8192, 64, 48), (2, 2048, 4096), (2051, 2320, 1040),
                                    (2040, 2032, 1016), (4096, 4096, 2048), (1040, 272, 1024)])
@pytest.mark.parametrize("name,kind", [("f32", "relu"), ("bf16", "silu"), ("f16", "gelu")])
def test_backward_larger(B, IN, H, name, kind):
    _check_backward(_backward(B, IN, H, kind, name), kind, name)


@pytest.mark.parametrize("B,IN,H", [s for s, c in COPIES.items() if c[1] and s[0] < 8192])
@pytest.mark.parametrize("name,kind", [("f32", "relu"), ("bf16", "silu"), ("f16", "gelu_tanh")])
def test_backward_of_copied_rows(B, IN, H, name, kind):
    _check_backward(_backward(B, IN, H, kind, name), kind, name)


@pytest.mark.parametrize("B,IN,H", [(2043, 2027, 1011), (2048, 2032, 1017), (4335, 823, 952)])
def test_copied_rows_one_gradient_and_any_workspace(B, IN, H):
    """dX or G alone; nothing depends on what the workspace held, and nothing behind it is written."""
    g = torch.Generator(device=dev()).manual_seed(5)
    ints = lambda *s: torch.randint(-128, 128, s, dtype=torch.int8, device=dev(), generator=g)  # noqa: E731
    X, W = ints(B, IN), ints(2 * H, IN)
    dY, Z = (torch.randn(B, n, device=dev(), generator=g).bfloat16() for n in (H, 2 * H))
    need = {"bwd": ops.dfp8_gated_bwd_workspace_bytes(B, IN, H), "fwd": ops.dfp8_gated_fwd_workspace_bytes(B, IN, H)}

    def run(names, byte):
        ws = torch.full((max(need.values()) + 64,), byte, dtype=torch.uint8, device=dev())
        out = {k: torch.full(s, 7.0, dtype=torch.bfloat16, device=dev()) for k, s in
               (("Y", (B, H)), ("dX", (B, IN)), ("G", (2 * H, IN))) if k in names}
        q, e = torch.empty(B, 2 * H, dtype=torch.int8, device=dev()), _e(0)
        say("copied rows", B, IN, H, names)
        if "Y" in names:
            ops.dfp8_gated_fwd(X, _e(-6), W, _e(-12), out["Y"], workspace=ws[:need["fwd"]])
            assert (ws[need["fwd"]:] == byte).all()
        ops.dfp8_gated_bwd(dY, Z, "silu", X, _e(-6), W, _e(-12), q, e, dX=out.get("dX"), G=out.get("G"), workspace=ws[:need["bwd"]])
        assert (ws[max(need.values()):] == byte).all()
        return out
    want = run(("Y", "dX", "G"), 0)
    for names, byte in ((("dX",), 0xff), (("G",), 0x7f), (("Y", "dX", "G"), 0x80)):
        for k, v in run(names, byte).items():
            assert torch.equal(v, want[k]), k


def test_backward_outputs_are_optional():
    whole = _backward(70, 40, 50, "silu", "bf16")
    for want in (("dX",), ("G",), ("gb",), ()):
        part = _backward(70, 40, 50, "silu", "bf16", want=want)
        np.testing.assert_array_equal(part["dZ8"], whole["dZ8"])
        for k in want:
            np.testing.assert_array_equal(part[k], whole[k])


def test_backward_empty_and_zero():
    d = _backward(0, 6, 5, "silu", "f32")
    assert d["e"] == 0 and d["status"] == 0 and not d["G"].any() and not d["gb"].any()
    d = _backward(4, 6, 0, "silu", "bf16")
    assert d["e"] == 0 and not d["dX"].any()
    d = _backward(4, 0, 5, "silu", "bf16")
    _check_backward({**d, "dX": None, "G": None}, "silu", "bf16")
    for kw in (dict(dY=np.zeros((9, 6))), dict(Z=-np.ones((9, 12)))):  # a ReLU that passes nothing
        d = _backward(9, 7, 6, "relu", "f16", **kw)
        assert d["e"] == 0 and not d["dZ8"].any() and not d["dX"].any() and not d["G"].any() and not d["gb"].any()


def test_backward_against_differences():
    """gb, the gradient of the sum of dY Y by the bias, against central
    differences of the float64 formula (third derivatives of these activations
    below 2: off by h^2 / 3 |dY u| and 1e-15 / h of cancellation)."""
    B, H, h = 5, 9, 2.0 ** -12
    for kind in ("none", "silu", "gelu", "gelu_tanh"):
        d = _backward(B, 4, H, kind, "f32")
        loss = lambda z: (d["dY"] * of.act(z[:, :H], kind) * z[:, H:]).sum()  # noqa: E731
        for o in range(2 * H):
            step = np.zeros((1, 2 * H))
            step[0, o] = h
            diff = (loss(d["Z"] + step) - loss(d["Z"] - step)) / (2 * h)
            scale = (np.abs(d["dY"]) * (1 + np.abs(d["Z"][:, :H])) * (1 + np.abs(d["Z"][:, H:]))).sum()
            assert abs(diff - d["gb"][o]) <= scale * (h * h + 2.0 ** -19)


def test_backward_reports_what_is_not_finite():
    for kind in ("relu", "silu"):
        Z = np.ones((3, 8))
        Z[1, 6] = np.nan
        assert _backward(3, 5, 4, kind, "f32", Z=Z)["status"] == 2
        # both float32, their product is not
        assert _backward(3, 5, 4, kind, "f32", dY=np.full((3, 4), 1e30), Z=np.full((3, 8), 1e30))["status"] == 2
        assert _backward(3, 5, 4, kind, "f32", dY=np.full((3, 4), 2.0 ** -130))["status"] == 1


def test_repeatable_and_on_another_stream():
    a, b = (_backward(1000, 300, 100, "silu", "bf16") for _ in range(2))
    for k in ("dZ8", "dX", "G", "gb"):
        np.testing.assert_array_equal(a[k], b[k])
    d = _case(300, 260, 135)
    want = _forward(d, "gelu", "bf16")[0].clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    got = _forward(d, "gelu", "bf16", stream=None)[0]
    assert torch.equal(got, want)
    X, W, b = to_dev(d["X"]), to_dev(d["W"]), to_dev(d["bias"])
    Y, eX, eW, w = torch.zeros_like(want), _e(d["eX"]), _e(d["eW"]), _ws(ops.dfp8_gated_fwd_workspace_bytes(300, 260, 135))
    s.wait_stream(torch.cuda.current_stream())
    ops.dfp8_gated_fwd(X, eX, W, eW, Y, bias=b, act="gelu", workspace=w, stream=s)
    s.synchronize()
    assert torch.equal(Y, want)


@pytest.mark.parametrize("B,IN,H", [(16, 300, 100), (2048, 2048, 1024), (300, 9001, 300), (2043, 2027, 1011)])
def test_captured_and_replayed(B, IN, H):
    g = torch.Generator(device=dev()).manual_seed(5)
    ints = lambda *s: torch.randint(-128, 128, s, device=dev(), generator=g, dtype=torch.int8)  # noqa: E731
    X, W, eX, eW = ints(B, IN), ints(2 * H, IN), _e(-6), _e(-12)
    new = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t, device=dev())  # noqa: E731
    Y, Z, dY, q, e = new(B, H), new(B, 2 * H), torch.randn(B, H, device=dev(), generator=g).bfloat16(), new(B, 2 * H, t=torch.int8), _e(0)
    dX, G, gb = new(B, IN), new(2 * H, IN), new(2 * H, t=torch.float32)
    ws = _ws(max(ops.dfp8_gated_fwd_workspace_bytes(B, IN, H), ops.dfp8_gated_bwd_workspace_bytes(B, IN, H)))

    def step():
        ops.dfp8_gated_fwd(X, eX, W, eW, Y, act="silu", Z=Z, workspace=ws)
        ops.dfp8_gated_bwd(dY, Z, "silu", X, eX, W, eW, q, e, dX=dX, G=G, gb=gb, workspace=ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(3):
        X.copy_(ints(B, IN))
        dY.copy_(torch.randn(B, H, device=dev(), generator=g))
        graph.replay()
        got = [t.clone() for t in (Y, Z, q, dX, G, gb)]
        torch.cuda.synchronize()
        step()
        assert all(torch.equal(a, b) for a, b in zip(got, (Y, Z, q, dX, G, gb)))
