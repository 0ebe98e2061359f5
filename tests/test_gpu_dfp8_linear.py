"""GPU: the Linear layer on DFP-8 operands (dfp8_linear_fwd / _bwd) and the
conversion that feeds it (dfp8_from_float) against the oracle.

Tolerances.  The int32 sum is exact; one half step of float32 (2^-24) each
for its conversion, the bias, the activation's arithmetic and the residual:
2^-20 of the magnitudes that enter covers 16 of them.  Activations of 16-bit
outputs may be evaluated to 2^-16 of their argument.  The store adds half a
step of the output's type (and of its smallest value).  The gradients'
products are exact functions of the stored dZ8, so they are compared bit for
bit."""
import math

import numpy as np
import pytest
import torch

from gpu_helpers import dev, host, say, to_dev
from integer_only_nn_amd import ops
from oracle import floats as of

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SMALLEST = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}


def _e(v):
    return torch.tensor([int(v)], dtype=torch.int32, device=dev())


def _np(t):
    return host(t.double() if t.is_floating_point() else t)


def _ws(nbytes):
    return torch.empty(nbytes, dtype=torch.uint8, device=dev())


def _round(x, name):
    """x as the values of type `name` (float64)."""
    return torch.from_numpy(np.ascontiguousarray(x)).float().to(TYPES[name]).double().numpy()


def _half(name):
    return torch.finfo(TYPES[name]).eps / 2


def _slack(name):
    return 2.0 ** -20 if name == "f32" else 2.0 ** -16


def _case(B, IN, OUT, name, bias=True, residual=True, seed=0):
    rng = np.random.default_rng(seed + 7 * B + 3 * IN + OUT)
    d = dict(X=rng.integers(-128, 128, (B, IN)).astype(np.int8), W=rng.integers(-128, 128, (OUT, IN)).astype(np.int8),
             eX=-6, eW=-round(math.log2(74 * math.sqrt(max(IN, 1)))),
             bias=rng.standard_normal(OUT).astype(np.float32) if bias else None,
             R=_round(rng.standard_normal((B, OUT)), name) if residual else None)
    return d


def _typed(x, name):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).to(dev()).to(TYPES[name])


def _forward(d, kind, name, save_z=True, absmax=True, inplace=False, workspace=None):
    B, IN = d["X"].shape
    OUT = d["W"].shape[0]
    R = _typed(d["R"], name)
    Y = R if inplace else torch.full((B, OUT), 3.0, dtype=TYPES[name], device=dev())
    Z = torch.full((B, OUT), 3.0, dtype=TYPES[name], device=dev()) if save_z else None
    m = torch.zeros(1, dtype=torch.int32, device=dev()) if absmax else None
    say("fwd", B, IN, OUT, kind, name)
    ops.dfp8_linear_fwd(to_dev(d["X"]), _e(d["eX"]), to_dev(d["W"]), _e(d["eW"]), Y,
                        bias=None if d["bias"] is None else to_dev(d["bias"]), act=kind, residual=R, Z=Z, absmax_Y=m,
                        workspace=_ws(ops.dfp8_linear_fwd_workspace_bytes(B, IN, OUT)))
    return Y, Z, m


def _check_forward(d, kind, name, **kw):
    Y, Z, m = _forward(d, kind, name, **kw)
    y, z = of.linear_fwd(d["X"], d["eX"], d["W"], d["eW"], d["bias"], kind, d["R"])
    s, _ = of.linear_fwd(d["X"], d["eX"], d["W"], d["eW"], None, "none", None)
    mag = np.abs(s) + (0 if d["bias"] is None else np.abs(d["bias"]))
    tol_z = 2.0 ** -20 * mag
    tol_y = _slack(name) * (mag + (0 if d["R"] is None else np.abs(d["R"])))
    bad = np.abs(_np(Y) - y) - tol_y - _half(name) * (np.abs(y) + tol_y) - SMALLEST[name]
    assert (bad <= 0).all(), f"Y off by {bad.max()} beyond the tolerance"
    if Z is not None:
        assert (np.abs(_np(Z) - z) <= tol_z + _half(name) * (np.abs(z) + tol_z) + SMALLEST[name]).all()
    if m is not None:
        got = float(host(m).view(np.float32)[0])
        top = np.abs(y).max(initial=0.0)
        assert abs(got - top) <= (tol_y.max(initial=0.0) + 2.0 ** -20 * top)


SIZES = [(1, 1, 1), (1, 100, 64), (3, 5, 7), (1, 129, 300), (16, 64, 33), (17, 300, 100), (64, 128, 64), (65, 127, 255),
         (130, 513, 129), (256, 784, 256)]


@pytest.mark.parametrize("B,IN,OUT", SIZES)
@pytest.mark.parametrize("name", list(TYPES))
def test_forward(B, IN, OUT, name):
    for i, kind in enumerate(of.ACTIVATIONS):
        _check_forward(_case(B, IN, OUT, name, bias=i != 1, residual=i % 2 == 0), kind, name, save_z=i != 2,
                       absmax=i != 3)


# whole tiles of 256, their edges, few rows against many columns, few tiles over a long reduction
@pytest.mark.parametrize("B,IN,OUT", [(512, 512, 768), (256, 4096, 256), (1000, 1023, 1025), (513, 1280, 769),
                                      (1024, 272, 1040), (2, 4096, 4096), (8, 1000, 2049), (33, 2048, 1024),
                                      (64, 8192, 64), (5, 20000, 40), (4096, 64, 96),
                                      # many whole and cut tiles of 256, reductions that end inside a step
                                      (2048, 512, 2304), (2100, 272, 2064), (2060, 400, 2321), (2049, 1168, 2050)])
@pytest.mark.parametrize("name,kind", [("f32", "relu"), ("bf16", "gelu"), ("f16", "silu")])
def test_forward_larger(B, IN, OUT, name, kind):
    _check_forward(_case(B, IN, OUT, name, bias=name != "f16", residual=name != "f32"), kind, name)


@pytest.mark.parametrize("B,IN,OUT", [
    # reductions that end in each of a wavefront's trips and inside a piece
    (16, 16, 16), (17, 17, 15), (1, 63, 33), (5, 65, 47), (16, 1023, 300), (20, 1025, 100), (1, 2047, 70), (15, 2049, 31),
    (3, 3071, 64), (9, 3100, 50), (2, 16384, 20), (16, 16383, 300), (4, 16385, 50),
    # groups of rows and outputs, whole and cut, around one workgroup per compute unit
    (256, 784, 256), (250, 785, 250), (257, 256, 255), (40, 520, 2100), (129, 1030, 1025), (130, 4097, 1000),
    (513, 1024, 1000), (500, 511, 1024), (500, 513, 1030), (70, 8192, 3000), (65, 8193, 3000),
    # few rows, many outputs
    (1, 48, 8200), (8, 100, 9001), (9, 100, 9001), (16, 2050, 8300), (17, 300, 12000), (32, 1100, 16384), (31, 70, 16385),
    # tiles of 64 cut along the reduction
    (33, 16500, 70), (300, 9001, 600), (600, 130, 900),
    # tiles of 128, whole and cut, reductions that end inside a step
    (2040, 1040, 2032), (2047, 2064, 1936), (4090, 1296, 4080), (2048, 1024, 2048)])
@pytest.mark.parametrize("name,kind", [("f32", "gelu_tanh"), ("bf16", "silu"), ("f16", "relu")])
def test_forward_ways_of_cutting(B, IN, OUT, name, kind):
    _check_forward(_case(B, IN, OUT, name, bias=name != "bf16", residual=name != "f16"), kind, name)


def test_forward_longest_reduction():
    """The largest sum that fits int32: IN = 131071 products of -128 * -128."""
    IN = 131071
    d = dict(X=np.full((2, IN), -128, np.int8), W=np.full((3, IN), -128, np.int8), eX=-20, eW=-11, bias=None, R=None)
    Y, _, _ = _forward(d, "none", "f32")
    want = np.float32(float(IN * 16384)) * np.float32(2.0 ** -31)
    assert (host(Y) == want).all()


def test_forward_empty_sizes():
    d = _case(4, 0, 6, "f32")
    _check_forward(d, "gelu", "f32")  # IN = 0: z = bias
    for B, OUT in ((0, 6), (4, 0)):
        Y, _, _ = _forward(_case(B, 8, OUT, "f32"), "gelu", "f32")
        assert tuple(Y.shape) == (B, OUT)


def test_forward_into_its_residual():
    for B, IN, OUT in ((20, 70, 90), (256, 512, 512), (3, 512, 512)):
        _check_forward(_case(B, IN, OUT, "bf16"), "gelu", "bf16", inplace=True)


def test_forward_extreme_exponents_and_values():
    # exponents at the ends of their range: the result leaves float32's range
    # upwards (infinity) and downwards (0), as the definition's would
    X, W = np.full((2, 64), 127, np.int8), np.full((2, 64), 127, np.int8)
    for eX, eW, want in ((127, 127, np.inf), (-128, -128, 0.0)):
        Y, _, _ = _forward(dict(X=X, W=W, eX=eX, eW=eW, bias=None, R=None), "none", "f32")
        assert (host(Y) == want).all()
    # infinities and NaN in the bias and the residual stay in their column / element
    d = _case(4, 32, 8, "f32")
    d["bias"][1], d["bias"][2], d["bias"][3] = np.inf, -np.inf, np.nan
    d["R"][0, 5] = np.nan
    for kind in of.ACTIVATIONS:
        Y = host(_forward(d, kind, "f32")[0])
        assert (Y[:, 1] == np.inf).all() and np.isnan(Y[:, 3]).all()
        assert (Y[:, 2] == -np.inf).all() if kind == "none" else (np.abs(Y[:, 2] - d["R"][:, 2]) < 1e-6).all()
        assert np.isnan(Y[0, 5]) and np.isfinite(np.delete(Y, (1, 2, 3, 5), 1)).all()


def test_unaligned_tensors():
    """Mantissas and outputs that start anywhere."""
    B, IN, OUT = 70, 256, 256
    d = _case(B, IN, OUT, "f16")
    for off in (1, 3, 8):
        say("offset", off)
        pad = lambda a: torch.cat([torch.zeros(off, dtype=torch.int8), torch.from_numpy(a.reshape(-1))]).to(dev())  # noqa: E731
        X, W = pad(d["X"])[off:].view(B, IN), pad(d["W"])[off:].view(OUT, IN)
        Y = torch.zeros(B * OUT + off, dtype=torch.float16, device=dev())[off:].view(B, OUT)
        ops.dfp8_linear_fwd(X, _e(d["eX"]), W, _e(d["eW"]), Y, bias=to_dev(d["bias"]), residual=_typed(d["R"], "f16"),
                            workspace=_ws(ops.dfp8_linear_fwd_workspace_bytes(B, IN, OUT)))
        want = _forward(d, "none", "f16")[0]
        assert torch.equal(Y, want)


# ---- backward ----------------------------------------------------------------

def _scaled(s, e, name):
    """T(fl(s) 2^e) for exact sums s."""
    with np.errstate(over="ignore"):
        return _round(np.ldexp(s.astype(np.float32), e), name)


def _backward(B, IN, OUT, kind, name, dY=None, Z=None, want=("dX", "G", "gb"), seed=0):
    rng = np.random.default_rng(seed + B + 5 * IN + 11 * OUT)
    d = _case(B, IN, OUT, name, seed=seed)
    dY = _round(0.1 * rng.standard_normal((B, OUT)) if dY is None else dY, name)
    Z = _round(2.0 * rng.standard_normal((B, OUT)) if Z is None else Z, name)
    out = {"dX": torch.full((B, IN), 7.0, dtype=TYPES[name], device=dev()) if "dX" in want else None,
           "G": torch.full((OUT, IN), 7.0, dtype=TYPES[name], device=dev()) if "G" in want else None,
           "gb": torch.full((OUT,), 7.0, device=dev()) if "gb" in want else None}
    dZ8, edZ, st = torch.full((B, OUT), 9, dtype=torch.int8, device=dev()), _e(99), _e(99)
    say("bwd", B, IN, OUT, kind, name)
    ops.dfp8_linear_bwd(_typed(dY, name), None if kind == "none" else _typed(Z, name), kind, to_dev(d["X"]),
                        _e(d["eX"]), to_dev(d["W"]), _e(d["eW"]), dZ8, edZ, **out, status_out=st,
                        workspace=_ws(ops.dfp8_linear_bwd_workspace_bytes(B, IN, OUT)))
    d.update(dY=dY, Z=Z, dZ8=host(dZ8), e=int(host(edZ)[0]), status=int(host(st)[0]),
             **{k: None if v is None else _np(v) for k, v in out.items()})
    return d


def _check_backward(d, kind, name):
    dz = d["dY"] * of.act_grad(d["Z"], kind)
    err = 0.0 if kind in ("none", "relu") else _slack(name) * np.abs(d["dY"])
    top, e = np.abs(dz).max(initial=0.0), d["e"]
    slack = np.max(err, initial=0.0)
    assert d["status"] == 0
    if top == 0:
        assert e == 0
    else:
        assert 64 * 2.0 ** e <= top + slack and top - slack < 128 * 2.0 ** e
    # rounded to the nearest mantissa (or the largest one)
    t = np.clip(np.ldexp(dz, -e), -128, 127)
    assert (np.abs(d["dZ8"] - t) <= 0.5 + np.ldexp(err, -e)).all()
    if kind in ("none", "relu"):
        np.testing.assert_array_equal(d["dZ8"], of.dfp8(dz)[0])
    if d["dX"] is not None:
        np.testing.assert_array_equal(d["dX"], _scaled(of.product(d["dZ8"], d["W"].T), e + d["eW"], name))
    if d["G"] is not None:
        np.testing.assert_array_equal(d["G"], _scaled(of.product(d["dZ8"].T, d["X"].T), e + d["eX"], name))
    if d["gb"] is not None:
        B = dz.shape[0]
        tol = (B + 8) * 2.0 ** -24 * np.abs(dz).sum(0) + np.sum(np.broadcast_to(err, dz.shape), 0) + 2.0 ** -149
        assert (np.abs(d["gb"] - dz.sum(0)) <= tol).all()


@pytest.mark.parametrize("B,IN,OUT", SIZES)
@pytest.mark.parametrize("name", list(TYPES))
def test_backward(B, IN, OUT, name):
    for kind in of.ACTIVATIONS:
        _check_backward(_backward(B, IN, OUT, kind, name), kind, name)


@pytest.mark.parametrize("B,IN,OUT", [(512, 768, 512), (256, 256, 256), (1000, 1023, 513), (513, 1281, 769),
                                      (1040, 272, 1024), (4000, 70, 130), (8192, 64, 48), (2, 2048, 4096),
                                      (64, 512, 8192), (768, 512, 1536), (2048, 2304, 2048), (2060, 2064, 2320),
                                      (2051, 2320, 2080), (2305, 2048, 272)])
@pytest.mark.parametrize("name,kind", [("f32", "relu"), ("bf16", "gelu"), ("f16", "silu")])
def test_backward_larger(B, IN, OUT, name, kind):
    _check_backward(_backward(B, IN, OUT, kind, name), kind, name)


@pytest.mark.parametrize("B,IN,OUT", [(2040, 2032, 1040), (517, 4080, 4064), (1029, 4080, 4064), (2048, 2048, 1024)])
@pytest.mark.parametrize("name,kind", [("f32", "none"), ("bf16", "relu"), ("f16", "gelu")])
def test_backward_in_tiles_of_128(B, IN, OUT, name, kind):
    """Both gradients, one of them, cut tiles and a batch that ends inside a step."""
    _check_backward(_backward(B, IN, OUT, kind, name), kind, name)


def test_backward_outputs_are_optional():
    whole = _backward(70, 40, 50, "gelu", "bf16")
    for want in (("dX",), ("G",), ("gb",), ()):
        part = _backward(70, 40, 50, "gelu", "bf16", want=want)
        np.testing.assert_array_equal(part["dZ8"], whole["dZ8"])
        for k in want:
            np.testing.assert_array_equal(part[k], whole[k])


def test_backward_empty_and_zero():
    d = _backward(0, 6, 5, "gelu", "f32")
    assert d["e"] == 0 and d["status"] == 0 and not d["G"].any() and not d["gb"].any()
    d = _backward(4, 6, 0, "gelu", "bf16")
    assert d["e"] == 0 and not d["dX"].any()
    d = _backward(4, 0, 5, "gelu", "bf16")
    _check_backward({**d, "dX": None, "G": None}, "gelu", "bf16")
    # an error that is zero everywhere, and behind a ReLU that passes nothing
    for kw in (dict(dY=np.zeros((9, 6))), dict(Z=-np.ones((9, 6)))):
        d = _backward(9, 7, 6, "relu", "f16", **kw)
        assert d["e"] == 0 and not d["dZ8"].any() and not d["dX"].any() and not d["G"].any() and not d["gb"].any()


def test_backward_saturated_activations():
    """Arguments far out, infinities among them: the derivatives' limits."""
    z = np.array([[-1e4, -60.0, -31.0, 31.0, 60.0, 1e4, np.inf, -np.inf, -0.0, 0.0]])
    limit = {"relu": [0, 0, 0, 1, 1, 1, 1, 0, 0, 0], "none": [1] * 10}
    for kind in of.ACTIVATIONS:
        want = np.array([limit.get(kind, [0, 0, 0, 1, 1, 1, 1, 0, 0.5, 0.5])])
        d = _backward(1, 4, 10, kind, "f32", dY=np.ones((1, 10)), Z=z)
        np.testing.assert_array_equal(np.ldexp(d["dZ8"].astype(float), d["e"]), want)


def test_backward_reports_what_is_not_finite():
    dY = np.ones((3, 4))
    dY[1, 2] = np.nan
    assert _backward(3, 5, 4, "relu", "f32", dY=dY)["status"] == 2
    # a magnitude below 2^-122: the exponent leaves its eight bits
    assert _backward(3, 5, 4, "none", "f32", dY=np.full((3, 4), 2.0 ** -130))["status"] == 1


def test_repeatable():
    a, b = (_backward(1000, 300, 200, "gelu", "bf16") for _ in range(2))
    for k in ("dZ8", "dX", "G", "gb"):
        np.testing.assert_array_equal(a[k], b[k])


# ---- conversion --------------------------------------------------------------

@pytest.mark.parametrize("n", [1, 7, 8, 1000, 65537, 1 << 20])
@pytest.mark.parametrize("name", list(TYPES))
def test_from_float(n, name):
    rng = np.random.default_rng(n)
    for scale in (1.0, 3e-3, 1e4 if name == "f16" else 1e30):
        x = _round(rng.standard_normal(n) * scale, name)
        I, e = of.dfp8(x)
        for given in (False, True):
            out, eo, st = torch.full((n,), 9, dtype=torch.int8, device=dev()), _e(99), _e(99)
            m = torch.from_numpy(np.array([np.abs(x).max()], np.float32).view(np.int32)).to(dev()) if given else None
            ops.dfp8_from_float(_typed(x, name), out, eo, absmax=m,
                                workspace=None if given else _ws(ops.dfp8_from_float_workspace_bytes()), status_out=st)
            assert (int(host(eo)[0]), int(host(st)[0])) == (e, 0)
            np.testing.assert_array_equal(host(out), I)


def test_from_float_ties_and_status():
    w = _ws(ops.dfp8_from_float_workspace_bytes())
    x = np.array([64.0, 0.5, 1.5, 2.5, -0.5, -1.5, 63.5, -64.0], np.float32)
    out, e, st = torch.empty(8, dtype=torch.int8, device=dev()), _e(0), _e(0)
    ops.dfp8_from_float(to_dev(x), out, e, workspace=w, status_out=st)
    assert host(out).tolist() == [64, 0, 2, 2, 0, -2, 64, -64] and int(host(e)[0]) == 0
    for v, want in ((np.nan, 2), (np.inf, 2), (2.0 ** -140, 1), (1.0, 0)):
        ops.dfp8_from_float(to_dev(np.array([v, 0.0], np.float32)), out[:2], e, workspace=w, status_out=st)
        assert int(host(st)[0]) == want


def test_forward_and_backward_on_another_stream():
    s = torch.cuda.Stream()
    d = _case(300, 260, 270, "bf16")
    want = _forward(d, "gelu", "bf16")[0].clone()
    X, W, b, R = to_dev(d["X"]), to_dev(d["W"]), to_dev(d["bias"]), _typed(d["R"], "bf16")
    Y, eX, eW = torch.zeros_like(R), _e(d["eX"]), _e(d["eW"])
    w = _ws(ops.dfp8_linear_fwd_workspace_bytes(300, 260, 270))
    s.wait_stream(torch.cuda.current_stream())
    ops.dfp8_linear_fwd(X, eX, W, eW, Y, bias=b, act="gelu", residual=R, workspace=w, stream=s)
    s.synchronize()
    assert torch.equal(Y, want)
