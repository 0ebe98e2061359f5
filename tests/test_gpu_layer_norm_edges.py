"""GPU: layer norm's gradient where a row's end cuts a thread's columns and
the mean times the reciprocal deviation leaves float32: the columns past the
end have no part in the row's sums."""
import numpy as np
import pytest
import torch

from gpu_helpers import dev, host, say, to_dev
from integer_only_nn_amd import ops
from oracle import floats as of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cols", [1, 5, 100, 258, 1002, 2050, 4095, 4097, 9001])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_far_from_zero(cols, dtype):
    rows = 3
    rng = np.random.default_rng(cols)
    x = torch.full((rows, cols), 1e37).to(dtype).double().numpy()  # constant rows: h = 0
    x[1] = rng.standard_normal(cols)
    x = torch.from_numpy(x).to(dtype)
    dy = torch.from_numpy(rng.standard_normal((rows, cols))).to(dtype)
    gamma = (1 + 0.1 * rng.standard_normal(cols)).astype(np.float32)
    mean, rstd = (v.astype(np.float32) for v in of.layer_norm_fwd(x.double().numpy(), None, None, 1e-5)[1:])
    say("norm bwd far", cols, dtype)
    xd, dyd = x.to(dev()), dy.to(dev())
    dx, dg, db = torch.empty_like(xd), torch.empty(cols, device=dev()), torch.empty(cols, device=dev())
    ws = torch.empty(ops.ionn_layer_norm_bwd_workspace_bytes(rows, cols), dtype=torch.uint8, device=dev())
    ops.ionn_layer_norm_bwd(dyd, xd, to_dev(mean), to_dev(rstd), dx, gamma=to_dev(gamma), dgamma=dg, dbeta=db, workspace=ws)
    wx, wg, wb = of.layer_norm_bwd(dy.double().numpy(), x.double().numpy(), mean, rstd, gamma, None)
    got = host(dx.double())
    assert np.isfinite(got).all() and np.isfinite(host(dg)).all()
    # sums of at most 128 half steps of float32 (2^-17) of terms of the size of
    # rstd |dy| here, in every row, and half a step of the type
    half = torch.finfo(dtype).eps / 2
    size = rstd.astype(np.float64)[:, None] * (np.abs(dy.double().numpy() * gamma) + 1.0)
    size[1] *= 20  # (h up to 5 in the row that is not constant, twice)
    assert (np.abs(got - wx) <= 2.0 ** -17 * size + half * np.abs(wx) * 1.01 + 1e-30).all()
    assert (np.abs(host(db) - wb) <= 67 * 2.0 ** -24 * np.abs(dy.double().numpy()).sum(0)).all()
