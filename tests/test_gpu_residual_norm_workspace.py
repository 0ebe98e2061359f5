"""GPU: ionn_residual_norm_bwd keeps to its workspace, and its gradients do not
depend on what that held."""
import pytest
import torch

from gpu_helpers import dev, say
from integer_only_nn_amd import ops

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,cols,gate_rows", [(1, 1, 0), (5, 70, 0), (300, 1000, 7), (1300, 100, 2), (700, 600, 1), (513, 70, 1),
                                                 (5000, 2000, 4000), (8192, 64, 64), (40000, 24, 600), (600, 5120, 0),
                                                 (9, 16384, 4), (4096, 4097, 4096)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_workspace(rows, cols, gate_rows, dtype):
    g = torch.Generator(device=dev()).manual_seed(rows + cols)
    rnd = lambda *s, t=dtype: torch.randn(s, device=dev(), generator=g).to(t)  # noqa: E731
    gates = -(-rows // gate_rows) if 0 < gate_rows < rows else 1
    dy, dn, a, y = (rnd(rows, cols) for _ in range(4))
    f32 = torch.float32
    gate, vecs = rnd(gates, cols, t=f32), {k: rnd(cols, t=f32) for k in ("gamma_a", "beta_a", "gamma_y")}
    stats = {k: rnd(rows, t=f32) for k in ("mean_a", "rstd_a", "mean_y", "rstd_y")}
    need = ops.ionn_residual_norm_bwd_workspace_bytes(rows, cols, gate_rows)
    for norms in (("layer", "layer"), ("rms", "rms")):
        out = []
        for fill in (0, 0xff):
            ws = torch.full((need + (1 << 16),), fill, dtype=torch.uint8, device=dev())
            got = {k: torch.full((cols,), 7.0, device=dev()) for k in ("dgamma_a", "dbeta_a", "dgamma_y", "dbeta_y")}
            got["dgate"] = torch.full((gates, cols), 7.0, device=dev())
            kw = dict(vecs, **stats)
            if norms[0] == "rms":
                for k in ("beta_a", "mean_a", "mean_y"):
                    kw.pop(k)
                for k in ("dbeta_a", "dbeta_y"):
                    got.pop(k)
            da, dx = torch.empty_like(a), torch.empty_like(a)
            say("residual norm bwd", rows, cols, gate_rows, norms, fill)
            ops.ionn_residual_norm_bwd(dy, dn, a, y, da, dx, norm_a=norms[0], norm_y=norms[1], gate=gate, gate_rows=gate_rows, **kw,
                                       **got, workspace=ws[:need])
            assert (ws[need:] == fill).all()
            out.append([da, dx, *got.values()])
        assert all(torch.equal(p, q) for p, q in zip(*out))
