"""The block norm's gradients against differences of the library's own forward, each row along itself: the
directions that the mean terms of the gradients decide (norm_radial.py has the bound)."""
import numpy as np
import pytest
import torch

from norm_radial import UB, Rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [16, 64, 256, 896, 2048, 4112, 8192, 8208])
def test_gradient_along_each_row(lib, d):
    c = Rows(d=d, seed=d)
    dev = dict(device="cuda")
    up = lambda a, dt=torch.float32: torch.from_numpy(np.ascontiguousarray(a)).to(dt).cuda()  # noqa: E731
    bf = torch.bfloat16
    g_pre, g_post, gate = up(c.g_pre, bf), up(c.g_post, bf), up(c.gate, bf)
    rstd = torch.empty(2 * c.T, **dev)

    def h_out(y, h):
        out = torch.empty(c.T, d, **dev)
        lib.sbl_block_norm(up(y), up(h), g_post, gate, c.period, c.s, g_pre, c.eps, c.T, d, lib.SBL_BLOCK_H_F32, out,
                           None, None, None, rstd)
        return out.cpu().numpy()

    stored = up(h_out(c.y, c.h))
    n = lib.sbl_block_norm_backward_workspace_bytes(d)
    ws = torch.empty(n, dtype=torch.uint8, **dev)
    dY, dH = torch.empty(c.T, d, dtype=bf, **dev), torch.empty(c.T, d, **dev)
    lib.sbl_block_norm_backward([up(c.w2)], up(c.w1), up(c.y), stored, g_post, gate, c.period, c.s, g_pre, rstd, c.T, d,
                                lib.SBL_BLOCK_H_F32, dY, dH, None, None, None, 0, ws, n)
    lib.sbl_check()
    errors = c.errors(dY.float().cpu().numpy(), dH.cpu().numpy(), h_out, UB)
    assert np.all(errors <= 1.0), errors
