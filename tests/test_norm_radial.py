"""The derivatives along a row tell a gradient of the block norm from one without its mean terms (CPU; the
kernels are held against them in test_gpu_norm_radial.py)."""
import numpy as np
import pytest

import oracle
from norm_radial import UB, Rows


def _bf16(x):
    return oracle.bf16_to_f32(oracle.f32_to_bf16(x.astype(np.float32)))


def _without(c, f, g, term):
    """dy, dh of the formula with one mean term left out."""
    f8 = lambda a: np.asarray(a).astype(np.float64)  # noqa: E731
    r1, r2, h = f8(f["r1"])[:, None], f8(f["r2"])[:, None], f8(f["h_out"])
    gate = f8(oracle.gate_rows(c.gate, c.period, c.T))
    yh, xh, t = f8(c.y) * r1, h * r2, f8(c.w2) * f8(c.g_pre)
    dh1 = f8(c.w1) + r2 * (t - (0.0 if term == "c2" else (t * xh).mean(1, keepdims=True)) * xh)
    dz = gate * dh1 * f8(c.g_post)
    dy = r1 * (dz - (0.0 if term == "c1" else (dz * yh).mean(1, keepdims=True)) * yh)
    return dy, c.s * dh1


@pytest.mark.parametrize("seed", range(5))
@pytest.mark.parametrize("d", [64, 256, 2048])
def test_gradients_without_a_mean_term_are_told_apart(seed, d):
    c = Rows(d=d, seed=seed)
    f = c.forward(c.y, c.h)
    g = c.gradients(f)
    h_out = lambda y, h: c.forward(y, h)["h_out"]  # noqa: E731
    assert np.all(c.errors(_bf16(g["dy"]), g["dh"].astype(np.float32), h_out, UB) <= 1.0)
    dy, dh = _without(c, f, g, None)
    np.testing.assert_allclose(dy, g["dy"], rtol=1e-9, atol=1e-12)
    np.testing.assert_allclose(dh, g["dh"], rtol=1e-9, atol=1e-12)
    for term, which in (("c1", 0), ("c2", 1)):
        dy, dh = _without(c, f, g, term)
        e = c.errors(_bf16(dy), dh.astype(np.float32), h_out, UB)
        assert np.median(e[which]) > 1.0, (term, e)  # most rows tell, each for itself
