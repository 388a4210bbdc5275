"""Pins of the oracle of the operators around the products (``oracle/block_oracle.py``)
to things other than itself: torch autograd in fp64, differences, exact integers, and
``torch.nn.utils.clip_grad_norm_``."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle


def _case(T, d, seed, post=True, period=None):
    r = np.random.default_rng(seed)
    bf = lambda a: oracle.bf16_to_f32(oracle.f32_to_bf16(a.astype(np.float32)))  # noqa: E731
    return dict(y=r.standard_normal((T, d)).astype(np.float32), h=bf(r.standard_normal((T, d))),
                g_pre=bf(1 + 0.2 * r.standard_normal(d)), g_post=bf(1 + 0.2 * r.standard_normal(d)) if post else None,
                gate=None if period is None else bf(r.standard_normal((-(-T // period), d))),
                period=1 if period is None else period)


def _torch_forward(c, y, h, g_pre, g_post, gate, s, eps):
    rms = lambda x: x * (x.square().mean(1, keepdim=True) + eps).rsqrt()  # noqa: E731
    u = y if g_post is None else rms(y) * g_post
    if gate is not None:
        u = gate[torch.arange(y.shape[0]) // c["period"]] * u
    h1 = s * h + u
    return h1, rms(h1) * g_pre


@pytest.mark.parametrize("post,period", [(True, None), (True, 3), (False, 1), (False, None), (True, 7)])
def test_forward_follows_the_formula(post, period):
    c = _case(7, 48, 1, post, period)
    out = oracle.block_norm(c["y"], c["h"], c["g_pre"], 0.5, 1e-6, c["g_post"], c["gate"], c["period"], h_bf16=False)
    t = lambda a: None if a is None else torch.from_numpy(a).double()  # noqa: E731
    h1, xn = _torch_forward(c, t(c["y"]), t(c["h"]), t(c["g_pre"]), t(c["g_post"]), t(c["gate"]), 0.5, 1e-6)
    # h': at most five fp32 roundings of terms no larger than |s h| + |gate u|
    np.testing.assert_allclose(out["h_out"], h1.numpy(), rtol=0, atol=8 * 2.0 ** -24 * (h1.abs().max().item() + 10))
    ref = xn.numpy()
    assert np.all(np.abs(oracle.bf16_to_f32(out["xn"]) - ref) <= 2.0 ** -8 * np.abs(ref) + 1e-5)


def test_forward_without_the_branch_parts_is_norm_and_quantiser_of_the_sum():
    c = _case(5, 32, 2, post=False)
    out = oracle.block_norm(c["y"], c["h"], c["g_pre"], 1.0, 1e-6)
    h1 = oracle.f32_to_bf16(c["h"] + c["y"])
    xn, xq, amax = oracle.rms_norm_act_quant(h1, oracle.f32_to_bf16(c["g_pre"]), 1e-6)
    assert np.array_equal(oracle.f32_to_bf16(out["h_out"]), h1)
    assert np.array_equal(out["xn"], xn) and np.array_equal(out["xq"], xq) and np.array_equal(out["amax"], amax)
    assert np.array_equal(out["r1"], np.ones(5, np.float32))


@pytest.mark.parametrize("post,period,readers", [(True, None, 1), (True, 3, 2), (False, 1, 3), (False, None, 2)])
def test_backward_is_torch_autograd_and_differences(post, period, readers):
    T, d, s, eps = 7, 32, 0.75, 1e-6
    c = _case(T, d, 3, post, period)
    r = np.random.default_rng(4)
    dxn = [r.standard_normal((T, d)).astype(np.float32) for _ in range(readers)]
    dh = r.standard_normal((T, d)).astype(np.float32)
    leaf = {k: torch.from_numpy(c[k]).double().requires_grad_() for k in ("y", "h", "g_pre", "g_post", "gate")
            if c[k] is not None}

    def loss(**over):
        v = {k: over.get(k, leaf.get(k)) for k in ("y", "h", "g_pre", "g_post", "gate")}
        h1, xn = _torch_forward(c, v["y"], v["h"], v["g_pre"], v["g_post"], v["gate"], s, eps)
        return (torch.from_numpy(sum(g.astype(np.float64) for g in dxn)) * xn).sum() + \
            (torch.from_numpy(dh).double() * h1).sum()

    loss().backward()
    with torch.no_grad():
        h1, _ = _torch_forward(c, *[leaf.get(k) for k in ("y", "h", "g_pre", "g_post", "gate")], s, eps)
        r1 = (leaf["y"].square().mean(1) + eps).rsqrt().numpy() if post else np.ones(T)
        r2 = (h1.square().mean(1) + eps).rsqrt().numpy()
    got = oracle.block_norm_backward(dxn, c["y"], h1.numpy(), r1, r2, c["g_pre"], s, dh, c["g_post"], c["gate"],
                                     c["period"])
    for name, leaf_name in (("dy", "y"), ("dh", "h"), ("dg_pre", "g_pre"), ("dg_post", "g_post"), ("dgate", "gate")):
        if leaf_name in leaf:
            np.testing.assert_allclose(got[name], leaf[leaf_name].grad.numpy(), rtol=1e-9, atol=1e-10)
            assert np.all(np.abs(got[name]) <= got["abs"][name] * (1 + 1e-12) + 1e-300)
            # a central difference along a random direction: error of order step^2 and fp64 noise / step
            x = leaf[leaf_name].detach()
            v = torch.from_numpy(np.random.default_rng(5).standard_normal(tuple(x.shape)))
            step = 1e-5
            diff = (loss(**{leaf_name: x + step * v}) - loss(**{leaf_name: x - step * v})).item() / (2 * step)
            assert diff == pytest.approx((torch.from_numpy(got[name]) * v).sum().item(), rel=1e-6, abs=1e-6)


def test_w8a8_out_is_the_exact_scaled_product():
    """Against exact rationals: fl32(acc), two divisions and two products are five roundings."""
    r = np.random.default_rng(6)
    acc = r.integers(-2 ** 30, 2 ** 30, (4, 6)).astype(np.int32)
    amax = (r.random(4) * 5 + 0.1).astype(np.float32)
    wmax = (r.random(6) * 0.1 + 0.01).astype(np.float32)
    y = oracle.w8a8_out(acc, amax, wmax)
    for t in range(4):
        for o in range(6):
            want = Fraction(int(acc[t, o])) * Fraction(float(amax[t])) * Fraction(float(wmax[o])) / (127 * 127)
            assert abs(Fraction(float(y[t, o])) - want) <= abs(want) * 5 * Fraction(1, 2 ** 24) * Fraction(101, 100)


def test_clip_is_torch_clip_grad_norm():
    r = np.random.default_rng(7)
    grads = [r.standard_normal(n).astype(np.float32) for n in (5, 1, 300, 64)]
    for max_norm in (0.5, 1.0, 100.0):
        S, norm, c, out = oracle.clip_grads(grads, max_norm)
        ps = [torch.nn.Parameter(torch.zeros(len(g), dtype=torch.float64)) for g in grads]
        for p, g in zip(ps, grads):
            p.grad = torch.from_numpy(g).double()
        total = torch.nn.utils.clip_grad_norm_(ps, max_norm)
        assert norm == pytest.approx(total.item(), rel=2.0 ** -23)
        for p, o in zip(ps, out):
            np.testing.assert_allclose(o, p.grad.numpy(), rtol=2.0 ** -22)
