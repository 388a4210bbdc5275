"""CPU oracle of the operators around the Sparse-BitLinear products of a block:
the block norm and its backward, the 8-bit product, and the clipped gradients.

Test infrastructure like ``sbl_oracle`` (which holds the quantiser and the
gradient norm that these build on).  Values are passed as fp32 arrays; a bf16
tensor is passed decoded.  Steps that decide integers or a stored type are
explicit IEEE fp32 operations in the operator's order; gradients are in fp64.
"""
from __future__ import annotations

import numpy as np

from .sbl_oracle import QMAX, act_quant, bf16_to_f32, f32_to_bf16, grad_clip_scale, grad_sqnorm

__all__ = ["rms_factor", "gate_rows", "block_norm", "block_norm_backward", "w8a8_out", "clip_grads"]

F32 = np.float32


def rms_factor(x: np.ndarray, eps: float) -> np.ndarray:
    """fl32(1 / fl32(sqrt(fl32(sum x^2 / d + eps)))) of each row, the sum in fp64."""
    ss = np.square(x.astype(np.float64)).sum(axis=1)
    v = (ss / x.shape[1] + float(F32(eps))).astype(F32)
    return np.divide(F32(1.0), np.sqrt(v, dtype=F32), dtype=F32)


def gate_rows(gate: np.ndarray, period: int, T: int) -> np.ndarray:
    """The gate row of every token: token t takes row t // period."""
    return gate[np.arange(T) // period]


def block_norm(y, h, g_pre, res_scale, eps, g_post=None, gate=None, period=1, h_bf16=True):
    """h' = T(s h + gate norm(y) g_post); xn = bf16(norm(h') g_pre); Q_a(xn).

    Returns a dict with h_out (fp32 values of its stored type), xn (bf16
    bits), xq, amax, r1, r2.  [summary] Algorithm 1 step (3).
    """
    T = y.shape[0]
    u = y.astype(F32)
    r1 = np.ones(T, F32)
    if g_post is not None:
        r1 = rms_factor(u, eps)
        u = np.multiply(np.multiply(u, r1[:, None], dtype=F32), g_post[None, :], dtype=F32)
    if gate is not None:
        u = np.multiply(gate_rows(gate, period, T), u, dtype=F32)
    h1 = np.add(np.multiply(F32(res_scale), h, dtype=F32), u, dtype=F32)
    if h_bf16:
        h1 = bf16_to_f32(f32_to_bf16(h1))
    r2 = rms_factor(h1, eps)
    xn = f32_to_bf16(np.multiply(np.multiply(h1, r2[:, None], dtype=F32), g_pre[None, :], dtype=F32))
    xq, amax = act_quant(xn)
    return dict(h_out=h1, xn=xn, xq=xq, amax=amax, r1=r1, r2=r2)


def block_norm_backward(dxn, y, h_out, r1, r2, g_pre, res_scale, dh_out=None, g_post=None, gate=None, period=1):
    """Gradients of the block norm in fp64, the quantiser passed by.

    dxn: list of the gradients of xn, one per reader.  r1, r2: the factors
    that the forward pass saved.  Returns dy, dh, dg_pre, dg_post, dgate, and
    under "abs" the sums of absolute terms behind each of them (what a bound
    on the rounding of an fp32 evaluation is proportional to).
    """
    f8 = np.float64
    T, d = y.shape
    mx = sum(np.abs(g.astype(f8)) for g in dxn)
    dxn, y, h = sum(g.astype(f8) for g in dxn), y.astype(f8), h_out.astype(f8)
    r1, r2, gp = r1.astype(f8)[:, None], r2.astype(f8)[:, None], g_pre.astype(f8)
    go = np.ones(d) if g_post is None else g_post.astype(f8)
    gt = np.ones((T, d)) if gate is None else gate_rows(gate, period, T).astype(f8)
    dhin = np.zeros((T, d)) if dh_out is None else dh_out.astype(f8)
    xh, t = h * r2, dxn * gp
    mt = mx * np.abs(gp)
    c2, a2 = (t * xh).mean(1, keepdims=True), (mt * np.abs(xh)).mean(1, keepdims=True)
    dh1 = dhin + r2 * (t - xh * c2)
    m1 = np.abs(dhin) + r2 * (mt + np.abs(xh) * a2)  # magnitudes of the terms of dh1
    yh = y * r1 if g_post is not None else y
    du, mu = gt * dh1, np.abs(gt) * m1
    out = {"dh": float(F32(res_scale)) * dh1, "dg_pre": (dxn * xh).sum(0)}
    ab = {"dh": abs(float(F32(res_scale))) * m1, "dg_pre": (mx * np.abs(xh)).sum(0)}
    if gate is not None:
        n = gate.shape[0]
        out["dgate"], ab["dgate"] = np.zeros((n, d)), np.zeros((n, d))
        np.add.at(out["dgate"], np.arange(T) // period, dh1 * yh * go)
        np.add.at(ab["dgate"], np.arange(T) // period, m1 * np.abs(yh * go))
    if g_post is not None:
        out["dg_post"], ab["dg_post"] = (du * yh).sum(0), (mu * np.abs(yh)).sum(0)
        c1, a1 = (du * go * yh).mean(1, keepdims=True), (mu * np.abs(go * yh)).mean(1, keepdims=True)
        out["dy"] = r1 * (du * go - yh * c1)
        ab["dy"] = r1 * (mu * np.abs(go) + np.abs(yh) * a1)
    else:
        out["dy"], ab["dy"] = du, mu
    out["abs"] = ab
    return out


def w8a8_out(acc: np.ndarray, amax: np.ndarray, wmax: np.ndarray) -> np.ndarray:
    """y = fl32(fl32(fl32(acc) * fl32(amax_t / 127)) * fl32(wmax_o / 127))."""
    sx = np.divide(amax.astype(F32), QMAX, dtype=F32)
    sw = np.divide(wmax.astype(F32), QMAX, dtype=F32)
    return np.multiply(np.multiply(acc.astype(F32), sx[:, None], dtype=F32), sw[None, :], dtype=F32)


def clip_grads(grads, max_norm):
    """(S, norm, clip, clipped gradients as fp32 products before a bf16 store)."""
    S = grad_sqnorm(*grads)
    c = grad_clip_scale(S, max_norm)
    return S, F32(np.sqrt(S)), c, [np.multiply(np.asarray(g, F32), c, dtype=F32) for g in grads]
