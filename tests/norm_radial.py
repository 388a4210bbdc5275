"""Derivatives of the block norm along its own rows, where the mean terms of its gradients are all there is.

A norm does not change when its row is scaled.  Along the row y_t of a branch that is normalised the loss changes
by eps alone, so <dY_t, y_t> is nearly 0: the term yh c1 of dY takes away as much as the rest brings.  Along the
stored stream row (h_t moved so that h'_t is scaled) the normalised row stays, and <dH_t, .> is <dH_out_t, h'_t>:
the term xh c2 takes away the rest.  A random direction meets either term only in one part in sqrt(d).
"""
import numpy as np

import oracle

U, UB = 2.0 ** -24, 2.0 ** -8
STEP = 2.0 ** -6


class Rows:
    """A case with an fp32 stream, a branch norm and gate rows, and the weights w1, w2 of a loss
    sum(w1 h') + sum(w2 norm(h') g_pre), which are the gradients that h' and xn get."""

    def __init__(self, T=6, d=256, period=2, s=0.75, eps=1e-6, seed=0):
        r = np.random.default_rng(seed)
        n = lambda *shape: r.standard_normal(shape).astype(np.float32)  # noqa: E731
        bf = lambda a: oracle.bf16_to_f32(oracle.f32_to_bf16(a.astype(np.float32)))  # noqa: E731
        self.T, self.d, self.period, self.s, self.eps = T, d, period, s, eps
        self.y, self.h, self.w1, self.w2 = 2 * n(T, d), 3 * n(T, d), n(T, d), n(T, d)
        self.g_pre, self.g_post, self.gate = bf(1 + 0.2 * n(d)), bf(1 + 0.2 * n(d)), bf(n(-(-T // period), d))

    def forward(self, y, h):
        """The oracle's forward pass."""
        return oracle.block_norm(y, h, self.g_pre, self.s, self.eps, self.g_post, self.gate, self.period, h_bf16=False)

    def gradients(self, f):
        """The oracle's gradients in fp64, from what the forward pass `f` saved."""
        return oracle.block_norm_backward([self.w2], self.y, f["h_out"], f["r1"], f["r2"], self.g_pre, self.s, self.w1,
                                          self.g_post, self.gate, self.period)

    def losses(self, h_out):
        """The loss of each row (no other row enters it) in fp64, from h'."""
        h = h_out.astype(np.float64)
        xh = h / np.sqrt((h * h).mean(1, keepdims=True) + self.eps)
        return (self.w1 * h + self.w2 * xh * self.g_pre).sum(1)

    def errors(self, dy, dh, h_out, dy_rounding):
        """dy and dh against central differences of h_out(y, h), each row along itself: [2, T], in units of the
        bound.  dy_rounding: half a step of dY's type, relative (dH is fp32).

        The bound, with g the gradient and v the direction:
        - half a step of the stored g, and 80 u of its absolute terms: 64 u as every element of dY and dH
          (test_gpu_block_norm.py), 16 u for the factor r that the forward saved, off by 3 u (three roundings, one
          of them under the root), which leaves 6 u of the two sums that cancel;
        - the moved row x + STEP v rounded at both ends: 2 u / (2 STEP) = 64 u of |g| |x + STEP v|;
        - h' at both ends: s h and the sum one rounding each, gate u six with its factor, so at most 7 u of
          |s h| + |h'| each, times |dh'|, over 2 STEP: 448 u;
        - no third order: along its row a norm changes by eps / mean square (below 1e-6), STEP^2 of that is nothing.
        """
        f = self.forward(self.y, self.h)
        ref = self.gradients(f)
        h1 = f["h_out"].astype(np.float64)
        h_noise = 448 * U * (np.abs(ref["dh"]) / self.s * (np.abs(self.s * self.h) + np.abs(h1))).sum(1)
        out = []
        for x, g, name, move, half_step in ((self.y, dy, "dy", STEP * self.y, dy_rounding),
                                            (self.h, dh, "dh", (STEP / self.s * h1).astype(np.float32), U)):
            ends = [x + move, x - move]
            at = [self.losses(h_out(e, self.h) if name == "dy" else h_out(self.y, e)) for e in ends]
            v = move.astype(np.float64) / STEP
            terms = g.astype(np.float64) * v
            bound = (half_step * np.abs(terms)).sum(1) + 80 * U * (ref["abs"][name] * np.abs(v)).sum(1) + \
                64 * U * (np.abs(ref[name]) * np.maximum(np.abs(ends[0]), np.abs(ends[1]))).sum(1) + h_noise
            out.append(np.abs((at[0] - at[1]) / (2 * STEP) - terms.sum(1)) / bound)
        return np.array(out)
