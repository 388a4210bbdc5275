"""The block norm and its backward against the CPU oracle.

Forward: every output bit for bit (the oracle uses the same fp32 operations and an fp64 sum whose
order does not show).  Backward: fp32 against fp64.  An element's rounding error is at most K u
times the sum of the absolute terms behind it, u = 2^-24: a row's mean is a sum over d terms with
at most 8 (columns of a thread) + 5 + 8 + 6 (warp, block and cluster) roundings on the path of a
term, each term with at most 12 roundings of its own, and the products around it 8 more: K = 64
covers dY and dH.  A column sum adds the rows of a lane in sequence (at most 40 here), then at most
8 lanes and 16 + 20 partial rows: K = 192.  A bf16 output is one rounding more, 2^-8 of the value.
"""
import numpy as np
import pytest
import torch

import oracle
import synth

pytestmark = pytest.mark.gpu

U, UB = 2.0 ** -24, 2.0 ** -8
EPS = 1e-6


def _f(t):
    return None if t is None else t.float().cpu().numpy()


class Case:
    def __init__(self, T, d, y_bf16=False, h_f32=False, post=True, period=None, readers=1, seed=0, s=0.75):
        g = synth.gen(seed, 31)
        rnd = lambda *shape: torch.randn(*shape, generator=g)  # noqa: E731
        self.T, self.d, self.s, self.period = T, d, s, period
        self.yt = torch.bfloat16 if y_bf16 else torch.float32
        self.ht = torch.float32 if h_f32 else torch.bfloat16
        self.Y = (2 * rnd(T, d)).to(self.yt).cuda()
        self.H = (3 * rnd(T, d)).to(self.ht).cuda()
        if T > 2:  # a padding token
            self.Y[T // 2] = 0
            self.H[T // 2] = 0
        self.g_pre = (1 + 0.2 * rnd(d)).to(torch.bfloat16).cuda()
        self.g_post = (1 + 0.2 * rnd(d)).to(torch.bfloat16).cuda() if post else None
        self.gate = rnd(-(-T // period), d).to(torch.bfloat16).cuda() if period else None
        self.dXn = [rnd(T, d).cuda() for _ in range(readers)]
        self.dH_out = rnd(T, d).to(self.ht).cuda()
        self.gen = g

    def flags(self, lib):
        return (lib.SBL_BLOCK_Y_BF16 if self.yt == torch.bfloat16 else 0) | \
            (lib.SBL_BLOCK_H_F32 if self.ht == torch.float32 else 0)

    def buffers(self):
        T, d = self.T, self.d
        # one row of guard values behind the last token
        e = lambda dt, n=1: torch.full((T + 1, n), 77, dtype=dt, device="cuda")  # noqa: E731
        self.H_out, self.Xn, self.Xq = e(self.ht, d), e(torch.bfloat16, d), e(torch.int8, d)
        self.amax = torch.full((T + 1,), 77.0, device="cuda")
        self.rstd = torch.full((2 * T + 1,), 77.0, device="cuda")

    def forward(self, lib, **kw):
        a = dict(H_out=self.H_out, Xn=self.Xn, Xq=self.Xq, amax=self.amax, rstd=self.rstd)
        a.update(kw)
        lib.sbl_block_norm(self.Y, self.H, self.g_post, self.gate, self.period or 0, self.s, self.g_pre, EPS, self.T,
                           self.d, self.flags(lib), a["H_out"], a["Xn"], a["Xq"], a["amax"], a["rstd"])

    def oracle_forward(self):
        return oracle.block_norm(_f(self.Y), _f(self.H), _f(self.g_pre), self.s, EPS, _f(self.g_post), _f(self.gate),
                                 self.period or 1, h_bf16=self.ht == torch.bfloat16)

    def check_forward(self):
        T = self.T
        ref = self.oracle_forward()
        assert np.array_equal(_f(self.H_out[:T]), ref["h_out"])
        assert np.array_equal(synth.bits(self.Xn[:T].cpu()), ref["xn"])
        assert np.array_equal(self.Xq[:T].cpu().numpy(), ref["xq"])
        assert np.array_equal(self.amax[:T].cpu().numpy(), ref["amax"])
        assert np.array_equal(self.rstd[:T].cpu().numpy(), ref["r1"])
        assert np.array_equal(self.rstd[T:2 * T].cpu().numpy(), ref["r2"])
        for b in (self.H_out[T:], self.Xn[T:], self.Xq[T:], self.amax[T:], self.rstd[2 * T:]):
            assert torch.all(b == 77)
        return ref

    def backward(self, lib, accumulate=0, dH_in_place=False, ws=None, dH_out="given"):
        T, d = self.T, self.d
        dev = dict(device="cuda")
        self.dY = torch.full((T + 1, d), 77, dtype=torch.bfloat16, **dev)
        dH_out = self.dH_out if isinstance(dH_out, str) else dH_out
        if dH_in_place:
            self.dH = self.dH_out.clone()
            dH_out = self.dH
        else:
            self.dH = torch.full((T + 1, d), 77, dtype=self.ht, **dev)
        if not accumulate:
            rows = -(-T // self.period) if self.period else 0
            self.grads = {"dg_pre": torch.full((d,), 77.0, **dev),
                          "dg_post": torch.full((d,), 77.0, **dev) if self.g_post is not None else None,
                          "dgate": torch.full((rows + 1, d), 77.0, **dev) if self.period else None}
        n = lib.sbl_block_norm_backward_workspace_bytes(d)
        ws = torch.full((n,), 255, dtype=torch.uint8, **dev) if ws is None else ws
        lib.sbl_block_norm_backward(self.dXn, dH_out, self.Y, self.H_out[:T], self.g_post, self.gate, self.period or 0,
                                    self.s, self.g_pre, self.rstd, T, d, self.flags(lib), self.dY, self.dH,
                                    self.grads["dg_post"], self.grads["dg_pre"], self.grads["dgate"], accumulate, ws, n)

    def check_backward(self, times=1, with_dh=True):
        T = self.T
        r = self.rstd.cpu().numpy()
        ref = oracle.block_norm_backward([_f(g) for g in self.dXn], _f(self.Y), _f(self.H_out[:T]), r[:T], r[T:2 * T],
                                         _f(self.g_pre), self.s, _f(self.dH_out) if with_dh else None, _f(self.g_post),
                                         _f(self.gate), self.period or 1)

        def near(got, name, K, bf16, times=1):
            tol = K * U * ref["abs"][name] * times
            if bf16:
                tol = tol + UB * (np.abs(ref[name]) + tol)
            worst = np.max(np.abs(got - times * ref[name]) - tol, initial=-1.0)
            assert worst <= 0.0, (name, worst)

        near(_f(self.dY[:T]), "dy", 64, True)
        near(_f(self.dH[:T]), "dh", 64, self.ht == torch.bfloat16)
        assert torch.all(self.dY[T:] == 77) and torch.all(self.dH[T:] == 77)
        for name, g in self.grads.items():
            if g is not None:
                got = _f(g[:-1] if name == "dgate" else g)
                near(got, name, 192, False, times)
        if self.grads["dgate"] is not None:
            assert torch.all(self.grads["dgate"][-1] == 77)


WIDTHS = [16, 48, 256, 272, 512, 528, 896, 1024, 1040, 2048, 2064, 4096, 4112, 8192, 8208, 16384]


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("T", [1, 2, 5, 37])
def test_forward_and_backward_at_every_width(lib, T, d):
    """Below, at and past every border between the kernels' shapes."""
    k = WIDTHS.index(d) + T
    c = Case(T, d, y_bf16=k % 2 == 0, h_f32=k % 3 == 0, period=[None, 1, 3, T][k % 4], readers=1 + k % 3, seed=d + T)
    c.buffers()
    c.forward(lib)
    lib.sbl_check()
    c.check_forward()
    c.backward(lib)
    lib.sbl_check()
    c.check_backward()


@pytest.mark.parametrize("y_bf16", [False, True])
@pytest.mark.parametrize("h_f32", [False, True])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("period", [None, 1, 7, 64, 10 ** 6])
def test_types_and_parts(lib, y_bf16, h_f32, post, period):
    c = Case(129, 272, y_bf16, h_f32, post, min(period, 129) if period else None, readers=2, seed=5)
    c.buffers()
    if period == 10 ** 6:  # one row for all tokens, named by a period beyond the batch
        c.period = 10 ** 6
    c.forward(lib)
    c.check_forward()
    c.backward(lib)
    c.check_backward()
    assert torch.equal(c.rstd[:129], torch.ones(129, device="cuda")) or post


@pytest.mark.parametrize("T,d,period,readers", [(6000, 256, 250, 3), (4100, 896, 1000, 2), (1999, 2048, 667, 3),
                                                (700, 4112, None, 1), (333, 8192, 5, 2), (5000, 64, 2, 1),
                                                (3001, 512, 1, 1), (24000, 256, 4096, 1), (23999, 48, 7, 2)])
def test_batches_that_cut_groups_into_segments(lib, T, d, period, readers):
    """More tokens than row lanes: several rows and segments per lane, ragged last group."""
    c = Case(T, d, period=period, readers=readers, seed=T)
    c.buffers()
    c.forward(lib)
    c.check_forward()
    c.backward(lib)
    c.check_backward()


def test_optional_outputs(lib):
    c = Case(33, 96, seed=8)
    c.buffers()
    c.forward(lib)
    ref = c.check_forward()
    keep = c.H_out.clone()
    c.H_out.fill_(77)
    c.forward(lib, Xq=None, amax=None, Xn=None, rstd=None)
    assert torch.equal(c.H_out, keep)
    # in place on the residual stream
    h = c.H.clone()
    lib.sbl_block_norm(c.Y, h, c.g_post, None, 0, c.s, c.g_pre, EPS, 33, 96, 0, h, None, c.Xq, c.amax, None)
    assert np.array_equal(_f(h), ref["h_out"])
    # gradients one at a time, and none
    n = lib.sbl_block_norm_backward_workspace_bytes(96)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    c.backward(lib)
    want = {k: v.clone() for k, v in c.grads.items() if v is not None}
    dY = c.dY.clone()
    for only in ("dg_post", "dg_pre", None):
        g = {k: torch.zeros_like(v) if k == only else None for k, v in want.items()}
        c.dY.fill_(77)
        lib.sbl_block_norm_backward(c.dXn, c.dH_out, c.Y, c.H_out[:33], c.g_post, None, 0, c.s, c.g_pre, c.rstd, 33, 96,
                                    0, c.dY, None, g["dg_post"], g["dg_pre"], None, 0, ws, n)
        assert torch.equal(c.dY, dY)
        if only:
            assert torch.equal(g[only], want[only])


@pytest.mark.parametrize("period", [None, 1, 40])
def test_accumulate_in_place_and_without_stream_gradient(lib, period):
    c = Case(200, 528, period=period, h_f32=True, seed=9)
    c.buffers()
    c.forward(lib)
    c.backward(lib)
    c.check_backward()
    first = {k: None if v is None else v.clone() for k, v in c.grads.items()}
    c.backward(lib, accumulate=1)
    for k, v in c.grads.items():
        if v is not None:
            rows = slice(0, -1) if k == "dgate" else slice(None)
            assert torch.equal(v[rows], 2 * first[k][rows])
    c.grads = first
    dH = c.dH[:200].clone()
    c.backward(lib, dH_in_place=True)
    assert torch.equal(c.dH, dH)
    c.dH = torch.cat([c.dH, torch.full((1, 528), 77.0, device="cuda")])
    c.check_backward()
    c.backward(lib, dH_out=None)
    c.check_backward(with_dh=False)


@pytest.mark.parametrize("period", [None, 3])
def test_backward_without_y(lib, period):
    """Neither a branch norm nor the gate's gradient: y is not read, and nothing else changes."""
    c = Case(41, 304, post=False, period=period, seed=15)
    c.buffers()
    c.forward(lib)
    c.backward(lib)
    want = [c.dY.clone(), c.dH.clone(), c.grads["dg_pre"].clone()]
    n = lib.sbl_block_norm_backward_workspace_bytes(304)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    c.dY.fill_(77)
    c.dH.fill_(77)
    lib.sbl_block_norm_backward(c.dXn, c.dH_out, None, c.H_out[:41], None, c.gate, period or 0, c.s, c.g_pre, c.rstd, 41,
                                304, 0, c.dY, c.dH, None, c.grads["dg_pre"], None, 0, ws, n)
    for a, b in zip(want, (c.dY, c.dH, c.grads["dg_pre"])):
        assert torch.equal(a, b)


def test_empty_batch(lib):
    e = torch.empty(0, 64, device="cuda")
    b = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    gain = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    lib.sbl_block_norm(e, b, gain, None, 0, 1.0, gain, EPS, 0, 64, 0, b, b, None, None, None)
    n = lib.sbl_block_norm_backward_workspace_bytes(64)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    dg = [torch.full((64,), 5.0, device="cuda") for _ in range(2)]
    lib.sbl_block_norm_backward([e], None, e, b, gain, None, 0, 1.0, gain, e, 0, 64, 0, b, b, dg[0], dg[1], None, 1,
                                ws, n)
    assert torch.all(dg[0] == 5) and torch.all(dg[1] == 5)
    lib.sbl_block_norm_backward([e], None, e, b, gain, None, 0, 1.0, gain, e, 0, 64, 0, b, b, dg[0], dg[1], None, 0,
                                ws, n)
    assert torch.all(dg[0] == 0) and torch.all(dg[1] == 0)
    lib.sbl_check()


def test_rows_with_nan_and_infinity_keep_to_themselves(lib):
    c = Case(9, 320, seed=11)
    c.buffers()
    c.forward(lib)
    clean = [t.clone() for t in (c.H_out, c.Xn, c.Xq, c.amax)]
    c.Y[2, 7] = float("nan")
    c.H[5, 300] = float("inf")
    c.Y[7, 0] = float("inf")
    c.forward(lib)
    lib.sbl_check()
    fine = [0, 1, 3, 4, 6, 8]
    for got, want in zip((c.H_out, c.Xn, c.Xq, c.amax), clean):
        assert torch.equal(got[fine], want[fine])
    for row in (2, 5, 7):
        assert not torch.isfinite(c.amax[row])
        assert torch.all(c.Xq[row] == 0)
    # every product of such a row is then NaN, and of no other row
    Wq = torch.ones(8, 320, dtype=torch.int8, device="cuda")
    gamma = torch.ones(1, device="cuda")
    out = torch.empty(9, 8, device="cuda")
    lib.sbl_forward(c.Xq[:9], c.amax[:9], Wq, gamma, 9, 320, 8, out)
    assert torch.isnan(out[[2, 5, 7]]).all() and torch.isfinite(out[fine]).all()


def test_other_stream_and_graph_replay(lib):
    c = Case(70, 2064, period=9, readers=2, seed=12)
    c.buffers()
    c.forward(lib)
    c.backward(lib)  # the buffers of the captured calls
    n = lib.sbl_block_norm_backward_workspace_bytes(2064)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        c.forward(lib)
        lib.sbl_block_norm_backward(c.dXn, c.dH_out, c.Y, c.H_out[:70], c.g_post, c.gate, 9, c.s, c.g_pre, c.rstd, 70,
                                    2064, 0, c.dY, c.dH, c.grads["dg_post"], c.grads["dg_pre"], c.grads["dgate"], 0,
                                    ws, n)
    for k in range(2):
        c.Y[:, 3 + k] += 1.0
        c.dXn[0].mul_(1.25)
        graph.replay()
        torch.cuda.synchronize()
        c.check_forward()
        c.check_backward()


def test_backward_is_deterministic(lib):
    c = Case(3000, 896, period=100, readers=3, seed=13)
    c.buffers()
    c.forward(lib)
    c.backward(lib)
    one = [c.dY.clone(), c.dH.clone()] + [g.clone() for g in c.grads.values()]
    c.backward(lib)
    for a, b in zip(one, [c.dY, c.dH] + list(c.grads.values())):
        assert torch.equal(a, b)


def test_gradient_against_differences_of_the_library_s_forward(lib):
    """Along random directions of y and h (fp32 stream, no quantiser): the change of
    sum(w1 h') + sum(w2 norm(h') g) over a step, with norm(h') g from the stored h' and r2 in fp64."""
    T, d, step = 4, 256, 1e-2
    c = Case(T, d, h_f32=True, period=2, seed=14)
    c.buffers()
    c.forward(lib)
    c.backward(lib)
    w1, w2 = c.dH_out.double(), c.dXn[0].double()
    y0, h0 = c.Y.clone(), c.H.clone()

    def value():
        c.forward(lib)
        h1 = c.H_out[:T].double()
        r2 = (h1.square().mean(1, keepdim=True) + EPS).rsqrt()
        return ((w1 * h1).sum() + (w2 * h1 * r2 * c.g_pre.double()).sum()).item()

    for k in range(4):
        vy = torch.randn(T, d, generator=c.gen).cuda()
        vh = torch.randn(T, d, generator=c.gen).cuda()
        vy[T // 2] = vh[T // 2] = 0  # the padding token: its norm turns too fast for a difference
        at = {}
        for sgn in (1, -1):
            c.Y.copy_(y0 + sgn * step * vy)
            c.H.copy_(h0 + sgn * step * vh)
            at[sgn] = value()
        diff = (at[1] - at[-1]) / (2 * step)
        c.Y.copy_(y0)
        c.H.copy_(h0)
        terms = c.dY[:T].double() * vy.double(), c.dH[:T].double() * vh.double()
        want = sum(t.sum().item() for t in terms)
        size = sum(t.abs().sum().item() for t in terms)
        # dY is rounded to bf16 (2^-8 of each term); fp32 noise of h' over the step, and the step's
        # third-order term (step^2 of the terms), stay below the same again
        assert abs(diff - want) <= 2 * UB * size


# At and past the widths where a thread gets another vector of 4 columns; K = 64 still covers 16 columns
# of a thread (16 + 5 + 8 + 6 + 12 + 8 = 55).
VECTORS = [320, 336, 384, 400, 640, 656, 768, 784, 896, 912, 1280, 1296, 1536, 1552, 1792, 1808, 2560, 2576, 3056, 3088,
           3584, 3600, 5120, 5136, 6144, 6160, 7168, 7184, 10240, 10256, 12288, 12304, 14336, 14352]


@pytest.mark.parametrize("h_f32", [False, True])
@pytest.mark.parametrize("d", VECTORS)
def test_widths_between_the_powers_of_two(lib, d, h_f32):
    k = VECTORS.index(d)
    T = 601 if d <= 4096 else 151
    c = Case(T, d, y_bf16=k % 4 < 2, h_f32=h_f32, post=k % 5 != 4, period=[None, 1, 200][k % 3], readers=1 + k // 2 % 3,
             seed=d)
    c.buffers()
    c.forward(lib)
    lib.sbl_check()
    c.check_forward()
    c.backward(lib)
    lib.sbl_check()
    c.check_backward()


@pytest.mark.parametrize("h_f32", [False, True])
@pytest.mark.parametrize("d", [112, 128, 144, 160, 176, 192, 208, 240, 272, 336, 400, 464])
def test_narrow_rows_in_great_number(lib, d, h_f32):
    k = d // 16
    c = Case(23711, d, y_bf16=k % 2 == 0, h_f32=h_f32, period=[None, 1, 5000][k % 3], readers=1 + k % 2, seed=d)
    c.buffers()
    c.forward(lib)
    lib.sbl_check()
    c.check_forward()
    c.backward(lib)
    lib.sbl_check()
    c.check_backward()
