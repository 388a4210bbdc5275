"""The operators around the products together, as a user runs them: a training step of two projections
with a block norm between them, up to the clipped gradients and the optimizer, and a decode step in a
CUDA graph.  Each stage is checked against the oracle on what the stage before it left on the GPU, so
the tolerances are those of the single operators."""
import numpy as np
import pytest
import torch

import oracle
import synth
from bwd_tol import abs_dw, abs_dx, check_bwd

pytestmark = pytest.mark.gpu

U, UB = 2.0 ** -24, 2.0 ** -8


def _f(t):
    return t.float().cpu().numpy()


def test_training_step(lib):
    from semi_structured_sparsity_step_b200.layer import (BlockNorm, GradClip, SparseBitLinearLayer, act_quant)
    T, d0, d1, d2, period, s = 333, 272, 512, 136, 100, 0.5
    g = synth.gen(50, 1)
    dev = dict(device="cuda")
    W1, W2 = synth.trimodal_weight(d1, d0, seed=51).cuda(), synth.trimodal_weight(d2, d1, seed=52).cuda()
    X = synth.activations(T, d0, seed=53).cuda()
    H = torch.randn(T, d1, generator=g).to(torch.bfloat16).cuda()
    gains = [(1 + 0.1 * torch.randn(d1, generator=g)).to(torch.bfloat16).cuda() for _ in range(2)]
    gate = torch.randn(-(-T // period), d1, generator=g).to(torch.bfloat16).cuda()
    dY2 = synth.grad_output(T, d2, seed=54).cuda()
    dH_out = torch.randn(T, d1, generator=g).to(torch.bfloat16).cuda()
    L1, L2 = SparseBitLinearLayer(W1, 6, 8, keep_mask=True), SparseBitLinearLayer(W2, 6, 8, keep_mask=True)
    N = BlockNorm(gains[0], gains[1], max_tokens=T, res_scale=s)
    e = lambda *sh, dt=torch.float32: torch.empty(*sh, dtype=dt, **dev)  # noqa: E731
    Xq, amax, Y1, Y2 = e(T, d0, dt=torch.int8), e(T), e(T, d1), e(T, d2)
    dX2, dY1, dH, dX1 = e(T, d1), e(T, d1, dt=torch.bfloat16), e(T, d1, dt=torch.bfloat16), e(T, d0)
    dW1, dW2, dgate = e(d1, d0), e(d2, d1), e(*gate.shape)

    # forward
    L1.weight_step()
    L2.weight_step()
    act_quant(X, Xq, amax)
    L1.forward(Xq, amax, Y1)
    h1, xn, xq2, amax2 = N.forward(Y1, H, gate, period)
    L2.forward(xq2, amax2, Y2)
    # backward
    L2.backward(dY2, xn, dX2, dW2)
    N.backward([dX2], dH_out, Y1, dY1, dH, gate, period, dgate)
    L1.backward(dY1, X, dX1, dW1)
    clip = GradClip([dW1, dW2, N.dg_pre, N.dg_post, dgate])
    raw = [_f(t).copy() for t in (dW1, dW2, N.dg_pre, N.dg_post, dgate)]
    clip.clip(1.0)
    lib.sbl_check()

    ref = oracle.block_norm(_f(Y1), _f(H), _f(gains[0]), s, 1e-6, _f(gains[1]), _f(gate), period)
    assert np.array_equal(_f(h1), ref["h_out"]) and np.array_equal(synth.bits(xn.cpu()), ref["xn"])
    assert np.array_equal(xq2.cpu().numpy(), ref["xq"]) and np.array_equal(amax2.cpu().numpy(), ref["amax"])
    weff2, gamma2, _ = oracle.effective_weight(synth.bits(W2.cpu()), 6, 8)
    assert np.array_equal(Y2.cpu().numpy(), oracle.forward_out(oracle.forward_acc(ref["xq"], weff2), gamma2, ref["amax"]))
    dyb = synth.bits(dY2.cpu())
    check_bwd(_f(dX2), oracle.backward_dx(dyb, weff2, gamma2), abs_dx(dyb, weff2, gamma2), "dX2")
    check_bwd(raw[1], oracle.backward_dw(dyb, ref["xn"]), abs_dw(dyb, ref["xn"]), "dW2")
    b = oracle.block_norm_backward([_f(dX2)], _f(Y1), _f(h1), ref["r1"], ref["r2"], _f(gains[0]), s, _f(dH_out),
                                   _f(gains[1]), _f(gate), period)
    for name, got, K, bf16 in (("dy", _f(dY1), 64, True), ("dh", _f(dH), 64, True), ("dg_pre", raw[2], 192, False),
                               ("dg_post", raw[3], 192, False), ("dgate", raw[4], 192, False)):
        tol = K * U * b["abs"][name]
        if bf16:
            tol = tol + UB * (np.abs(b[name]) + tol)
        assert np.all(np.abs(got - b[name]) <= tol), name
    dyb1, xb = synth.bits(dY1.cpu()), synth.bits(X.cpu())
    weff1, gamma1, _ = oracle.effective_weight(synth.bits(W1.cpu()), 6, 8)
    check_bwd(_f(dX1), oracle.backward_dx(dyb1, weff1, gamma1), abs_dx(dyb1, weff1, gamma1), "dX1")
    check_bwd(raw[0], oracle.backward_dw(dyb1, xb), abs_dw(dyb1, xb), "dW1")
    S, norm, c, clipped = oracle.clip_grads(raw, 1.0)
    assert clip.sumsq.item() == pytest.approx(S, rel=1e-12) and clip.factor.item() == pytest.approx(float(c), rel=2 * U)
    for t, want in zip((dW1, dW2, N.dg_pre, N.dg_post, dgate), clipped):
        assert np.all(np.abs(_f(t) - want) <= 2 * U * np.abs(want) + 2.0 ** -149)

    # the clipped gradient through the optimizer, with no further clip
    m, v = torch.zeros(d1, d0, **dev), torch.zeros(d1, d0, **dev)
    before, grad = synth.bits(W1.cpu()), _f(dW1)
    lib.sbl_adamw_step(W1, None, dW1, m, v, d1, d0, 6, 8, 1e-3, 0.9, 0.95, 1e-5, 0.1, 1, None, 0.0, L1.W_eff,
                       L1.W_eff_bf16, L1.mask_bits, L1.gamma, None, L1.ws, L1.ws_bytes)
    lib.sbl_check()
    z = np.zeros((d1, d0), np.float32)
    step = oracle.adamw_weight_step(before, grad, z, z, 6, 8, oracle.adamw_scalars(1e-3, 0.9, 0.95, 1e-5, 0.1, 1))
    assert np.array_equal(synth.bits(W1.cpu()), step["w_bits"])
    assert np.array_equal(L1.W_eff.cpu().numpy(), step["weff"])


def test_int8_projection_trains(lib):
    """Forward in 8 bits, the straight-through gradients, an update of W and its new codes."""
    from semi_structured_sparsity_step_b200.layer import Int8Linear, act_quant
    T, d_in, d_out = 77, 272, 136
    w, x, dy = synth.normal_weight(d_out, d_in, seed=55), synth.activations(T, d_in, seed=56), \
        synth.grad_output(T, d_out, seed=57)
    L = Int8Linear(w.cuda())
    dev = dict(device="cuda")
    X, Xq, amax = x.cuda(), torch.empty(T, d_in, dtype=torch.int8, **dev), torch.empty(T, **dev)
    Y, dX, dW = torch.empty(T, d_out, **dev), torch.empty(T, d_in, **dev), torch.empty(d_out, d_in, **dev)
    act_quant(X, Xq, amax)
    L.forward(Xq, amax, Y)
    L.backward(dy.cuda(), X, dX, dW)
    lib.sbl_check()
    xq, am = oracle.act_quant(synth.bits(x))
    wq, wm = oracle.act_quant(synth.bits(w))
    assert np.array_equal(_f(Y), oracle.w8a8_out(oracle.forward_acc(xq, wq), am, wm))
    # dX = dY W: the oracle's product with W in the ternary weight's place and gamma = 1
    wf = w.float().numpy().astype(np.float64)
    ref = oracle.bf16_to_f32(synth.bits(dy)).astype(np.float64) @ wf
    check_bwd(_f(dX), ref, np.abs(oracle.bf16_to_f32(synth.bits(dy))).astype(np.float64) @ np.abs(wf), "dX")
    check_bwd(_f(dW), oracle.backward_dw(synth.bits(dy), synth.bits(x)), abs_dw(synth.bits(dy), synth.bits(x)), "dW")
    L.W.sub_((0.01 * dW).to(torch.bfloat16))
    L.weight_step()
    wq, wm = oracle.act_quant(synth.bits(L.W.cpu()))
    assert np.array_equal(L.Wq.cpu().numpy(), wq) and np.array_equal(L.wmax.cpu().numpy(), wm)


@pytest.mark.parametrize("batch", [1, 5])
def test_decode_step_in_a_graph(lib, batch):
    """Packed ternary projection, block norm, 8-bit head: one graph, replayed on new inputs."""
    from semi_structured_sparsity_step_b200.layer import BlockNorm, Int8Linear
    d0, d1, d2 = 512, 896, 4864
    dev = dict(device="cuda")
    weff = torch.randint(-1, 2, (d1, d0), generator=synth.gen(60, 2)).to(torch.int8)
    gamma = torch.tensor([0.02], **dev)
    dense = torch.empty(lib.sbl_dense2_bytes(d1, d0), dtype=torch.uint8, **dev)
    lib.sbl_pack_dense2(weff.cuda(), d1, d0, dense, dense.numel())
    head_w = synth.normal_weight(d2, d1, seed=61)
    head = Int8Linear(head_w.cuda())
    gain = (1 + 0.1 * torch.randn(d1, generator=synth.gen(60, 3))).to(torch.bfloat16).cuda()
    norm = BlockNorm(gain, None, max_tokens=batch)
    X = torch.zeros(batch, d0, dtype=torch.bfloat16, **dev)
    H = torch.zeros(batch, d1, dtype=torch.bfloat16, **dev)
    Xq, amax = torch.empty(batch, d0, dtype=torch.int8, **dev), torch.empty(batch, **dev)
    Y, out = torch.empty(batch, d1, **dev), torch.empty(batch, d2, **dev)

    def step():
        lib.sbl_act_quant(X, batch, d0, Xq, amax)
        lib.sbl_gemv_dense2_group([(dense, Xq, amax, gamma, Y, d0, d1)], batch)
        _, _, xq, am = norm.forward(Y, H)
        head.forward(xq, am, out)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    wq, wmax = oracle.act_quant(synth.bits(head_w))
    assert np.array_equal(head.Wq.cpu().numpy(), wq) and np.array_equal(head.wmax.cpu().numpy(), wmax)
    for k in range(3):
        x = synth.activations(batch, d0, seed=62 + k)
        h = synth.activations(batch, d1, seed=72 + k)
        X.copy_(x)
        H.copy_(h)
        graph.replay()
        torch.cuda.synchronize()
        lib.sbl_check()
        xq, am = oracle.act_quant(synth.bits(x))
        y = oracle.forward_out(oracle.forward_acc(xq, weff.numpy()), np.float32(gamma.item()), am)
        ref = oracle.block_norm(y, h.float().numpy(), _f(gain), 1.0, 1e-6)
        acc = oracle.forward_acc(ref["xq"], wq)
        assert np.array_equal(out.cpu().numpy(), oracle.w8a8_out(acc, ref["amax"], wmax))


def test_calls_on_two_streams_at_once(lib):
    """The same operators on two streams, each with buffers and workspace of its own."""
    from semi_structured_sparsity_step_b200.layer import BlockNorm, GradClip
    T, d = 2500, 1024
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    sets = []
    for k in range(2):
        g = torch.Generator(device="cuda").manual_seed(80 + k)
        r = lambda *sh: torch.randn(*sh, generator=g, device="cuda")  # noqa: E731
        n = BlockNorm((1 + 0.1 * r(d)).to(torch.bfloat16), (1 + 0.1 * r(d)).to(torch.bfloat16), max_tokens=T)
        sets.append(dict(n=n, Y=r(T, d), H=r(T, d).to(torch.bfloat16), dx=[r(T, d)], gate=r(25, d).to(torch.bfloat16),
                         dY=torch.empty(T, d, dtype=torch.bfloat16, device="cuda"), dgate=torch.empty(25, d, device="cuda")))

    def run(q):
        q["n"].forward(q["Y"], q["H"], q["gate"], 100)
        q["n"].backward(q["dx"], None, q["Y"], q["dY"], None, q["gate"], 100, q["dgate"])
        c = GradClip([q["n"].dg_pre, q["n"].dg_post, q["dgate"]])
        c.norm_only()
        return [q["n"].Xq.clone(), q["dY"].clone(), q["n"].dg_pre.clone(), q["dgate"].clone(), c.sumsq.clone()]

    alone = [run(q) for q in sets]
    torch.cuda.synchronize()
    for _ in range(3):
        both = [None, None]
        for k, (s, q) in enumerate(zip(streams, sets)):
            with torch.cuda.stream(s):
                both[k] = run(q)
        torch.cuda.synchronize()
        for a, b in zip(alone, both):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    lib.sbl_check()


# ---- positions past 32 bits: a block of rows repeated until the tensors hold more than 2^31 elements,
# so every later copy of the block has to come out as the first

def _repeats(base, times):
    return base.repeat(times, 1)


def test_block_norm_past_2_31_elements(lib):
    rows, times, d = 1000, 530, 4096  # 2.17e9 elements
    T = rows * times
    g = torch.Generator(device="cuda").manual_seed(90)
    r = lambda *sh: torch.randn(*sh, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    y, h, gate, gain = r(rows, d), r(rows, d), r(rows // 100, d), r(d)
    dev = dict(device="cuda")

    def call(times):
        T = rows * times
        Y, H, G = _repeats(y, times), _repeats(h, times), _repeats(gate, times)
        xn, xq = torch.empty(T, d, dtype=torch.bfloat16, **dev), torch.empty(T, d, dtype=torch.int8, **dev)
        amax = torch.empty(T, **dev)
        rstd = torch.empty(2 * T, **dev)
        lib.sbl_block_norm(Y, H, gain, G, 100, 0.5, gain, 1e-6, T, d, lib.SBL_BLOCK_Y_BF16, H, xn, xq, amax, rstd)
        return Y, H, G, xn, xq, amax, rstd

    _, H1, _, xn1, xq1, amax1, _ = call(1)
    Y, H, G, xn, xq, amax, rstd = call(times)
    lib.sbl_check()
    assert torch.equal(H.view(times, rows, d), H1.expand(times, rows, d))
    assert torch.equal(xq.view(times, rows, d), xq1.expand(times, rows, d))
    assert torch.equal(xn.view(times, rows, d), xn1.expand(times, rows, d))
    assert torch.equal(amax.view(times, rows), amax1.expand(times, rows))
    del xq, xq1
    # backward: every copy of the block gives the same dY and dgate rows
    dx = torch.randn(rows, d, generator=g, device="cuda")
    dX = _repeats(dx, times)
    dY = torch.empty(T, d, dtype=torch.bfloat16, **dev)
    dgate = torch.empty(T // 100, d, **dev)
    n = lib.sbl_block_norm_backward_workspace_bytes(d)
    ws = torch.empty(n, dtype=torch.uint8, **dev)
    lib.sbl_block_norm_backward([dX], None, Y, H, gain, G, 100, 0.5, gain, rstd, T, d, lib.SBL_BLOCK_Y_BF16, dY, None,
                                None, None, dgate, 0, ws, n)
    lib.sbl_check()
    assert torch.equal(dY.view(times, rows, d), dY[:rows].expand(times, rows, d))
    # every group of tokens is cut into the same segments, added up in the same order
    assert torch.equal(dgate.view(times, rows // 100, d), dgate[: rows // 100].expand(times, rows // 100, d))


def test_w8a8_past_2_31_outputs(lib):
    rows, times, d_in, d_out = 1024, 68, 64, 32768  # 2.28e9 outputs
    g = torch.Generator(device="cuda").manual_seed(91)
    x = torch.randint(-127, 128, (rows, d_in), generator=g, device="cuda", dtype=torch.int32).to(torch.int8)
    w = torch.randint(-127, 128, (d_out, d_in), generator=g, device="cuda", dtype=torch.int32).to(torch.int8)
    am, wm = torch.rand(rows, generator=g, device="cuda"), torch.rand(d_out, generator=g, device="cuda")
    T = rows * times
    Y = torch.empty(T, d_out, dtype=torch.bfloat16, device="cuda")
    lib.sbl_forward_w8a8(_repeats(x, times), am.repeat(times), w, wm, T, d_in, d_out, lib.SBL_W8A8_Y_BF16, Y)
    one = torch.empty(rows, d_out, dtype=torch.bfloat16, device="cuda")
    lib.sbl_forward_w8a8(x, am, w, wm, rows, d_in, d_out, lib.SBL_W8A8_Y_BF16, one)
    lib.sbl_check()
    assert torch.equal(Y.view(times, rows, d_out), one.expand(times, rows, d_out))


def test_clip_past_2_32_elements(lib):
    n = 2 ** 32 + 5
    g = torch.full((n,), 2.0 ** -17, dtype=torch.bfloat16, device="cuda")
    g[-1] = 3.0
    s, nm, c = torch.empty(1, dtype=torch.float64, device="cuda"), torch.empty(1, device="cuda"), \
        torch.empty(1, device="cuda")
    nb = lib.sbl_grad_group_workspace_bytes(1)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    lib.sbl_grad_clip_group([(g, g, n, True)], 1.0, s, nm, c, ws, nb)
    lib.sbl_check()
    S = (n - 1) * 2.0 ** -34 + 9.0  # exact in fp64
    assert s.item() == pytest.approx(S, rel=1e-13)
    factor = np.float32(1.0 / (np.sqrt(S) + 1e-6))
    assert c.item() == pytest.approx(float(factor), rel=2.0 ** -23)
    want = torch.tensor([3.0 * c.item(), 2.0 ** -17 * c.item()]).to(torch.bfloat16).cuda()
    assert g[-1] == want[0] and torch.all(g[:-1] == want[1])


def test_stream_argument_and_refused_tensors(lib):
    """Every call takes a stream, as an object or a handle; tensors that it would misread are refused
    before a launch."""
    T, d = 37, 256
    dev = dict(device="cuda")
    Y, H = torch.randn(T, d, **dev), torch.randn(T, d, **dev).to(torch.bfloat16)
    gain = torch.ones(d, dtype=torch.bfloat16, **dev)
    W, wmax = torch.ones(64, d, dtype=torch.int8, **dev), torch.ones(64, **dev)
    n = lib.sbl_block_norm_backward_workspace_bytes(d)
    ws = torch.empty(n, dtype=torch.uint8, **dev)

    def run(stream):
        o = dict(h=torch.zeros_like(H), xq=torch.zeros(T, d, dtype=torch.int8, **dev), am=torch.zeros(T, **dev),
                 r=torch.zeros(2 * T, **dev), out=torch.zeros(T, 64, **dev), dY=torch.zeros_like(H),
                 dg=torch.zeros(d, **dev), s=torch.zeros(1, dtype=torch.float64, **dev), c=torch.zeros(d, **dev))
        torch.cuda.synchronize()  # the buffers were filled on the current stream
        lib.sbl_block_norm(Y, H, gain, None, 0, 1.0, gain, 1e-6, T, d, 0, o["h"], None, o["xq"], o["am"], o["r"], stream)
        lib.sbl_forward_w8a8(o["xq"], o["am"], W, wmax, T, d, 64, 0, o["out"], stream)
        lib.sbl_block_norm_backward([Y], None, Y, o["h"], gain, None, 0, 1.0, gain, o["r"], T, d, 0, o["dY"], None,
                                    o["dg"], None, None, 0, ws, n, stream)
        lib.sbl_grad_clip_group([(o["dg"], o["c"], d, False)], 1.0, o["s"], None, None, ws, n, stream)
        torch.cuda.synchronize()
        return o

    side = torch.cuda.Stream()
    want = run(None)
    for stream in (side, side.cuda_stream):
        got = run(stream)
        assert all(torch.equal(got[k], want[k]) for k in want)
    o = want
    bad = [torch.zeros(T, d), Y.to(torch.bfloat16), Y.t().contiguous().t(), Y[:-1]]  # host, type, strides, size
    for b in bad:
        with pytest.raises(lib.SblError):
            lib.sbl_block_norm(b, H, gain, None, 0, 1.0, gain, 1e-6, T, d, 0, o["h"], None, o["xq"], o["am"], o["r"])
        with pytest.raises(lib.SblError):
            lib.sbl_block_norm_backward([b], None, Y, o["h"], gain, None, 0, 1.0, gain, o["r"], T, d, 0, o["dY"], None,
                                        o["dg"], None, None, 0, ws, n)
        with pytest.raises(lib.SblError):
            lib.sbl_grad_clip_group([(b, Y, T * d, False)], 1.0, o["s"], None, None, ws, n)
        with pytest.raises(lib.SblError):
            lib.sbl_forward_w8a8(o["xq"], o["am"], W, wmax, T, d, 64, 0, b[:, :64])
    with pytest.raises(lib.SblError):  # a workspace shorter than it is said to be
        lib.sbl_grad_clip_group([(Y, Y, T * d, False)], 1.0, o["s"], None, None, ws[:64], n)
    lib.sbl_check()
