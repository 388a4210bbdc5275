"""The gradient norm over many tensors and the clipped gradients, against the CPU oracle.

S differs from the oracle's correctly rounded sum by fp64 summation order alone (rel 1e-12 over
these sizes); norm, clip and the fp32 products are then at most one fp32 rounding step away, and a
bf16 output one bf16 rounding (half a step, 2^-8 of the value) more.
"""
import numpy as np
import pytest
import torch

import oracle
import synth

pytestmark = pytest.mark.gpu

U32, U16 = 2.0 ** -23, 2.0 ** -8


def _grads(sizes, bf16, seed, scale=1e-2):
    """Device buffers that end 8 elements after the gradient, with a guard value there."""
    out = []
    for i, (n, b) in enumerate(zip(sizes, bf16)):
        g = synth.optimizer_state(1, max(n, 1), seed=seed + i, g_std=scale)[0].reshape(-1)[:n]
        buf = torch.full((n + 8,), 7.0, dtype=torch.bfloat16 if b else torch.float32, device="cuda")
        buf[:n] = g.cuda()
        out.append(buf)
    return out


class Clip:
    def __init__(self, lib, count):
        self.lib = lib
        self.bytes = lib.sbl_grad_group_workspace_bytes(count)
        self.ws = torch.full((self.bytes,), 255, dtype=torch.uint8, device="cuda")
        self.sumsq = torch.full((1,), -1.0, dtype=torch.float64, device="cuda")
        self.norm = torch.full((1,), -1.0, device="cuda")
        self.clip = torch.full((1,), -1.0, device="cuda")

    def __call__(self, tensors, max_norm):
        self.lib.sbl_grad_clip_group(tensors, max_norm, self.sumsq, self.norm, self.clip, self.ws, self.bytes)


def _check(c, bufs, outs, sizes, bf16, max_norm):
    host = [b[:n].float().cpu().numpy() for b, n in zip(bufs, sizes)]
    S, norm, clip, ref = oracle.clip_grads(host, max_norm)
    assert c.sumsq.item() == pytest.approx(S, rel=1e-12)
    assert c.norm.item() == pytest.approx(float(norm), rel=U32)
    assert c.clip.item() == pytest.approx(float(clip), rel=U32)
    for o, r, n, b in zip(outs, ref, sizes, bf16):
        got = o[:n].float().cpu().numpy()
        assert np.all(np.abs(got - r) <= (U32 + (U16 if b else 0.0)) * np.abs(r) + 2.0 ** -149)
        assert torch.all(o[n:] == 7.0)  # nothing behind the end


# 4096 fp32 or 8192 bf16 elements are one tile of the kernels
SIZES = [1, 3, 4, 5, 0, 4095, 4096, 4097, 8191, 8192, 8193, 100003, 2048, 7]


@pytest.mark.parametrize("kind", ["f32", "bf16", "mixed"])
@pytest.mark.parametrize("max_norm", [0.5, 1e6])
def test_clip_ragged_sizes(lib, kind, max_norm):
    bf16 = [{"f32": False, "bf16": True, "mixed": i % 2 == 1}[kind] for i in range(len(SIZES))]
    bufs = _grads(SIZES, bf16, 100)
    outs = [torch.full_like(b, 7.0) for b in bufs]
    c = Clip(lib, len(SIZES))
    c([(b, o, n, f) for b, o, n, f in zip(bufs, outs, SIZES, bf16)], max_norm)
    lib.sbl_check()
    _check(c, bufs, outs, SIZES, bf16, max_norm)
    if max_norm == 1e6:
        assert c.clip.item() == 1.0
        for b, o in zip(bufs, outs):
            assert torch.equal(b, o)


def test_clip_more_tensors_than_one_launch_and_more_tiles_than_blocks(lib):
    sizes = [(37 * i) % 3001 for i in range(300)] + [5_000_001, 1]
    bf16 = [i % 3 == 0 for i in range(len(sizes))]
    bufs = _grads(sizes, bf16, 500, scale=1e-3)
    outs = [torch.full_like(b, 7.0) for b in bufs]
    c = Clip(lib, len(sizes))
    args = [(b, o, n, f) for b, o, n, f in zip(bufs, outs, sizes, bf16)]
    c(args, 0.25)
    _check(c, bufs, outs, sizes, bf16, 0.25)
    s = torch.empty(1, dtype=torch.float64, device="cuda")
    n = torch.empty(1, device="cuda")
    lib.sbl_grad_norm_group([(b, None, k, f) for b, k, f in zip(bufs, sizes, bf16)], s, n, c.ws, c.bytes)
    assert s.item() == c.sumsq.item() and n.item() == c.norm.item()  # the same bits
    c(args, 0.25)
    assert s.item() == c.sumsq.item()


def test_clip_in_place_and_below_the_limit_leaves_the_bits(lib):
    sizes, bf16 = [1000, 4099], [False, True]
    bufs = _grads(sizes, bf16, 700)
    before = [b.clone() for b in bufs]
    c = Clip(lib, 2)
    c([(b, b, n, f) for b, n, f in zip(bufs, sizes, bf16)], 1e6)
    assert all(torch.equal(a, b) for a, b in zip(bufs, before))
    c([(b, b, n, f) for b, n, f in zip(bufs, sizes, bf16)], 0.125)
    _check(c, before, bufs, sizes, bf16, 0.125)


def test_clip_of_nothing(lib):
    c = Clip(lib, 0)
    c([], 1.0)
    assert (c.sumsq.item(), c.norm.item(), c.clip.item()) == (0.0, 0.0, 1.0)
    e = torch.empty(0, device="cuda")
    c = Clip(lib, 1)
    c([(e, e, 0, False)], 1.0)
    assert (c.sumsq.item(), c.norm.item(), c.clip.item()) == (0.0, 0.0, 1.0)
    lib.sbl_grad_norm_group([], c.sumsq, c.norm, c.ws, c.bytes)
    assert (c.sumsq.item(), c.norm.item()) == (0.0, 0.0)


def test_clip_with_nan_infinity_and_large_values(lib):
    g = torch.ones(5000, device="cuda")
    h = torch.ones(33, dtype=torch.bfloat16, device="cuda")
    c = Clip(lib, 2)
    og, oh = torch.zeros_like(g), torch.zeros_like(h)
    g[77] = 3e38  # its square does not fit fp32
    c([(g, og, 5000, False), (h, oh, 33, True)], 1.0)
    assert c.norm.item() == pytest.approx(3e38, rel=1e-6) and og[77].item() == pytest.approx(1.0, rel=1e-6)
    g[77] = float("inf")
    c([(g, og, 5000, False), (h, oh, 33, True)], 1.0)
    assert c.norm.item() == float("inf") and c.clip.item() == 0.0
    assert torch.isnan(og[77]) and og[76].item() == 0.0 and torch.all(oh == 0)
    g[77] = float("nan")
    c([(g, og, 5000, False), (h, oh, 33, True)], 1.0)
    assert torch.isnan(c.norm).item() and torch.isnan(c.clip).item()
    assert torch.isnan(og).all() and torch.isnan(oh).all()


def test_clip_captured_and_replayed_on_another_stream(lib):
    sizes, bf16 = [4097, 513], [False, True]
    bufs = _grads(sizes, bf16, 900)
    outs = [torch.full_like(b, 7.0) for b in bufs]
    c = Clip(lib, 2)
    args = [(b, o, n, f) for b, o, n, f in zip(bufs, outs, sizes, bf16)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            c(args, 0.5)
    for k in range(3):
        for b, n in zip(bufs, sizes):
            b[:n] *= 1.5
        graph.replay()
        torch.cuda.synchronize()
        _check(c, bufs, outs, sizes, bf16, 0.5)


def test_group_norm_feeds_the_optimizer_step(lib):
    """S of sbl_grad_norm_group in the place of sbl_grad_sqnorm's: the same AdamW step."""
    d_out, d_in = 136, 272
    w = synth.trimodal_weight(d_out, d_in, seed=41)
    dw, m0, v0 = synth.optimizer_state(d_out, d_in, seed=41, g_std=1.0)
    extra = torch.randn(777, generator=synth.gen(41, 9)).cuda()
    dW = dw.cuda()
    ws_bytes = max(lib.sbl_mask_quant_workspace_bytes(d_out, d_in), lib.sbl_grad_group_workspace_bytes(2))
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device="cuda")
    S = torch.empty(1, dtype=torch.float64, device="cuda")
    lib.sbl_grad_norm_group([(dW, None, dW.numel(), False), (extra, None, 777, False)], S, None, ws, ws_bytes)
    W, m, v = w.cuda(), m0.cuda(), v0.cuda()
    weff = torch.empty(d_out, d_in, dtype=torch.int8, device="cuda")
    bits = torch.empty(d_out, d_in // 8, dtype=torch.uint8, device="cuda")
    gamma = torch.empty(1, device="cuda")
    lib.sbl_adamw_step(W, None, dW, m, v, d_out, d_in, 6, 8, 1e-3, 0.9, 0.95, 1e-5, 0.1, 1, S, 1.0, weff, None, bits,
                       gamma, None, ws, ws_bytes)
    lib.sbl_check()
    c = oracle.grad_clip_scale(oracle.grad_sqnorm(dw.numpy(), extra.cpu().numpy()), 1.0)
    assert c < 1.0
    ref = oracle.adamw_weight_step(synth.bits(w), dw.numpy(), m0.numpy(), v0.numpy(), 6, 8,
                                   oracle.adamw_scalars(1e-3, 0.9, 0.95, 1e-5, 0.1, 1), c)
    assert np.array_equal(synth.bits(W.cpu()), ref["w_bits"]) and np.array_equal(weff.cpu().numpy(), ref["weff"])


def test_a_gradient_listed_twice_counts_twice(lib):
    sizes, kinds = [4097, 4097, 5], [False, False, True]
    a, b = _grads([4097, 5], [False, True], seed=77)
    bufs, outs = [a, a, b], [torch.full_like(x, 7.0) for x in (a, a, b)]
    c = Clip(lib, 3)
    tensors = [(g, o, n, k) for g, o, n, k in zip(bufs, outs, sizes, kinds)]
    c(tensors, 0.25)
    _check(c, bufs, outs, sizes, kinds, 0.25)
    with pytest.raises(lib.SblError):
        c([(a, a, 4097, False), (a, a, 4097, False)], 0.25)
