"""The 8-bit product against the CPU oracle: bit for bit in fp32, and the oracle's value rounded to
bf16 for a bf16 output (exact int32 sums and the same fp32 operations on both sides)."""
import numpy as np
import pytest
import torch

import oracle
import synth

pytestmark = pytest.mark.gpu


def _codes(shape, seed, full=False):
    g = synth.gen(seed, 17)
    lo, hi = (-128, 128) if full else (-127, 128)
    return torch.randint(lo, hi, shape, generator=g, dtype=torch.int32).to(torch.int8)


def _acc(xq, wq):
    """Exact: every product and partial sum is an integer below 2^53 in fp64."""
    return (xq.double() @ wq.double().t()).numpy().astype(np.int64)


def _run(lib, T, d_in, d_out, bf16, seed=0, full=False, sample=None):
    xq, wq = _codes((T, d_in), seed, full), _codes((d_out, d_in), seed + 1, full)
    g = synth.gen(seed, 18)
    amax, wmax = torch.rand(T, generator=g) * 4 + 0.1, torch.rand(d_out, generator=g) * 0.1 + 0.001
    Y = torch.full((T + 1, d_out), 77, dtype=torch.bfloat16 if bf16 else torch.float32, device="cuda")
    lib.sbl_forward_w8a8(xq.cuda(), amax.cuda(), wq.cuda(), wmax.cuda(), T, d_in, d_out,
                         lib.SBL_W8A8_Y_BF16 if bf16 else 0, Y)
    lib.sbl_check()
    assert torch.all(Y[T:] == 77)
    rows = np.arange(T) if sample is None else np.unique(np.linspace(0, T - 1, sample).astype(int))
    acc = _acc(xq[rows], wq)
    assert np.abs(acc).max(initial=0) < 2 ** 31
    ref = oracle.w8a8_out(acc.astype(np.int32), amax.numpy()[rows], wmax.numpy())
    got = Y[:T][torch.from_numpy(rows).cuda()].cpu()
    if bf16:
        assert np.array_equal(synth.bits(got), oracle.f32_to_bf16(ref))
    else:
        assert np.array_equal(got.numpy(), ref)


# borders of the token tiles (16, 32, 64, 128, 256), of the 128-row weight tiles and of the 128-byte K blocks
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 32, 33, 64, 65, 127, 128, 129, 256, 257, 300])
@pytest.mark.parametrize("d_in,d_out", [(16, 8), (128, 128), (144, 136), (2048, 264), (4112, 1000)])
@pytest.mark.parametrize("bf16", [False, True])
def test_every_token_tile(lib, T, d_in, d_out, bf16):
    _run(lib, T, d_in, d_out, bf16, seed=T)


@pytest.mark.parametrize("d_in", [16, 128, 240, 256, 272, 512, 1040, 2064, 11008])
def test_every_split_of_k(lib, d_in):
    for d_out in (8, 256, 2048, 11008):
        _run(lib, 3, d_in, d_out, False, seed=d_in)


@pytest.mark.parametrize("T,d_in,d_out,bf16", [(509, 2048, 2048, False), (1000, 272, 5000, True), (4097, 528, 2056, True),
                                               (2304, 64, 2304, False), (8192, 256, 1032, True)])
def test_full_batches(lib, T, d_in, d_out, bf16):
    """Past the border to the CTA-pair kernel (74 tiles of 256 x 256) and just before it."""
    _run(lib, T, d_in, d_out, bf16, seed=T, sample=200)


# Token tile and K splits that the plan takes there: 32 (1 to 8 splits), 64, 128, 256 (1 to 5), CTA pairs.
STREAMED = [(1451, 16, 160, 0), (168, 16, 3416, 1), (17, 2016, 6816, 0), (958, 2288, 24, 0), (771, 2112, 32, 1),
            (551, 3120, 16, 1), (552, 2720, 16, 0), (476, 2640, 16, 1), (437, 3616, 16, 0), (260, 16, 4520, 0),
            (70, 2064, 3456, 1), (1913, 4128, 16, 0), (1722, 4896, 16, 1), (1462, 4816, 16, 0), (1282, 4496, 16, 1),
            (1102, 7760, 16, 1), (943, 5856, 16, 0), (500, 16, 4848, 0), (325, 16, 7040, 1), (143, 3424, 3184, 0),
            (66, 3152, 4424, 1), (65, 4112, 3552, 1), (2505, 9248, 24, 0), (2803, 9616, 16, 1), (70, 6976, 2000, 0),
            (65, 7808, 1776, 1), (462, 528, 4776, 0), (131, 5808, 6376, 1), (131, 4976, 5264, 0), (130, 7056, 3896, 1),
            (131, 8320, 3176, 0), (265, 1168, 6808, 0), (2634, 16, 2112, 1)]


@pytest.mark.parametrize("T,d_in,d_out,bf16", STREAMED)
def test_every_tile_and_split_of_the_plan(lib, T, d_in, d_out, bf16):
    _run(lib, T, d_in, d_out, bool(bf16), seed=d_in + T)


def test_the_two_kernels_agree(lib):
    """The same tokens in a short and in a full batch."""
    d_in, d_out = 1040, 5000
    xq, wq = _codes((1024, d_in), 3).cuda(), _codes((d_out, d_in), 4).cuda()
    amax, wmax = torch.rand(1024, device="cuda") + 0.1, torch.rand(d_out, device="cuda") + 0.1
    full = torch.empty(1024, d_out, device="cuda")
    lib.sbl_forward_w8a8(xq, amax, wq, wmax, 1024, d_in, d_out, 0, full)
    for T in (1, 20, 70, 200):
        part = torch.empty(T, d_out, device="cuda")
        lib.sbl_forward_w8a8(xq, amax, wq, wmax, T, d_in, d_out, 0, part)
        assert torch.equal(part, full[:T])


def test_largest_sums(lib):
    """Every code -128: sums of 16384 per term, up to the int32 limit at the largest d_in."""
    for d_in in (1024, 131056):
        for T in (2, 300):
            x = torch.full((T, d_in), -128, dtype=torch.int8, device="cuda")
            w = torch.full((40, d_in), -128, dtype=torch.int8, device="cuda")
            amax, wmax = torch.full((T,), 127.0, device="cuda"), torch.full((40,), 127.0, device="cuda")
            Y = torch.empty(T, 40, device="cuda")
            lib.sbl_forward_w8a8(x, amax, w, wmax, T, d_in, 40, 0, Y)
            assert torch.all(Y == float(np.float32(16384 * d_in)))
    _run(lib, 5, 4096, 512, False, seed=9, full=True)


def test_nan_scale_stays_in_its_row_and_zero_work(lib):
    xq, wq = _codes((4, 64), 5).cuda(), _codes((24, 64), 6).cuda()
    amax, wmax = torch.ones(4, device="cuda"), torch.ones(24, device="cuda")
    amax[2] = float("nan")
    Y = torch.empty(4, 24, device="cuda")
    lib.sbl_forward_w8a8(xq, amax, wq, wmax, 4, 64, 24, 0, Y)
    assert torch.isnan(Y[2]).all() and torch.isfinite(Y[[0, 1, 3]]).all()
    keep = Y.clone()
    lib.sbl_forward_w8a8(xq, amax, wq, wmax, 0, 64, 24, 0, Y)
    lib.sbl_forward_w8a8(xq, amax, wq, wmax, 4, 64, 0, 0, Y)
    assert torch.equal(Y.nan_to_num(5.0), keep.nan_to_num(5.0))


def test_many_products_back_to_back_on_two_streams_and_in_a_graph(lib):
    """Dependent launches: each product reads what the previous kernels of its stream wrote."""
    d = 512
    w = synth.normal_weight(d, d, seed=21)
    Wq = torch.empty(d, d, dtype=torch.int8, device="cuda")
    wmax = torch.empty(d, device="cuda")
    lib.sbl_act_quant(w.cuda(), d, d, Wq, wmax)
    x = [synth.activations(33, d, seed=22 + k).cuda() for k in range(2)]

    def chain(x, out):
        xq = torch.empty(33, d, dtype=torch.int8, device="cuda")
        amax = torch.empty(33, device="cuda")
        for y in out:
            lib.sbl_act_quant(x, 33, d, xq, amax)
            lib.sbl_forward_w8a8(xq, amax, Wq, wmax, 33, d, d, lib.SBL_W8A8_Y_BF16, y)
            x = y

    def buffers():
        return [torch.empty(33, d, dtype=torch.bfloat16, device="cuda") for _ in range(8)]

    outs = [buffers(), buffers()]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for s, xk, o in zip(streams, x, outs):
        with torch.cuda.stream(s):
            chain(xk, o)
    torch.cuda.synchronize()
    lib.sbl_check()
    wq, wm = Wq.cpu(), wmax.cpu().numpy()
    for xk, o in zip(x, outs):
        cur = xk.cpu()
        for y in o:
            xq, amax = oracle.act_quant(synth.bits(cur))
            ref = oracle.f32_to_bf16(oracle.w8a8_out(_acc(torch.from_numpy(xq), wq).astype(np.int32), amax, wm))
            assert np.array_equal(synth.bits(y.cpu()), ref)
            cur = synth.from_bits(ref)
    again = buffers()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain(x[0], again)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(again, outs[0]))


def test_the_head_of_a_block(lib):
    """Block norm, 8-bit product: the codes that the norm writes go straight into it."""
    T, d, d_out = 19, 896, 4864
    g = synth.gen(30, 1)
    Y, H = torch.randn(T, d, generator=g), torch.randn(T, d, generator=g).to(torch.bfloat16)
    gain = (1 + 0.1 * torch.randn(d, generator=g)).to(torch.bfloat16)
    w = synth.normal_weight(d_out, d, seed=31)
    dev = dict(device="cuda")
    h1, xq, amax = torch.empty(T, d, dtype=torch.bfloat16, **dev), torch.empty(T, d, dtype=torch.int8, **dev), \
        torch.empty(T, **dev)
    Wq, wmax, out = torch.empty(d_out, d, dtype=torch.int8, **dev), torch.empty(d_out, **dev), torch.empty(T, d_out, **dev)
    lib.sbl_act_quant(w.cuda(), d_out, d, Wq, wmax)
    lib.sbl_block_norm(Y.cuda(), H.cuda(), None, None, 0, 1.0, gain.cuda(), 1e-6, T, d, 0, h1, None, xq, amax, None)
    lib.sbl_forward_w8a8(xq, amax, Wq, wmax, T, d, d_out, 0, out)
    lib.sbl_check()
    ref = oracle.block_norm(Y.numpy(), H.float().numpy(), gain.float().numpy(), 1.0, 1e-6)
    wq, wm = oracle.act_quant(synth.bits(w))
    acc = _acc(torch.from_numpy(ref["xq"]), torch.from_numpy(wq)).astype(np.int32)
    assert np.array_equal(out.cpu().numpy(), oracle.w8a8_out(acc, ref["amax"], wm))
