"""The block norm's layer helper on another stream than the current one."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("handle", [False, True])
def test_workspace_of_the_first_backward_is_no_memory_in_use(lib, handle):
    """A tensor freed on the current stream, whose last reader there has not run yet, keeps its values."""
    from semi_structured_sparsity_step_b200.layer import BlockNorm
    T, d = 700, 2048
    dev = dict(device="cuda")
    side = torch.cuda.Stream()
    gain = torch.ones(d, dtype=torch.bfloat16, **dev)
    Y, dx = torch.randn(T, d, **dev), torch.randn(T, d, **dev)
    H = torch.randn(T, d, **dev).to(torch.bfloat16)
    dY = torch.empty(T, d, dtype=torch.bfloat16, **dev)
    N = BlockNorm(gain, gain, max_tokens=T)
    out = torch.zeros(N.ws_bytes, dtype=torch.uint8, **dev)
    N.forward(Y, H)
    torch.cuda.synchronize()
    x = torch.full((N.ws_bytes,), 3, dtype=torch.uint8, **dev)
    torch.cuda.synchronize()
    torch.cuda._sleep(40_000_000)  # about 20 ms of the current stream
    out.copy_(x)
    del x  # what the allocator gives to the next request of the current stream
    N.backward([dx], None, Y, dY, None, stream=side.cuda_stream if handle else side)
    torch.cuda.synchronize()
    assert torch.all(out == 3)
    lib.sbl_check()


def test_a_captured_fork_and_join(lib):
    """The norm on one stream, two products of its codes on two, and the clip of both outputs behind the join, in
    one graph: every launch that may start early waits for all that it reads."""
    T, d, d1, d2, rounds = 24, 1024, 2048, 11008, 4
    g = torch.Generator(device="cuda").manual_seed(5)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    bf, i8 = torch.bfloat16, torch.int8
    Y, H, gain = rnd(T, d), rnd(T, d).to(bf), (1 + 0.1 * rnd(d)).to(bf)
    W = [torch.randint(-127, 128, (n, d), generator=g, device="cuda", dtype=torch.int32).to(i8) for n in (d1, d2)]
    wmax = [torch.rand(n, generator=g, device="cuda") for n in (d1, d2)]
    ws = torch.empty(lib.sbl_grad_group_workspace_bytes(2), dtype=torch.uint8, device="cuda")
    xq, amax = torch.empty(T, d, dtype=i8, device="cuda"), torch.empty(T, device="cuda")
    outs = [torch.empty(T, n, device="cuda") for n in (d1, d2)]
    clipped = [torch.empty_like(o) for o in outs]
    S, norm, factor = torch.empty(1, dtype=torch.float64, device="cuda"), torch.empty(1, device="cuda"), \
        torch.empty(1, device="cuda")
    side = torch.cuda.Stream()

    def step(between, other):
        main = torch.cuda.current_stream()
        lib.sbl_block_norm(Y, H, gain, None, 0, 0.5, gain, 1e-6, T, d, 0, H, None, xq, amax, None)
        between()
        other.wait_stream(main)
        lib.sbl_forward_w8a8(xq, amax, W[0], wmax[0], T, d, d1, 0, outs[0], other)
        between()
        lib.sbl_forward_w8a8(xq, amax, W[1], wmax[1], T, d, d2, 0, outs[1])
        between()
        main.wait_stream(other)
        lib.sbl_grad_clip_group([(o, c, o.numel(), False) for o, c in zip(outs, clipped)], 1.0, S, norm, factor, ws,
                                ws.numel())
        between()

    def state():
        return [t.clone() for t in (H, xq, amax, *outs, *clipped, S, norm, factor)]

    h0 = H.clone()
    want = []
    for _ in range(rounds):  # in place on H: every round has other inputs
        step(torch.cuda.synchronize, side)
        want.append(state())
    H.copy_(h0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(lambda: None, side)
    H.copy_(h0)
    for k in range(rounds):
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(state(), want[k]))
    lib.sbl_check()
