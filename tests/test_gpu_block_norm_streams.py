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
