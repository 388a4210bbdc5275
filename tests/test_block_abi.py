"""Refusals of the block norm and the group clip: on the host, before a device is needed."""
import ctypes
import math

import pytest


@pytest.fixture(scope="module")
def cl():
    from semi_structured_sparsity_step_b200 import build
    build.build()
    from semi_structured_sparsity_step_b200 import _binding
    return _binding.load()


AL = 1 << 12  # a fake aligned address: never dereferenced on these paths


def _norm(cl, **kw):
    a = dict(Y=AL, H=AL, g_post=AL, gate=None, period=0, s=1.0, g_pre=AL, eps=1e-6, T=4, d=32, flags=0, H_out=AL,
             Xn=AL, Xq=AL, amax=AL, rstd=AL)
    a.update(kw)
    return cl.sbl_block_norm(*a.values(), None)


@pytest.mark.parametrize("status,kw", [
    (1, dict(flags=4)), (1, dict(eps=0.0)), (1, dict(eps=math.nan)), (1, dict(s=math.inf)), (1, dict(s=math.nan)),
    (1, dict(gate=AL, period=0)), (1, dict(gate=AL, period=-1)), (1, dict(Y=None)), (1, dict(H=None)),
    (1, dict(H_out=None)), (1, dict(g_pre=None)), (1, dict(Xq=None)), (1, dict(amax=None)),
    (2, dict(T=-1)), (2, dict(T=2 ** 30 + 1)), (2, dict(d=24)), (2, dict(d=0)), (2, dict(d=-16)), (2, dict(d=16400)),
    (3, dict(Y=AL + 8)), (3, dict(H=AL + 4)), (3, dict(gate=AL + 2, period=1)), (3, dict(rstd=AL + 4)),
    (3, dict(Xn=AL + 8)), (0, dict(T=0)),
])
def test_block_norm_refuses(cl, status, kw):
    assert _norm(cl, **kw) == status


def _bwd(cl, readers=1, n_ptr=None, **kw):
    ptrs = (ctypes.c_void_p * 4)(*([AL] * 4 if n_ptr is None else n_ptr))
    a = dict(dXn=ctypes.addressof(ptrs), readers=readers, dH_out=AL, Y=AL, H_out=AL, g_post=AL, gate=None, period=0,
             s=1.0, g_pre=AL, rstd=AL, T=4, d=32, flags=0, dY=AL, dH=AL, dg_post=AL, dg_pre=AL, dgate=None, acc=0,
             ws=AL, ws_bytes=1 << 30)
    a.update(kw)
    return cl.sbl_block_norm_backward(*a.values(), None)


@pytest.mark.parametrize("status,kw", [
    (1, dict(readers=0)), (1, dict(readers=4)), (1, dict(dXn=None)), (1, dict(readers=2, n_ptr=[AL, None, AL, AL])),
    (1, dict(flags=8)), (1, dict(acc=2)), (1, dict(g_post=None)), (1, dict(dgate=AL)), (1, dict(s=math.inf)),
    (1, dict(Y=None)), (1, dict(H_out=None)), (1, dict(rstd=None)), (1, dict(dY=None)), (1, dict(ws=None)),
    (1, dict(gate=AL, period=0)),
    (1, dict(Y=None, g_post=None, dg_post=None, gate=AL, period=2, dgate=AL)), (2, dict(T=-1)), (2, dict(d=8)), (2, dict(d=16400)),
    (3, dict(Y=AL + 8)), (3, dict(n_ptr=[AL + 4, AL, AL, AL])), (3, dict(ws=AL + 16)), (3, dict(dg_pre=AL + 4)),
    (5, dict(ws_bytes=16)),
])
def test_block_norm_backward_refuses(cl, status, kw):
    assert _bwd(cl, **kw) == status


def test_block_norm_backward_workspace(cl):
    assert cl.sbl_block_norm_backward_workspace_bytes(0) == 0
    assert cl.sbl_block_norm_backward_workspace_bytes(20) == 0
    assert cl.sbl_block_norm_backward_workspace_bytes(16400) == 0
    for d in (16, 256, 272, 896, 2048, 2064, 8192, 16384):
        assert 0 < cl.sbl_block_norm_backward_workspace_bytes(d) <= 64 << 20


def _clip(cl, tensors, count=None, max_norm=1.0, sumsq=AL, norm=AL, clip=AL, ws=AL, ws_bytes=1 << 30):
    from semi_structured_sparsity_step_b200 import _binding as B
    arr = (B.GradTensor * max(1, len(tensors)))(*[B.GradTensor(*t) for t in tensors])
    return cl.sbl_grad_clip_group(ctypes.addressof(arr), len(tensors) if count is None else count, max_norm, sumsq,
                                  norm, clip, ws, ws_bytes, None)


@pytest.mark.parametrize("status,tensors,kw", [
    (1, [(AL, AL, 4, 2, 0)], {}), (1, [(AL, AL, 4, 0, 7)], {}), (1, [(None, AL, 4, 0, 0)], {}),
    (1, [(AL, None, 4, 0, 0)], {}), (1, [], dict(count=-1)), (1, [(AL, AL, 4, 0, 0)], dict(max_norm=0.0)),
    (1, [(AL, AL, 4, 0, 0)], dict(max_norm=math.nan)), (1, [(AL, AL, 4, 0, 0)], dict(sumsq=None)),
    (1, [(AL, AL, 4, 0, 0)], dict(ws=None)), (2, [(AL, AL, 1 << 41, 0, 0)], {}),
    (3, [(AL + 8, AL, 4, 0, 0)], {}), (3, [(AL, AL + 4, 4, 1, 0)], {}), (3, [(AL, AL, 4, 0, 0)], dict(sumsq=AL + 4)),
    (3, [(AL, AL, 4, 0, 0)], dict(ws=AL + 16)), (3, [(AL, AL, 4, 0, 0)], dict(clip=AL + 2)),
    (5, [(AL, AL, 4, 0, 0)], dict(ws_bytes=64)), (5, [(AL, AL, 4, 0, 0)] * 200, dict(ws_bytes=1 << 14)),
])
def test_grad_clip_group_refuses(cl, status, tensors, kw):
    assert _clip(cl, tensors, **kw) == status


def test_grad_norm_group_refuses_and_ignores_out(cl):
    from semi_structured_sparsity_step_b200 import _binding as B
    t = (B.GradTensor * 1)(B.GradTensor(AL + 4, None, 4, 0, 0))
    assert cl.sbl_grad_norm_group(ctypes.addressof(t), 1, AL, AL, AL, 1 << 30, None) == 3
    t[0].g = None
    assert cl.sbl_grad_norm_group(ctypes.addressof(t), 1, AL, AL, AL, 1 << 30, None) == 1
    assert cl.sbl_grad_norm_group(None, 1, AL, AL, AL, 1 << 30, None) == 1
    assert cl.sbl_grad_group_workspace_bytes(-1) == 0
    assert cl.sbl_grad_group_workspace_bytes(129) > cl.sbl_grad_group_workspace_bytes(128)


def test_binding_refuses_tensors_that_the_call_would_misread(monkeypatch):
    """A host tensor, a wrong type, a strided view and a short buffer never reach the library."""
    import torch
    from semi_structured_sparsity_step_b200 import _binding as B
    monkeypatch.setattr(B, "_device", lambda: 0)
    a = B._args("sbl_block_norm")
    assert a(None, torch.float32, 4) is None and a(AL, torch.float32, 4) == AL
    with pytest.raises(B.SblError):
        a(torch.zeros(4), torch.float32, 4)  # on the host
    monkeypatch.setattr(B, "_device", lambda: -1)  # what get_device() gives for a host tensor
    a = B._args("sbl_block_norm")
    x = torch.zeros(4, 8)
    assert a(x, torch.float32, 32) == x.data_ptr()
    for bad in (x.to(torch.bfloat16), x[:, ::2], x[:2], x.t()):
        with pytest.raises(B.SblError) as e:
            a(bad, torch.float32, 32)
        assert e.value.status == 1


@pytest.mark.parametrize("status,kw", [
    (1, dict(flags=2)), (1, dict(Xq=None)), (1, dict(amax=None)), (1, dict(Wq=None)), (1, dict(wmax=None)),
    (1, dict(Y=None)), (2, dict(T=-1)), (2, dict(T=2 ** 30 + 1)), (2, dict(d_out=2 ** 30 + 8)), (2, dict(d_in=24)), (2, dict(d_in=0)), (2, dict(d_in=131072)),
    (2, dict(d_out=12)), (2, dict(d_out=-8)), (3, dict(Xq=AL + 8)), (3, dict(wmax=AL + 4)), (3, dict(Y=AL + 2)),
    (0, dict(T=0)), (0, dict(d_out=0)),
])
def test_forward_w8a8_refuses(cl, status, kw):
    a = dict(Xq=AL, amax=AL, Wq=AL, wmax=AL, T=4, d_in=32, d_out=16, flags=0, Y=AL)
    a.update(kw)
    assert cl.sbl_forward_w8a8(*a.values(), None) == status


B2 = AL + 4096


@pytest.mark.parametrize("tensors", [
    [(AL, AL, 4, 0, 0), (AL, AL, 4, 0, 0)],              # clipped twice in place
    [(AL, AL, 4, 0, 0), (AL, B2, 4, 0, 0)],              # read while it is clipped in place
    [(AL, B2, 4, 0, 0), (AL + 64, B2, 4, 1, 0)],         # one output for two
    [(AL, B2, 4, 0, 0), (B2, B2 + 64, 4, 0, 0)],         # the output of one is the gradient of another
    [(AL + 64 * i, AL + 64 * i, 4, 0, 0) for i in range(300)] + [(AL + 64 * 7, B2 * 64, 4, 0, 0)],
])
def test_grad_clip_group_refuses_outputs_that_race(cl, tensors):
    assert _clip(cl, tensors) == 1


@pytest.mark.parametrize("period", [5, 2 ** 31 - 1, 2 ** 32 + 1, 2 ** 63 - 1])
def test_gate_period_reaches_the_library_whole(monkeypatch, period):
    """One gate row for all tokens, whatever the period beyond them: never cut down to an int of fewer bits."""
    import torch
    from semi_structured_sparsity_step_b200 import _binding as B
    calls = []
    monkeypatch.setattr(B, "_torch", torch)
    monkeypatch.setattr(B, "_device", lambda: -1)  # what get_device() gives for a host tensor
    monkeypatch.setattr(B, "_call", lambda name, *args: calls.append(args))
    T, d = 5, 32
    Y, H, gain = torch.zeros(T, d), torch.zeros(T, d, dtype=torch.bfloat16), torch.ones(1, d, dtype=torch.bfloat16)
    B.sbl_block_norm(Y, H, None, gain, period, 1.0, gain, 1e-6, T, d, 0, H, None, None, None, None, 0)
    B.sbl_block_norm_backward([Y], None, None, H, None, gain, period, 1.0, gain, Y, T, d, 0, H, None, None, None, None,
                              0, None, 0, 0)
    assert [ctypes.c_int(c[i]).value for c, i in zip(calls, (4, 7))] == [min(period, 2 ** 31 - 1)] * 2


def test_layers_refuse_what_their_calls_would_misread(monkeypatch):
    """A tensor of another device, type or size, and a backward of another number of tokens."""
    import torch
    from semi_structured_sparsity_step_b200 import _binding as B
    from semi_structured_sparsity_step_b200 import layer
    monkeypatch.setattr(B, "_torch", torch)
    monkeypatch.setattr(B, "_call", lambda *args: None)
    bf16 = torch.bfloat16
    L = object.__new__(layer.Int8Linear)
    L.W, L.d_out, L.d_in = torch.zeros(16, 32, dtype=bf16), 16, 32
    L.Wq, L.wmax, L.one = torch.zeros(16, 32, dtype=torch.int8), torch.zeros(16), torch.ones(1)
    good = dict(dY=torch.zeros(4, 16, dtype=bf16), X=torch.zeros(4, 32, dtype=bf16), dX=torch.zeros(4, 32),
                dW=torch.zeros(16, 32))
    monkeypatch.setattr(B, "_device", lambda: 0)  # the host tensors are not there
    with pytest.raises(B.SblError):
        L.weight_step(0)
    with pytest.raises(B.SblError):
        L.backward(**good, stream=0)
    monkeypatch.setattr(B, "_device", lambda: -1)
    L.weight_step(0)
    L.backward(**good, stream=0)
    L.backward(**dict(good, dX=None), stream=0)
    for k, bad in (("dY", torch.zeros(4, 16)), ("X", good["X"][:3]), ("dX", good["dX"].to(bf16)),
                   ("dW", torch.zeros(32, 16).t())):
        with pytest.raises(B.SblError):
            L.backward(**dict(good, **{k: bad}), stream=0)
    N = object.__new__(layer.BlockNorm)
    N.T = 4
    with pytest.raises(AssertionError):
        N.backward([good["dX"]], None, None, good["X"][:3], None, stream=0)
