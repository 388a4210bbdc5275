"""The binding and the layer helpers of the operators around the products, on the CPU: the library call is
replaced by one that records what would reach it, host tensors stand for device tensors."""
import ctypes

import pytest
import torch

from semi_structured_sparsity_step_b200 import _binding as B

BF16, I8 = torch.bfloat16, torch.int8


@pytest.fixture
def calls(monkeypatch):
    got = []
    monkeypatch.setattr(B, "_torch", torch)
    monkeypatch.setattr(B, "_device", lambda: -1)  # what get_device() gives for a host tensor
    monkeypatch.setattr(B, "_call", lambda name, *args: got.append((name, args)))
    return got


T, D, D_OUT = 5, 32, 16


def _norm(**kw):
    h = torch.zeros(T, D, dtype=BF16)
    a = dict(Y=torch.zeros(T, D), H=h, g_post=h[0], gate=h, gate_period=1, res_scale=1.0, g_pre=h[0], eps=1e-6, T=T, d=D,
             flags=0, H_out=h, Xn=h, Xq=torch.zeros(T, D, dtype=I8), amax=torch.zeros(T), rstd=torch.zeros(2 * T), stream=0)
    return B.sbl_block_norm(**dict(a, **kw))


def _norm_backward(**kw):
    h, x = torch.zeros(T, D, dtype=BF16), torch.zeros(T, D)
    a = dict(dXn=[x], dH_out=h, Y=x, H_out=h, g_post=h[0], gate=h, gate_period=1, res_scale=1.0, g_pre=h[0],
             rstd=torch.zeros(2 * T), T=T, d=D, flags=0, dY=h, dH=h, dg_post=x[0], dg_pre=x[0], dgate=x, accumulate=0,
             workspace=torch.zeros(64, dtype=torch.uint8), workspace_bytes=64, stream=0)
    return B.sbl_block_norm_backward(**dict(a, **kw))


def _w8a8(**kw):
    a = dict(Xq=torch.zeros(T, D, dtype=I8), amax=torch.zeros(T), Wq=torch.zeros(D_OUT, D, dtype=I8),
             wmax=torch.zeros(D_OUT), T=T, d_in=D, d_out=D_OUT, flags=0, Y=torch.zeros(T, D_OUT), stream=0)
    return B.sbl_forward_w8a8(**dict(a, **kw))


def _grads(fn):
    def call(**kw):
        g = torch.zeros(64)
        a = dict(tensors=[(g, g, 64, False)], sumsq=torch.zeros(1, dtype=torch.float64), norm=torch.zeros(1),
                 workspace=torch.zeros(64, dtype=torch.uint8), workspace_bytes=64, stream=0)
        if fn is B.sbl_grad_clip_group:
            a.update(max_norm=1.0, clip=torch.zeros(1))
        return fn(**dict(a, **kw))
    return call


CALLS = {"norm": _norm, "norm_backward": _norm_backward, "w8a8": _w8a8, "clip": _grads(B.sbl_grad_clip_group),
         "grad_norm": _grads(B.sbl_grad_norm_group)}
INT = 2 ** 32  # an int or an unsigned of the library keeps its last 32 bits


@pytest.mark.parametrize("which,name,value", [
    ("norm", "T", T - INT), ("norm", "d", D - INT), ("norm", "flags", -INT), ("norm", "flags", INT),
    ("norm_backward", "T", T - INT), ("norm_backward", "d", D - INT), ("norm_backward", "flags", INT), ("norm_backward", "flags", -INT), ("norm_backward", "accumulate", INT),
    ("norm_backward", "accumulate", 1 - INT),
    ("w8a8", "T", T - INT), ("w8a8", "d_in", D - INT), ("w8a8", "d_out", D_OUT - INT), ("w8a8", "flags", INT),
    # a size_t keeps the last 64: one byte too few would arrive as more than any workspace needs
    ("norm_backward", "workspace_bytes", -1), ("norm_backward", "workspace_bytes", 64 - 2 ** 64),
    ("clip", "workspace_bytes", -1), ("grad_norm", "workspace_bytes", -1),
    ("clip", "tensors", [(1 << 12, 1 << 12, -1, False)]), ("grad_norm", "tensors", [(1 << 12, None, 2 ** 64, False)]),
])
def test_integers_that_the_library_would_cut_are_refused(calls, which, name, value):
    call = CALLS[which]
    call()
    assert len(calls) == 1
    with pytest.raises(B.SblError):
        call(**{name: value})
    assert len(calls) == 1


def test_integers_of_the_library_s_width_reach_it(calls):
    """The library answers for what its own types can hold: both ends of an int arrive as they are."""
    for T_ in (-1, -2 ** 31):
        _norm(T=T_)
        _w8a8(T=T_)
    assert [ctypes.c_int(c[1][i]).value for c, i in zip(calls, (8, 4, 8, 4))] == [-1, -1, -2 ** 31, -2 ** 31]


@pytest.mark.parametrize("period", [0, -1, -2 ** 31, 1 - INT, -2 ** 63])
def test_a_gate_period_below_one_never_arrives_as_a_period(calls, period):
    """1 - 2^32 would be cut to 1, one gate row per token, with no row of the gate asked for."""
    _norm(gate_period=period)
    _norm_backward(gate_period=period)
    assert all(ctypes.c_int(c[1][i]).value < 1 for c, i in zip(calls, (4, 7)))


@pytest.mark.parametrize("fn", ["sbl_grad_group_workspace_bytes", "sbl_block_norm_backward_workspace_bytes"])
@pytest.mark.parametrize("value", [2 ** 32 + 16, 16 - 2 ** 32])
def test_workspace_of_a_size_that_is_no_int_is_none(fn, value):
    from semi_structured_sparsity_step_b200 import build
    build.build()
    assert getattr(B, fn)(16) > 0
    assert getattr(B, fn)(value) == 0


# ---- layer helpers: [tokens, width] and nothing that would be read as something else

def _block_norm(post=True):
    from semi_structured_sparsity_step_b200 import layer
    gain = torch.ones(D, dtype=BF16)
    N = object.__new__(layer.BlockNorm)  # the constructor asks for a device
    N.g_pre, N.g_post, N.d, N.res_scale, N.eps, N.flags = gain, gain if post else None, D, 1.0, 1e-6, 0
    N.H_out, N.Xn = torch.zeros(28, D, dtype=BF16), torch.zeros(28, D, dtype=BF16)
    N.Xq, N.amax, N.rstd = torch.zeros(28, D, dtype=I8), torch.zeros(28), torch.zeros(56)
    N.dg_pre, N.dg_post = torch.zeros(D), torch.zeros(D) if post else None
    N.ws_bytes, N.ws, N.T = 64, torch.zeros(64, dtype=torch.uint8), None
    return N


@pytest.mark.parametrize("name,bad", [
    ("Y", (2, 7, D)), ("Y", (28, D // 2)), ("Y", (7, 2 * D)), ("Y", (14 * D,)), ("Y", (1, 14, D)), ("Y", (29, D)),
    ("H", (2, 7, D)), ("H", (28, D // 2)), ("H", (7, 2 * D)), ("H", (13, D)), ("gate", (2, 2 * D)),
    ("gate", (4, D // 2)), ("gate", (1, 2, D)), ("gate", (1, D)), ("gate", (D,)), ("gate", (2 * D,)), ("Y", (D,)),
    ("H", (D,)),
])
def test_block_norm_forward_refuses_other_shapes(calls, name, bad):
    N = _block_norm()
    good = dict(Y=(14, D), H=(20, D), gate=(2, D))
    types = dict(Y=torch.float32, H=BF16, gate=BF16)

    def args(**over):
        return {k: torch.zeros(*s, dtype=types[k]) for k, s in dict(good, **over).items()}

    out = N.forward(**args(), gate_period=7, stream=0)
    assert [tuple(x.shape) for x in out] == [(14, D)] * 3 + [(14,)]
    N.forward(**args(gate=(D,)), gate_period=14, stream=0)  # a gate for each channel
    assert len(calls) == 2
    with pytest.raises(B.SblError):
        N.forward(**args(**{name: bad}), gate_period=7, stream=0)
    assert len(calls) == 2 and N.T == 14


@pytest.mark.parametrize("name,bad", [
    ("dXn", (2, 7, D)), ("dXn", (13, D)), ("dXn", (7, 2 * D)), ("dH_out", (2, 7, D)), ("dH_out", (7, 2 * D)),
    ("Y", (2, 7, D)), ("Y", (28, D // 2)), ("Y", (13, D)), ("dY", (14, 2 * D)), ("dY", (14, 1, D)), ("dH", (13, D)),
    ("dH", (2, 7, D)), ("gate", (2, 2 * D)), ("dgate", (2, 2 * D)), ("dgate", (4, D // 2)),
])
def test_block_norm_backward_refuses_other_shapes(calls, name, bad):
    N = _block_norm()
    N.T = 14
    good = dict(dXn=(14, D), dH_out=(14, D), Y=(14, D), dY=(14, D), dH=(14, D), gate=(2, D), dgate=(2, D))
    f32 = ("dXn", "Y", "dgate")

    def args(**over):
        a = {k: torch.zeros(*s, dtype=torch.float32 if k in f32 else BF16) for k, s in dict(good, **over).items()}
        return dict(a, dXn=[a["dXn"]])

    N.backward(**args(), gate_period=7, stream=0)
    N.backward(**dict(args(), dH_out=None, dH=None, gate=None, dgate=None), stream=0)
    assert len(calls) == 2
    with pytest.raises(B.SblError):
        N.backward(**args(**{name: bad}), gate_period=7, stream=0)
    assert len(calls) == 2


@pytest.mark.parametrize("name,bad", [
    ("Xq", (2, 7, D)), ("Xq", (28, D // 2)), ("Xq", (7, 2 * D)), ("Xq", (14 * D,)), ("amax", (13,)),
    ("Y", (2, 7, D_OUT)), ("Y", (13, D_OUT)), ("Y", (7, 2 * D_OUT)), ("dY", (2, 7, D_OUT)), ("dY", (7, 2 * D_OUT)),
    ("X", (2, 7, D)), ("X", (13, D)), ("X", (7, 2 * D)), ("dX", (2, 7, D)), ("dX", (13, D)),
    ("dW", (D, D_OUT)), ("dW", (2, D_OUT // 2, D)),
])
def test_int8_linear_refuses_other_shapes(calls, name, bad):
    from semi_structured_sparsity_step_b200 import layer
    L = object.__new__(layer.Int8Linear)
    L.W, L.d_out, L.d_in = torch.zeros(D_OUT, D, dtype=BF16), D_OUT, D
    L.Wq, L.wmax, L.one = torch.zeros(D_OUT, D, dtype=I8), torch.zeros(D_OUT), torch.ones(1)
    fwd = dict(Xq=(14, D), amax=(14,), Y=(14, D_OUT))
    bwd = dict(dY=(14, D_OUT), X=(14, D), dX=(14, D), dW=(D_OUT, D))
    types = dict(Xq=I8, dY=BF16, X=BF16)

    def args(good, **over):
        return {k: torch.zeros(*s, dtype=types.get(k, torch.float32)) for k, s in dict(good, **over).items()}

    L.forward(**args(fwd), stream=0)
    L.backward(**args(bwd), stream=0)
    L.backward(**dict(args(bwd), dX=None), stream=0)
    L.backward(**dict(args(bwd), dW=None), stream=0)
    L.backward(**args(bwd, dW=(D_OUT * D,)), stream=0)
    L.backward(**dict(args(bwd), dW=1 << 12), stream=0)  # a raw pointer
    L.forward(**args(fwd, amax=(20,), Y=(20, D_OUT)), stream=0)  # buffers for more tokens
    assert len(calls) == 7
    call, good = (L.forward, fwd) if name in fwd else (L.backward, bwd)
    with pytest.raises(B.SblError):
        call(**args(good, **{name: bad}), stream=0)
    assert len(calls) == 7


def test_clipped_gradients_are_not_clipped_again_by_the_optimizer(calls):
    """sumsq stays the sum of the gradients as they came, so after a clip in place the optimizer gets none."""
    from semi_structured_sparsity_step_b200 import layer
    C = object.__new__(layer.GradClip)  # the constructor's tensors are on a device
    g = torch.zeros(64)
    C.tensors, C.ws, C.ws_bytes = [(g, g, 64, False)], torch.zeros(64, dtype=torch.uint8), 64
    C.sumsq, C.norm, C.factor, C.grad_sqnorm = torch.zeros(1, dtype=torch.float64), torch.zeros(1), torch.zeros(1), None
    for _ in range(2):
        C.norm_only(stream=0)
        assert C.grad_sqnorm is C.sumsq
        C.clip(1.0, stream=0)
        assert C.grad_sqnorm is None
    assert [c[0] for c in calls] == ["sbl_grad_norm_group", "sbl_grad_clip_group"] * 2


@pytest.mark.parametrize("stream", ["none", "object", "handle"])
def test_workspace_of_the_first_backward_belongs_to_its_stream(calls, monkeypatch, stream):
    """Allocated under another stream, it could be memory whose last reader there still runs."""
    from contextlib import contextmanager
    from types import SimpleNamespace
    from semi_structured_sparsity_step_b200 import layer
    current, allocated = ["the caller's"], []

    @contextmanager
    def use(s):
        current.append(current[-1] if s is None else s)
        yield
        current.pop()

    def empty(*size, **kw):
        allocated.append(current[-1])
        return torch.empty(*size, dtype=kw["dtype"])

    monkeypatch.setattr(layer, "torch", SimpleNamespace(
        empty=empty, uint8=torch.uint8, cuda=SimpleNamespace(
            stream=use, ExternalStream=lambda handle, device=None: ("external", handle))))
    side = SimpleNamespace(cuda_stream=1234)
    arg, owner = {"none": (None, "the caller's"), "object": (side, side), "handle": (1234, ("external", 1234))}[stream]
    monkeypatch.setattr(B, "_stream", lambda s: 0)
    N = _block_norm()
    N.T, N.ws = 14, None
    x, h = torch.zeros(14, D), torch.zeros(14, D, dtype=BF16)
    for _ in range(2):
        N.backward([x], None, x, h, None, stream=arg)
    assert allocated == [owner] and len(calls) == 2
