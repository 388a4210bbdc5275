"""Cases of the operators that stand around the Sparse-BitLinear products of a block.

* ``block_norm``: the norm after a block's output product, its gate, the scaled residual, the norm
  before the next product and the int8 quantiser, in one call; and its backward pass.
* ``w8a8``: the product of int8 activations (a scale for each token) with int8 weights (a scale for
  each output channel), for projections that are not ternary.
* ``grad_clip``: the global norm of the gradients of many tensors, and the gradients clipped by it.

Each case runs in a plain form (torch operations, one at a time) or, with ``own`` set, through the
library's entry points.  Inputs are synthetic and made from a seed alone.
"""
import math

import torch

own = False

EPS = 1e-6

# hidden, feed-forward, key/value and query widths of the layer sets that the benchmark runs
LAYER_SETS = {
    "0.5b": (896, 4864, 128),
    "3b": (2048, 11008, 256),
}


def listed():
    return [
        # one token of a decode step between two products, on the hidden width of the 3B set
        dict(name="norm_decode_1x2048", op="block_norm", T=1, d=2048, y="f32", h="bf16", post=True, period=0),
        # a padded prefill of several sequences, a gate row for every 512 tokens, fp32 residual stream
        dict(name="norm_ragged_4093x896", op="block_norm", T=4093, d=896, y="bf16", h="f32", post=True, period=512),
        # the training batch of the 3B set: 16 sequences of 2048 tokens, a gate row for each sequence
        dict(name="norm_train_32768x2048", op="block_norm", T=32768, d=2048, y="f32", h="bf16", post=True, period=2048),
        # the backward of a short batch: two products (gate and up) read the normalised row
        dict(name="norm_bwd_509x896", op="block_norm_backward", T=509, d=896, y="f32", h="f32", post=True, period=0,
             readers=2),
        # the backward of the training batch: q, k and v read the normalised row
        dict(name="norm_bwd_32768x2048", op="block_norm_backward", T=32768, d=2048, y="f32", h="bf16", post=True,
             period=2048, readers=3),
        # a wide residual stream with one gate for each channel
        dict(name="norm_bwd_4096x8192", op="block_norm_backward", T=4096, d=8192, y="bf16", h="bf16", post=True,
             period=4096, readers=1),
        # one token through the up projection of the 3B set
        dict(name="w8a8_decode_1", op="w8a8", T=1, d_in=2048, d_out=11008, y="f32"),
        # a decode batch through the down projection
        dict(name="w8a8_decode_16", op="w8a8", T=16, d_in=11008, d_out=2048, y="bf16"),
        # a short prefill whose length fills no tile
        dict(name="w8a8_prefill_509", op="w8a8", T=509, d_in=2048, d_out=2048, y="f32"),
        # a prefill of 8 sequences of 1024 tokens
        dict(name="w8a8_prefill_8192", op="w8a8", T=8192, d_in=2048, d_out=11008, y="bf16"),
        # the gradients of one layer of the 0.5B set, held in bf16
        dict(name="clip_0.5b_1_layer", op="grad_clip", model="0.5b", layers=1, dtype="bf16", max_norm=1.0),
        # the gradients of four layers of the 3B set in fp32, as the products leave them
        dict(name="clip_3b_4_layers", op="grad_clip", model="3b", layers=4, dtype="f32", max_norm=1.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["block_norm", "block_norm_backward", "w8a8", "w8a8", "grad_clip"])
    if op.startswith("block_norm"):
        d = 16 * _log_int(rng, 8, 512)
        T = _log_int(rng, 1, min(32768, (1 << 25) // d))
        period = rng.choice([0, 1, T, max(1, _log_int(rng, 1, T))])
        case = dict(op=op, T=T, d=d, y=rng.choice(["f32", "bf16"]), h=rng.choice(["f32", "bf16"]),
                    post=rng.random() < 0.75, period=period)
        if op == "block_norm_backward":
            case["readers"] = rng.randint(1, 3)
        return case
    if op == "w8a8":
        d_in, d_out = 16 * _log_int(rng, 8, 688), 8 * _log_int(rng, 16, 1376)
        T = _log_int(rng, 1, min(8192, (1 << 37) // (d_in * d_out)))
        return dict(op=op, T=T, d_in=d_in, d_out=d_out, y=rng.choice(["f32", "bf16"]))
    return dict(op=op, model=rng.choice(sorted(LAYER_SETS)), layers=rng.randint(1, 4),
                dtype=rng.choice(["f32", "bf16"]), max_norm=rng.choice([0.5, 1.0, 1e6]) * rng.uniform(0.5, 2.0))


def _type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _rows(gen, T, d, outliers=True):
    """Activations: N(0, 1) with a few channels ten times as large."""
    x = torch.randn(T, d, generator=gen, device="cuda")
    if outliers:
        at = torch.randint(0, d, (max(1, d // 1000),), generator=gen, device="cuda")
        x[:, at] *= 10
    return x


def _gain(gen, d):
    return (1 + 0.1 * torch.randn(d, generator=gen, device="cuda")).to(torch.bfloat16)


def _codes(x):
    """Row-wise absmax int8 codes and the rows' largest magnitudes."""
    amax = x.abs().amax(1).clamp_min(1e-5)
    return torch.round(x * (127 / amax)[:, None]).to(torch.int8), amax


def _shapes(model, layers):
    hidden, ff, kv = LAYER_SETS[model]
    one = [(hidden, hidden), (kv, hidden), (kv, hidden), (hidden, hidden), (ff, hidden), (ff, hidden), (hidden, ff),
           (hidden,), (hidden,)]
    return one * layers


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = dict(case)
    if op.startswith("block_norm"):
        T, d, period = case["T"], case["d"], case["period"]
        s["Y"] = _rows(gen, T, d).to(_type(case["y"]))
        s["H"] = (3 * _rows(gen, T, d)).to(_type(case["h"]))
        if T > 8:  # a padding token
            s["Y"][T - 1] = 0
            s["H"][T - 1] = 0
        s["g_post"] = _gain(gen, d) if case["post"] else None
        s["g_pre"] = _gain(gen, d)
        s["gate"] = (0.5 * torch.randn(-(-T // period), d, generator=gen, device="cuda")).to(torch.bfloat16) \
            if period else None
        s["res_scale"] = 0.75
        empty = lambda *shape, dtype: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
        if op == "block_norm":
            s["H_out"] = empty(T, d, dtype=_type(case["h"]))
            s["Xn"] = empty(T, d, dtype=torch.bfloat16)
            s["Xq"] = empty(T, d, dtype=torch.int8)
            s["amax"] = empty(T, dtype=torch.float32)
            s["rstd"] = empty(2, T, dtype=torch.float32)
        else:
            # the residual stream and the two norms' factors, as the forward pass left them
            r1 = (s["Y"].double().square().mean(1) + EPS).rsqrt() if case["post"] else torch.ones(T, device="cuda")
            s["H_out"] = s.pop("H")
            r2 = (s["H_out"].double().square().mean(1) + EPS).rsqrt()
            s["rstd"] = torch.stack([r1.float(), r2.float()])
            s["dXn"] = [0.01 * torch.randn(T, d, generator=gen, device="cuda") for _ in range(case["readers"])]
            s["dH_out"] = (0.02 * torch.randn(T, d, generator=gen, device="cuda")).to(_type(case["h"]))
            s["dY"] = empty(T, d, dtype=torch.bfloat16)
            s["dH"] = empty(T, d, dtype=_type(case["h"]))
            s["dg_post"] = empty(d, dtype=torch.float32) if case["post"] else None
            s["dg_pre"] = empty(d, dtype=torch.float32)
            s["dgate"] = empty(-(-T // period), d, dtype=torch.float32) if period else None
    elif op == "w8a8":
        T, d_in, d_out = case["T"], case["d_in"], case["d_out"]
        s["Xq"], s["amax"] = _codes(_rows(gen, T, d_in))
        s["Wq"], s["wmax"] = _codes(0.02 * torch.randn(d_out, d_in, generator=gen, device="cuda"))
        s["Y"] = torch.empty(T, d_out, dtype=_type(case["y"]), device="cuda")
    else:
        shapes = _shapes(case["model"], case["layers"])
        s["grads"] = [(1e-3 * torch.randn(*shape, generator=gen, device="cuda")).to(_type(case["dtype"]))
                      for shape in shapes]
        s["outs"] = [torch.empty_like(g) for g in s["grads"]]
        s["sumsq"] = torch.empty(1, dtype=torch.float64, device="cuda")
        s["norm"] = torch.empty(1, dtype=torch.float32, device="cuda")
        s["clip"] = torch.empty(1, dtype=torch.float32, device="cuda")
    # scratch that a caller keeps; the library says how much it needs, and this is never less
    s["workspace"] = torch.empty(64 << 20, dtype=torch.uint8, device="cuda") if op != "w8a8" else None
    return s


# ------------------------------------------------------------------------------------ plain forms

def _rstd(x):
    """1 / sqrt(mean(x^2) + eps) of each row: the sum in 64 bits, because the int8 codes behind it
    sit next to rounding borders, then one rounding to 32 bits for each step."""
    d = torch.tensor(float(x.shape[1]), dtype=torch.float64, device=x.device)
    eps = torch.tensor(EPS, dtype=torch.float32).double().item()
    v = (x.double().square().sum(1) / d + eps).float()
    return torch.div(torch.ones_like(v), v.sqrt())


def _gate_rows(gate, period, T):
    return gate.float().repeat_interleave(period, 0)[:T]


def _plain_block_norm(s):
    T = s["T"]
    y, h = s["Y"].float(), s["H"].float()
    r1 = torch.ones(T, device=y.device)
    if s["g_post"] is not None:
        r1 = _rstd(y)
        y = (y * r1[:, None]) * s["g_post"].float()
    if s["gate"] is not None:
        y = _gate_rows(s["gate"], s["period"], T) * y
    h_out = (h * s["res_scale"] + y).to(s["H"].dtype)
    h = h_out.float()
    r2 = _rstd(h)
    xn = ((h * r2[:, None]) * s["g_pre"].float()).to(torch.bfloat16)
    x = xn.float()
    amax = x.abs().amax(1).clamp_min(1e-5)
    scale = torch.div(torch.full_like(amax, 127.0), amax)
    xq = torch.round(x * scale[:, None]).clamp(-128, 127).to(torch.int8)
    return dict(H_out=h_out, Xn=xn, Xq=xq, amax=amax, rstd=torch.stack([r1, r2]))


def _plain_block_norm_backward(s):
    T, d, period = s["T"], s["d"], s["period"]
    y, h = s["Y"].float(), s["H_out"].float()
    r1, r2 = s["rstd"][0][:, None], s["rstd"][1][:, None]
    dxn = s["dXn"][0] if len(s["dXn"]) == 1 else torch.stack(s["dXn"]).sum(0)
    xhat = h * r2
    t = dxn * s["g_pre"].float()
    dh = s["dH_out"].float() + r2 * (t - xhat * (t * xhat).mean(1, keepdim=True))
    out = dict(dH=(dh * s["res_scale"]).to(s["H_out"].dtype), dg_pre=(dxn * xhat).sum(0))
    yhat = y * r1 if s["g_post"] is not None else y
    u = yhat * s["g_post"].float() if s["g_post"] is not None else y
    du = dh
    if s["gate"] is not None:
        groups = -(-T // period)
        prod = torch.zeros(groups * period, d, device=y.device)
        prod[:T] = dh * u
        out["dgate"] = prod.view(groups, period, d).sum(1)
        du = _gate_rows(s["gate"], period, T) * dh
    if s["g_post"] is not None:
        out["dg_post"] = (du * yhat).sum(0)
        t = du * s["g_post"].float()
        du = r1 * (t - yhat * (t * yhat).mean(1, keepdim=True))
    out["dY"] = du.to(torch.bfloat16)
    return out


def _plain_w8a8(s):
    acc = s["Xq"].float() @ s["Wq"].float().t()
    return dict(Y=(acc * (s["amax"] / 127)[:, None] * (s["wmax"] / 127)).to(s["Y"].dtype))


def _plain_grad_clip(s):
    sumsq = torch.stack([g.double().square().sum() for g in s["grads"]]).sum()
    norm = sumsq.sqrt()
    clip = (s["max_norm"] / (norm + 1e-6)).clamp_max(1.0).float()
    return dict(outs=[(g.float() * clip).to(g.dtype) for g in s["grads"]], norm=norm.float(), clip=clip)


# ----------------------------------------------------------------------------- the library's calls

def _own_block_norm(s):
    import semi_structured_sparsity_step_b200 as sbl
    flags = (sbl.SBL_BLOCK_Y_BF16 if s["y"] == "bf16" else 0) | (sbl.SBL_BLOCK_H_F32 if s["h"] == "f32" else 0)
    sbl.sbl_block_norm(s["Y"], s["H"], s["g_post"], s["gate"], s["period"], s["res_scale"], s["g_pre"], EPS, s["T"],
                       s["d"], flags, s["H_out"], s["Xn"], s["Xq"], s["amax"], s["rstd"])
    return dict(H_out=s["H_out"], Xn=s["Xn"], Xq=s["Xq"], amax=s["amax"], rstd=s["rstd"])


def _own_block_norm_backward(s):
    import semi_structured_sparsity_step_b200 as sbl
    flags = (sbl.SBL_BLOCK_Y_BF16 if s["y"] == "bf16" else 0) | (sbl.SBL_BLOCK_H_F32 if s["h"] == "f32" else 0)
    sbl.sbl_block_norm_backward(s["dXn"], s["dH_out"], s["Y"], s["H_out"], s["g_post"], s["gate"], s["period"],
                                s["res_scale"], s["g_pre"], s["rstd"], s["T"], s["d"], flags, s["dY"], s["dH"],
                                s["dg_post"], s["dg_pre"], s["dgate"], 0, s["workspace"], s["workspace"].numel())
    out = dict(dH=s["dH"], dg_pre=s["dg_pre"], dY=s["dY"])
    if s["gate"] is not None:
        out["dgate"] = s["dgate"]
    if s["g_post"] is not None:
        out["dg_post"] = s["dg_post"]
    return out


def _own_w8a8(s):
    import semi_structured_sparsity_step_b200 as sbl
    flags = sbl.SBL_W8A8_Y_BF16 if s["y"] == "bf16" else 0
    sbl.sbl_forward_w8a8(s["Xq"], s["amax"], s["Wq"], s["wmax"], s["T"], s["d_in"], s["d_out"], flags, s["Y"])
    return dict(Y=s["Y"])


def _own_grad_clip(s):
    import semi_structured_sparsity_step_b200 as sbl
    bf16 = s["dtype"] == "bf16"
    sbl.sbl_grad_clip_group([(g, o, g.numel(), bf16) for g, o in zip(s["grads"], s["outs"])], s["max_norm"],
                            s["sumsq"], s["norm"], s["clip"], s["workspace"], s["workspace"].numel())
    return dict(outs=s["outs"], norm=s["norm"][0], clip=s["clip"][0])


def run(state):
    op = state["op"]
    if own:
        return {"block_norm": _own_block_norm, "block_norm_backward": _own_block_norm_backward, "w8a8": _own_w8a8,
                "grad_clip": _own_grad_clip}[op](state)
    return {"block_norm": _plain_block_norm, "block_norm_backward": _plain_block_norm_backward, "w8a8": _plain_w8a8,
            "grad_clip": _plain_grad_clip}[op](state)


# ------------------------------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    size = {"f32": 4, "bf16": 2}
    if op.startswith("block_norm"):
        T, d, period = case["T"], case["d"], case["period"]
        n, y, h = T * d, size[case["y"]], size[case["h"]]
        gate = 2 * d * -(-T // period) if period else 0
        gains = 2 * d * (2 if case["post"] else 1)
        if op == "block_norm":
            # Y, H in; H_out, Xn, Xq out; amax and the two factors of each row
            return dict(bytes=n * (y + 2 * h + 2 + 1) + gate + gains + 12 * T, flops=16 * n)
        # dXn of each reader, dH_out, Y, H_out in; dY, dH out; the gradients of the gains and of the gate
        return dict(bytes=n * (4 * case["readers"] + 3 * h + y + 2) + 3 * gate + 3 * gains + 8 * T, flops=32 * n)
    if op == "w8a8":
        T, d_in, d_out = case["T"], case["d_in"], case["d_out"]
        return dict(bytes=T * d_in + d_out * d_in + T * d_out * size[case["y"]] + 4 * (T + d_out),
                    flops=2 * T * d_in * d_out)
    n = sum(math.prod(shape) for shape in _shapes(case["model"], case["layers"]))
    return dict(bytes=2 * n * size[case["dtype"]], flops=3 * n)


# ------------------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    """The operators' definitions in 64 bits.  The stored residual stream is rounded to its type, as
    the second norm reads what is stored; amax and the int8 codes are those of the bf16 row, which
    64 bits do not give."""
    s = prepare(case, seed)
    f = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor) and v.numel() and v.dtype != torch.uint8}
    op = case["op"]
    if op == "w8a8":
        return dict(Y=torch.einsum("ti,oi->to", f["Xq"], f["Wq"]) * torch.outer(f["amax"], f["wmax"]) / 127.0 ** 2)
    if op == "grad_clip":
        norm = math.sqrt(sum(torch.linalg.vector_norm(g.double()).item() ** 2 for g in s["grads"]))
        c = min(1.0, case["max_norm"] / (norm + 1e-6))
        return dict(outs=[g.double() * c for g in s["grads"]], norm=norm, clip=c)
    T, d = case["T"], case["d"]
    token_gate = 1.0
    if case["period"]:
        group = torch.arange(T, device="cuda") // case["period"]
        token_gate = f["gate"][group]
    if op == "block_norm":
        r1 = 1 / torch.sqrt(torch.linalg.vector_norm(f["Y"], dim=1) ** 2 / d + EPS) if case["post"] \
            else torch.ones(T, dtype=torch.float64, device="cuda")
        branch = torch.einsum("td,t,d->td", f["Y"], r1, f["g_post"]) if case["post"] else f["Y"]
        h_out = 0.75 * f["H"] + token_gate * branch
        h = h_out.to(s["H"].dtype).double()
        r2 = 1 / torch.sqrt(torch.linalg.vector_norm(h, dim=1) ** 2 / d + EPS)
        return dict(H_out=h_out, Xn=torch.einsum("td,t,d->td", h, r2, f["g_pre"]), Xq=None, amax=None,
                    rstd=torch.stack([r1, r2]))

    def through_norm(dz, x, r):
        """Gradient of the row x with z = x * r, r = rms(x)^-1 given: J = r I - r^3 x x^T / d."""
        return r[:, None] * dz - (r ** 3 * torch.einsum("td,td->t", dz, x) / d)[:, None] * x

    dxn = sum(g.double() for g in s["dXn"])
    r1, r2 = f["rstd"]
    d_stream = f["dH_out"] + through_norm(dxn * f["g_pre"], f["H_out"], r2)
    out = dict(dH=0.75 * d_stream, dg_pre=torch.einsum("td,td,t->d", dxn, f["H_out"], r2))
    branch = torch.einsum("td,t,d->td", f["Y"], r1, f["g_post"]) if case["post"] else f["Y"]
    if case["period"]:
        out["dgate"] = torch.zeros_like(f["gate"]).index_add_(0, group, d_stream * branch)
    d_branch = d_stream * token_gate
    if case["post"]:
        out["dg_post"] = torch.einsum("td,td,t->d", d_branch, f["Y"], r1)
        out["dY"] = through_norm(d_branch * f["g_post"], f["Y"], r1)
    else:
        out["dY"] = d_branch
    return out
