"""Device buffers of one Sparse-BitLinear layer and its step through the C ABI.

PyTorch only provides device memory and the stream here; every step of the
operator runs in libsbl's kernels:

    weight_step()  -> sbl_mask_quant   (mask, gamma, ternary, quant-then-mask)
                      + sbl_compress24 for a 2:4 layer built with sparse24=True
    forward(X)     -> sbl_act_quant, sbl_forward (or sbl_forward_sparse24)
    backward(dY)   -> sbl_backward     (dX and the dense dW)

and of what stands around it: the seam between two products (BlockNorm:
sbl_block_norm and its backward), a projection in 8 bits (Int8Linear:
sbl_forward_w8a8) and the clipped gradients of a step (GradClip:
sbl_grad_clip_group).
"""
from __future__ import annotations

import torch

from . import _binding as B


class SparseBitLinearLayer:
    def __init__(self, W: torch.Tensor, N: int, M: int, keep_mask: bool = False, sparse24: bool = True):
        assert W.is_cuda and W.dtype == torch.bfloat16 and W.is_contiguous()
        self.W = W
        self.d_out, self.d_in = W.shape
        self.N, self.M = N, M
        dev = W.device
        self.W_eff = torch.empty(self.d_out, self.d_in, dtype=torch.int8, device=dev)
        self.W_eff_bf16 = torch.empty(self.d_out, self.d_in, dtype=torch.bfloat16, device=dev)
        self.mask_bits = (torch.empty(self.d_out, self.d_in // 8, dtype=torch.uint8, device=dev)
                          if keep_mask else None)
        self.gamma = torch.empty(1, dtype=torch.float32, device=dev)
        self.ws_bytes = B.sbl_mask_quant_workspace_bytes(self.d_out, self.d_in)
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device=dev)
        # 2:4 weights go to the sparse tensor core through the compressed
        # format (the same int32 sums as the dense product, bit for bit; on B200
        # about 1.2x faster than the dense int8 product at the measured shapes).
        # sparse24=False keeps the dense product for them.
        self.sparse24 = bool(sparse24) and (N, M) == (2, 4)
        self.w24_bytes = B.sbl_compress24_bytes(self.d_out, self.d_in) if self.sparse24 else 0
        self.w24 = torch.empty(self.w24_bytes, dtype=torch.uint8, device=dev) if self.sparse24 else None

    def weight_step(self, stream=None):
        B.sbl_mask_quant(self.W, self.d_out, self.d_in, self.N, self.M, self.W_eff, self.W_eff_bf16,
                         self.mask_bits, self.gamma, self.ws, self.ws_bytes, stream)
        if self.sparse24:
            B.sbl_compress24(self.W_eff, self.d_out, self.d_in, self.w24, self.w24_bytes, stream)

    def forward(self, Xq, amax, Y, T=None, acc=None, stream=None):
        T = Xq.shape[0] if T is None else T
        if self.sparse24:
            B.sbl_forward_sparse24(Xq, amax, self.w24, self.gamma, T, self.d_in, self.d_out, Y, acc, stream)
        else:
            B.sbl_forward(Xq, amax, self.W_eff, self.gamma, T, self.d_in, self.d_out, Y, acc, stream)

    def backward(self, dY, X, dX, dW, accumulate_dW=False, T=None, stream=None):
        T = dY.shape[0] if T is None else T
        B.sbl_backward(dY, X, self.W_eff_bf16, self.gamma, T, self.d_in, self.d_out, dX, dW,
                       int(accumulate_dW), None, 0, stream)


def act_quant(X: torch.Tensor, Xq: torch.Tensor, amax: torch.Tensor, stream=None):
    T, d_in = X.shape
    B.sbl_act_quant(X, T, d_in, Xq, amax, stream)


def _rows_of(fn, width, *tensors):
    """Refuses tensors that are not [rows, width], or [width] for one row.  A call takes a contiguous buffer of at least as many
    elements as it has tokens: it would read [batch, sequence, width] as its first rows, and halves of
    wider rows as rows.  A buffer may hold more rows than the call has tokens; they stay as they are."""
    for x in tensors:
        if x is not None and x.__class__ is not int and (x.dim() not in (1, 2) or x.shape[-1] != width):
            raise B.SblError(fn, 2)


class BlockNorm:
    """Norm of a branch output, gate, scaled residual, next norm and int8 codes
    (sbl_block_norm), with its backward, for up to `max_tokens` tokens.

    g_pre, g_post: bf16 gains of the norms after and before the sum (g_post
    None: the branch is not normalised).  The outputs and the factors that the
    backward needs live here and are overwritten by the next call.

    Activations and their gradients are [tokens, d], with as many tokens as Y
    has (a [batch, sequence, d] is flattened by the caller), gates [rows, d] or
    [d] for one row; tensors of other dimensions or widths raise SblError."""

    def __init__(self, g_pre: torch.Tensor, g_post: torch.Tensor | None = None, max_tokens: int = 1,
                 res_scale: float = 1.0, eps: float = 1e-6, y_dtype=torch.float32, h_dtype=torch.bfloat16):
        assert g_pre.is_cuda and g_pre.dtype == torch.bfloat16
        assert y_dtype in (torch.float32, torch.bfloat16) and h_dtype in (torch.float32, torch.bfloat16)
        dev, d = g_pre.device, g_pre.numel()
        assert g_post is None or g_post.numel() == d
        self.g_pre, self.g_post, self.d, self.res_scale, self.eps = g_pre, g_post, d, res_scale, eps
        self.flags = (B.SBL_BLOCK_Y_BF16 if y_dtype == torch.bfloat16 else 0) | \
            (B.SBL_BLOCK_H_F32 if h_dtype == torch.float32 else 0)
        self.H_out = torch.empty(max_tokens, d, dtype=h_dtype, device=dev)
        self.Xn = torch.empty(max_tokens, d, dtype=torch.bfloat16, device=dev)
        self.Xq = torch.empty(max_tokens, d, dtype=torch.int8, device=dev)
        self.amax = torch.empty(max_tokens, dtype=torch.float32, device=dev)
        self.rstd = torch.empty(2 * max_tokens, dtype=torch.float32, device=dev)
        self.dg_pre = torch.zeros(d, dtype=torch.float32, device=dev)
        self.dg_post = torch.zeros(d, dtype=torch.float32, device=dev) if g_post is not None else None
        self.ws_bytes = B.sbl_block_norm_backward_workspace_bytes(d)
        self.ws = None  # allocated by the first backward
        self.T = None  # tokens of the last forward

    def forward(self, Y, H, gate=None, gate_period=0, stream=None):
        """-> (H_out, Xn, Xq, amax) of the call's tokens."""
        T = Y.shape[0]
        _rows_of("sbl_block_norm", self.d, Y, H, gate)
        B.sbl_block_norm(Y, H, self.g_post, gate, gate_period, self.res_scale, self.g_pre, self.eps, T, self.d,
                         self.flags, self.H_out, self.Xn, self.Xq, self.amax, self.rstd, stream)
        self.T = T
        return self.H_out[:T], self.Xn[:T], self.Xq[:T], self.amax[:T]

    def backward(self, dXn, dH_out, Y, dY, dH, gate=None, gate_period=0, dgate=None, accumulate=False, stream=None):
        """dXn: the gradients of Xn from each product that read it (1 to 3); the gains' gradients go
        to dg_pre and dg_post.  The tokens are those of the last forward, whose H_out and factors it
        uses; Y may be None where nothing needs it (no g_post, no dgate)."""
        assert dY.shape[0] == self.T  # the factors lie as that many tokens left them
        _rows_of("sbl_block_norm_backward", self.d, *dXn, dH_out, Y, dY, dH, gate, dgate)
        if self.ws is None:
            # of the stream that writes it: memory freed on the current one may still be read there
            s = torch.cuda.ExternalStream(stream, device=self.g_pre.device) if isinstance(stream, int) else stream
            with torch.cuda.stream(s):
                self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device=self.g_pre.device)
        B.sbl_block_norm_backward(dXn, dH_out, Y, self.H_out, self.g_post, gate, gate_period, self.res_scale,
                                  self.g_pre, self.rstd, dY.shape[0], self.d, self.flags, dY, dH, self.dg_post,
                                  self.dg_pre, dgate, int(accumulate), self.ws, self.ws_bytes, stream)


class Int8Linear:
    """A projection held in 8 bits: W [d_out, d_in] bf16, quantised row by row.

    weight_step() quantises W again after it has changed.  backward() is the
    straight-through estimator on the bf16 W: dX = dY . W, dW = dY^T . X.
    Activations and their gradients are [tokens, d_in] and [tokens, d_out], dW
    [d_out, d_in] or flat; tensors of other dimensions or widths raise SblError."""

    def __init__(self, W: torch.Tensor):
        assert W.is_cuda and W.dtype == torch.bfloat16 and W.is_contiguous()
        self.W = W
        self.d_out, self.d_in = W.shape
        self.Wq = torch.empty(self.d_out, self.d_in, dtype=torch.int8, device=W.device)
        self.wmax = torch.empty(self.d_out, dtype=torch.float32, device=W.device)
        self.one = torch.ones(1, dtype=torch.float32, device=W.device)
        self.weight_step()

    def weight_step(self, stream=None):
        a = B._args("sbl_act_quant")
        B.sbl_act_quant(a(self.W, torch.bfloat16, self.d_out * self.d_in), self.d_out, self.d_in, self.Wq, self.wmax,
                        stream)

    def forward(self, Xq, amax, Y, stream=None):
        """Y [T, d_out] in fp32 or bf16, by its type."""
        _rows_of("sbl_forward_w8a8", self.d_in, Xq)
        _rows_of("sbl_forward_w8a8", self.d_out, Y)
        flags = B.SBL_W8A8_Y_BF16 if Y.dtype == torch.bfloat16 else 0
        B.sbl_forward_w8a8(Xq, amax, self.Wq, self.wmax, Xq.shape[0], self.d_in, self.d_out, flags, Y, stream)

    def backward(self, dY, X, dX, dW, accumulate_dW=False, stream=None):
        """dY, X: bf16, of one number of tokens; dX, dW: float out, each may be None."""
        T, a = dY.shape[0], B._args("sbl_backward")
        f32, bf16 = torch.float32, torch.bfloat16
        n = self.d_out * self.d_in
        _rows_of("sbl_backward", self.d_out, dY)
        flat = isinstance(dW, torch.Tensor) and dW.dim() == 1
        _rows_of("sbl_backward", self.d_in, X, dX, None if flat else dW)
        B.sbl_backward(a(dY, bf16, T * self.d_out), a(X, bf16, T * self.d_in), a(self.W, bf16, n), self.one, T,
                       self.d_in, self.d_out, a(dX, f32, T * self.d_in), a(dW, f32, n), int(accumulate_dW), None, 0,
                       stream)


class GradClip:
    """The global norm of a step's gradients and the clip by it, over a fixed list of
    tensors (fp32 or bf16), in place.

    grad_sqnorm is what sbl_adamw_step takes under that name: after norm_only()
    the sum of the squares, by which it clips itself; after clip(), whose
    gradients are scaled already, None (sumsq is still the sum before the
    clip, and would scale them a second time)."""

    def __init__(self, grads):
        self.tensors = [(g, g, g.numel(), g.dtype == torch.bfloat16) for g in grads]
        dev = grads[0].device
        self.sumsq = torch.zeros(1, dtype=torch.float64, device=dev)
        self.grad_sqnorm = None
        self.norm = torch.zeros(1, dtype=torch.float32, device=dev)
        self.factor = torch.zeros(1, dtype=torch.float32, device=dev)
        self.ws_bytes = B.sbl_grad_group_workspace_bytes(len(grads))
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device=dev)

    def norm_only(self, stream=None):
        B.sbl_grad_norm_group(self.tensors, self.sumsq, self.norm, self.ws, self.ws_bytes, stream)
        self.grad_sqnorm = self.sumsq

    def clip(self, max_norm: float, stream=None):
        B.sbl_grad_clip_group(self.tensors, max_norm, self.sumsq, self.norm, self.factor, self.ws, self.ws_bytes,
                              stream)
        self.grad_sqnorm = None
