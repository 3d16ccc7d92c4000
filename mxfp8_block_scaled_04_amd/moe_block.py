"""Blocks of a transformer around the expert computation, forward and backward:
the residual's addition and the root-mean-square norm in front, then the routed
experts with their router (MoEBlock) or one dense MXFP8 layer (DenseBlock, as
the first layers of such a model are).  A block takes the output of the
sub-layer before it and the residual stream, and returns its own output and the
new stream; the next block adds the two.

  MoEBlock    h = x + residual, y = norm(h)            mx_rms_norm
              logits = y gate^T                        mx_grouped_gemm_bf16 (one group)
              experts, weights                         mx_router
              out = experts of y, weighted             RoutedMoELayer.forward
    backward  d weights = dout . expert outputs        mx_combine_dweights
              d logits                                 mx_router_backward
              d gate, d y (the router's part)          mx_grouped_gemm_bf16_wgrad, _dgrad
              d y (the experts' part), dW1, dW2        RoutedMoELayer.backward
              d h, d norm                              mx_rms_norm_backward (both parts of d y, and the stream's)
  DenseBlock  h, y, and MXFP8 rows of y                mx_rms_norm
              y^T in MXFP8 for the weight gradient     mx_quantize_cols
              out = SwiGLU layer of y                  MoELayer.forward_experts (one group)
    backward  MoELayer.backward, mx_rms_norm_backward

Gradients of the weights are those of one step (MoELayer's in bf16, the gate's
and the norm's in float32).  backward returns the gradient of the sum in the
stream's type, which the block before takes as its dh, and leaves it in dx in
bf16, which that block takes as its dout.  The router's logits are bf16, as the
product writes them: equal ones go to the lower index.  Without a residual the
input is the stream itself, which backward reads again: it has to stay as it is
until then.  Buffers are allocated once; every step runs in the library's
kernels on the current stream of the block's GPU and can be captured.  A block's
outputs are its own buffers: they hold until its next call.
"""
import contextlib

import torch

from . import mx_quantize_cols
from .block import (_current_device, _matrix, _one_gpu, mx_combine_dweights, mx_rms_norm, mx_rms_norm_backward,
                    mx_rms_norm_backward_workspace_bytes, mx_router, mx_router_backward)
from .moe_layer import MoELayer, RoutedMoELayer
from .training import (mx_grouped_gemm_bf16, mx_grouped_gemm_bf16_dgrad, mx_grouped_gemm_bf16_wgrad,
                       mx_grouped_gemm_bf16_wgrad_workspace_bytes)


def _gpu_of(buffer):
    """The block's GPU as the current one: the calls of moe_layer and the products run on the current GPU's stream."""
    at = buffer.get_device()  # -1: not on a GPU
    return contextlib.nullcontext() if at < 0 or at == _current_device() else torch.cuda.device(at)


class _Norm:
    """Buffers and calls of the norm in front of a block of T tokens."""

    def __init__(self, T, H, eps, stream_dtype, device):
        self.eps = eps
        self.sum = torch.empty((T, H), dtype=stream_dtype, device=device)
        self.h = None  # the sum, or the input where there is no residual
        self.y = torch.empty((T, H), dtype=torch.bfloat16, device=device)
        self.rstd = torch.empty(T, dtype=torch.float32, device=device)
        self.dh = torch.empty((T, H), dtype=stream_dtype, device=device)
        # in bf16, as the sub-layer whose output x is takes it
        self.dx = self.dh if stream_dtype is torch.bfloat16 else torch.empty((T, H), dtype=torch.bfloat16, device=device)
        self.dweight = torch.empty(H, dtype=torch.float32, device=device)
        self.workspace = torch.empty(mx_rms_norm_backward_workspace_bytes(T, H), dtype=torch.uint8, device=device)

    def forward(self, x, residual, weight, q=None, s=None):
        if residual is None and x.dtype != self.sum.dtype:
            raise ValueError("without a residual the input is the stream, and has its type")
        h = mx_rms_norm(x, weight, residual=residual, eps=self.eps, h=None if residual is None else self.sum, y=self.y,
                        q=q, s=s, rstd=self.rstd)[1]
        self.h = x if residual is None else h
        return self.y

    def check(self, dout):
        """Before a backward pass: there is a forward pass whose rows it reads, and dout is of its rows."""
        if self.h is None:
            raise ValueError("backward needs a forward pass before it")
        _matrix(dout, "dout", (torch.bfloat16,), *self.y.shape)
        _one_gpu(self.y, dout)

    def backward(self, dy, weight, dh, dy2=None):
        mx_rms_norm_backward(dy, self.h, weight, self.rstd, dy2=dy2, dh_in=dh, dh=self.dh,
                             dx=None if self.dx is self.dh else self.dx, dweight=self.dweight, workspace=self.workspace)
        return self.dh


class MoEBlock:
    """T tokens of H columns, routed to k of E experts of width I (E % 8 == 0).
    score, renorm, scale, groups, groups_kept, group_top: as mx_router.
    stream_dtype: bf16 or float32, of the residual stream."""

    def __init__(self, T, k, E, H, I, device="cuda", score="softmax", renorm=True, scale=1.0, groups=1,
                 groups_kept=None, group_top=2, eps=1e-6, stream_dtype=torch.bfloat16):
        if E % 8:
            raise ValueError("the number of experts must be a multiple of 8 (of the gate's product)")
        self.T, self.k, self.E, self.H, self.I = T, k, E, H, I
        self.routed = RoutedMoELayer(T, k, E, H, I, device)
        self.norm = _Norm(T, H, eps, stream_dtype, device)
        self.dx = self.norm.dx
        self.weighting = {"score": score, "renorm": renorm, "scale": scale}
        self.choice = {"groups": groups, "groups_kept": groups_kept, "group_top": group_top}
        self.all_rows = torch.tensor([0, T], dtype=torch.int32, device=device)
        self.logits = torch.empty((T, E), dtype=torch.bfloat16, device=device)
        self.dlogits = torch.empty((T, E), dtype=torch.bfloat16, device=device)
        self.experts = torch.empty((T, k), dtype=torch.int32, device=device)
        self.weights = torch.empty((T, k), dtype=torch.float32, device=device)
        self.dweights = torch.empty((T, k), dtype=torch.float32, device=device)
        self.dy = torch.empty((T, H), dtype=torch.bfloat16, device=device)
        self.dgate = torch.empty((1, E, H), dtype=torch.float32, device=device)
        self.gate_workspace = torch.empty(max(0, mx_grouped_gemm_bf16_wgrad_workspace_bytes(1, T, E, H)),
                                          dtype=torch.uint8, device=device)

    def quantize_weights(self, W1, W2):
        """After every change of the experts' weights: bf16 [E, 2I, H] in swiglu_interleave order and [E, H, I]."""
        _one_gpu(self.norm.y, W1, W2)
        with _gpu_of(self.norm.y):
            self.routed.layer.quantize_weights(W1, W2)

    def forward(self, x, residual, norm_weight, gate, bias=None):
        """x bf16 [T, H] (or the stream itself, with residual None), gate bf16
        [E, H], bias float32 [E] or None (for the choice only).  Returns (out
        bf16 [T, H], h): the block's output and the new residual stream."""
        with _gpu_of(self.norm.y):
            y = self.norm.forward(x, residual, norm_weight)
            mx_grouped_gemm_bf16(y, gate.unsqueeze(0), self.all_rows, out=self.logits)
            mx_router(self.logits, self.k, bias=bias, experts=self.experts, weights=self.weights, **self.choice,
                      **self.weighting)
            return self.routed.forward(y, self.experts, self.weights), self.norm.h

    def backward(self, dout, dh, norm_weight, gate):
        """After forward: dout bf16 [T, H] and dh (the stream's gradient, or
        None) -> (dh of x and of the residual, dW1, dW2, dgate [E, H], dnorm)."""
        self.norm.check(dout)
        with _gpu_of(self.norm.y):
            mx_combine_dweights(dout, self.routed.layer.y, self.routed.slot_of, dweights=self.dweights)
            mx_router_backward(self.logits, self.experts, self.dweights, dlogits=self.dlogits, **self.weighting)
            mx_grouped_gemm_bf16_wgrad(self.dlogits, self.norm.y, self.all_rows, dw=self.dgate,
                                       workspace=self.gate_workspace)
            mx_grouped_gemm_bf16_dgrad(self.dlogits, gate.unsqueeze(0), self.all_rows, dx=self.dy)
            dy, dW1, dW2 = self.routed.backward(dout)
            dx = self.norm.backward(dy, norm_weight, dh, self.dy)
            return dx, dW1, dW2, self.dgate[0], self.norm.dweight


class DenseBlock:
    """T tokens of H columns through one SwiGLU layer of width I in MXFP8.
    training=False leaves out the column-wise quantization of y, which only the
    backward pass reads, and refuses that pass."""

    def __init__(self, T, H, I, device="cuda", eps=1e-6, stream_dtype=torch.bfloat16, training=True):
        self.T, self.H, self.I, self.training = T, H, I, training
        self.all_rows = torch.tensor([0, T], dtype=torch.int32, device=device)
        self.layer = MoELayer(self.all_rows, T, H, I, device)
        self.norm = _Norm(T, H, eps, stream_dtype, device)
        self.dx = self.norm.dx

    def quantize_weights(self, W1, W2):
        """After every change of the weights: bf16 [1, 2I, H] in swiglu_interleave order and [1, H, I]."""
        _one_gpu(self.norm.y, W1, W2)
        with _gpu_of(self.norm.y):
            self.layer.quantize_weights(W1, W2)

    def forward(self, x, residual, norm_weight):
        """x bf16 [T, H] (or the stream itself, with residual None).  Returns (out bf16 [T, H], h)."""
        with _gpu_of(self.norm.y):
            X = self.layer.x
            y = self.norm.forward(x, residual, norm_weight, X.q, X.s)
            if self.training:
                mx_quantize_cols(y, self.all_rows, X.Mcap, X.qT, X.sT, X.P)
            return self.layer.forward_experts(), self.norm.h

    def backward(self, dout, dh, norm_weight):
        """After forward -> (dh of x and of the residual, dW1, dW2, dnorm)."""
        if not self.training:
            raise ValueError("a block made with training=False has no backward pass")
        self.norm.check(dout)
        with _gpu_of(self.norm.y):
            dy, dW1, dW2 = self.layer.backward(dout)
            return self.norm.backward(dy, norm_weight, dh), dW1, dW2, self.norm.dweight
