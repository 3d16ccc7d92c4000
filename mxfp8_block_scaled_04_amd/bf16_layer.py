"""The expert computation of one MoE layer in bf16, forward and backward: the
unquantized counterpart of moe_layer.MoELayer, for layers that a recipe keeps
out of MXFP8 and for judging the quantized ones.  Same shapes and the same
weight layout (W1 [G, 2I, H] in swiglu_interleave order, W2 [G, H, I], group
offsets [G+1]), so that a layer can be switched between the two.

  forward   preact = X W1^T               mx_grouped_gemm_bf16
            h = silu(gate) up             mx_swiglu_backward (its h output)
            Y = h W2^T                    mx_grouped_gemm_bf16
  backward  dH = dY W2                    mx_grouped_gemm_bf16_dgrad
            d(gate, up)                   mx_swiglu_backward
            dW2 (+)= dY^T h               mx_grouped_gemm_bf16_wgrad
            dX = d(gate, up) W1           mx_grouped_gemm_bf16_dgrad
            dW1 (+)= d(gate, up)^T X      mx_grouped_gemm_bf16_wgrad

h comes from the backward kernel, which writes d(gate, up) too: 133 us at 32768
rows and I 2048, about twice what h alone has to move, in a step of 8.0 ms
(H 7168, 16 groups, fp32 gradients; 1.08 PFLOP/s of its products).

With fp32_grads the weight gradients are float32 and backward(accumulate=True)
adds to them (micro-batches); else they are bf16.  Buffers are allocated once;
every step runs in the library's kernels on the current stream.
"""
import torch

from . import mx_swiglu_backward
from .training import mx_grouped_gemm_bf16, mx_grouped_gemm_bf16_dgrad, mx_grouped_gemm_bf16_wgrad


class Bf16Layer:
    """Buffers and calls of one layer for fixed M, H, I and group count."""

    def __init__(self, offsets, M, H, I, device="cuda", fp32_grads=False):
        G = offsets.numel() - 1

        def bf16(*shape):
            return torch.empty(shape, dtype=torch.bfloat16, device=device)

        self.offsets, self.M, self.H, self.I, self.G = offsets, M, H, I, G
        self.preact, self.dpre = bf16(M, 2 * I), bf16(M, 2 * I)
        self.h, self.dh = bf16(M, I), bf16(M, I)
        self.y, self.dx = bf16(M, H), bf16(M, H)
        kind = torch.float32 if fp32_grads else torch.bfloat16
        self.dW1 = torch.zeros((G, 2 * I, H), dtype=kind, device=device)
        self.dW2 = torch.zeros((G, H, I), dtype=kind, device=device)

    def flops(self):
        """Matrix flops of one forward + backward over the routed rows."""
        return 3 * (2 * self.M * (2 * self.I) * self.H + 2 * self.M * self.H * self.I)

    def forward(self, X, W1, W2):
        mx_grouped_gemm_bf16(X, W1, self.offsets, out=self.preact)
        # h does not depend on dh, and d(gate, up) is written again by backward()
        mx_swiglu_backward(self.preact, self.dh, dpre=self.dpre, h=self.h)
        return mx_grouped_gemm_bf16(self.h, W2, self.offsets, out=self.y)

    def backward(self, X, dY, W1, W2, accumulate=False):
        """After forward(X, W1, W2).  Returns (dX, dW1, dW2)."""
        off = self.offsets
        mx_grouped_gemm_bf16_dgrad(dY, W2, off, dx=self.dh)
        mx_swiglu_backward(self.preact, self.dh, dpre=self.dpre)
        mx_grouped_gemm_bf16_wgrad(dY, self.h, off, dw=self.dW2, accumulate=accumulate)
        mx_grouped_gemm_bf16_dgrad(self.dpre, W1, off, dx=self.dx)
        mx_grouped_gemm_bf16_wgrad(self.dpre, X, off, dw=self.dW1, accumulate=accumulate)
        return self.dx, self.dW1, self.dW2
