"""A mixture of experts' gated MLP over quantized weights.

``RoutedExperts`` runs what follows a router's logits:

    moe_route -> product with the experts' gate and up weights, silu(gate) * up
              -> product with their down weights -> moe_combine

with NVFP4 W4A4 products for prompts and INT4 weight-only ones for decoding, as
the pages split a model between prefill and decode (Disaggregated
Quantization).  Nothing is read back: how many rows an expert gets stays on the
device.  Every kernel is the library's; this module holds the weights and the
order of the calls.
"""

import torch

from . import qlin
from .attention import DECODE_TOKENS


class RoutedExperts:
    """up fp32 [experts, 2 * inter, hidden] (each expert's gate rows, then its
    up rows) and down fp32 [experts, hidden, inter] on the GPU, quantized to
    INT4 group-128 (for decoding) and NVFP4 (for prompts)."""

    def __init__(self, up, down, top_k, renormalize=True):
        experts, rows, hidden = up.shape
        if rows % 2 or down.shape != (experts, hidden, rows // 2):
            raise ValueError(f"up must be [experts, 2 * inter, hidden] and down [experts, hidden, inter], got "
                             f"{list(up.shape)}, {list(down.shape)}")
        self.experts, self.top_k, self.renormalize = experts, top_k, renormalize
        self.hidden, self.inter = hidden, rows // 2
        self.weights = []
        for w in (up, down):
            n, k = w.shape[1:]
            few = self._stack(w, qlin.QL_INT4_G128, qlin.quantize_int4_g128)
            many = self._stack(w, qlin.QL_NVFP4, qlin.quantize_nvfp4)
            self.weights.append((few, many, n, k))

    def _stack(self, w, fmt, quantize):
        n, k = w.shape[1:]
        stack = torch.empty((self.experts, qlin.repack_weights_bytes(fmt, n, k)), dtype=torch.uint8,
                            device=w.device)
        for blob, we in zip(stack, w):
            qlin.repack_weights(fmt, n, k, *quantize(we.contiguous()), packed=blob)
        return stack

    def product(self, x, which, plan, prompt):
        """Product `which` (0 gate and up with their activation, 1 down) of the
        plan's rows, in its order."""
        few, many, n, k = self.weights[which]
        up = which == 0
        if prompt:
            return qlin.moe_gemm_w4a4(*qlin.quantize_nvfp4(x), many, plan, n, k, gather=up, silu_mul=up)
        return qlin.moe_gemm_w4a16(x, few, plan, n, k, gather=up, silu_mul=up)

    def forward(self, x, logits, prompt=None):
        """x bf16 [tokens, hidden] and the router's logits [tokens, experts] (an
        expert at -infinity is not chosen; a token that may choose none gets
        zeros) -> bf16 [tokens, hidden].  prompt: whether these are tokens of
        prompts (NVFP4 weights and activations, these under one tensor scale for
        all rows of a product) or of decoding (INT4 weights); not told: by their
        number."""
        if logits.shape[1] != self.experts or logits.shape[0] != x.shape[0]:
            raise ValueError(f"logits must be [{x.shape[0]}, {self.experts}], got {list(logits.shape)}")
        if prompt is None:
            prompt = x.shape[0] > DECODE_TOKENS
        _, weights, plan = qlin.moe_route(logits, self.top_k, self.renormalize)
        h = self.product(x, 0, plan, prompt)
        return qlin.moe_combine(self.product(h, 1, plan, prompt), plan, weights)
