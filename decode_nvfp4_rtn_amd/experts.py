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
        with torch.cuda.device(up.device):     # the quantizers go by the current device
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

    def forward(self, x, logits, prompt=None, step=None):
        """x bf16 [tokens, hidden] and the router's logits [tokens, experts] (an
        expert at -infinity is not chosen; a token that may choose none gets
        zeros) -> bf16 [tokens, hidden].  prompt: whether these are tokens of
        prompts (NVFP4 weights and activations, these under one tensor scale for
        all rows of a product, so that rows of tokens without an expert have to be
        finite too) or of decoding (INT4 weights).  step: instead, the
        attention.Step whose new tokens they are, each sequence's by its kind, with
        the calls made for every run of sequences of one kind.  Neither told: by
        their number."""
        if torch._C._cuda_getDevice() != x.device.index:   # the quantizer goes by the current device
            with torch.cuda.device(x.device):
                return self.forward(x, logits, prompt, step)
        if logits.shape[1] != self.experts or logits.shape[0] != x.shape[0]:
            raise ValueError(f"logits must be [{x.shape[0]}, {self.experts}], got {list(logits.shape)}")
        runs = None
        if step is not None:
            if prompt is not None or sum(step.nodes) != x.shape[0]:
                raise ValueError(f"a step of {sum(step.nodes)} new tokens takes as many rows, got {x.shape[0]}, "
                                 f"and no prompt")
            runs = step.runs()
        if runs is not None and len(runs) < 2:
            prompt = runs[0][0] if runs else False
        elif runs is not None:
            out = torch.empty((x.shape[0], self.hidden), dtype=torch.bfloat16, device=x.device)
            at = 0
            for kind, n in runs:
                self._rows(x[at:at + n], logits[at:at + n], kind, out[at:at + n])
                at += n
            return out
        elif prompt is None:
            prompt = x.shape[0] > DECODE_TOKENS
        return self._rows(x, logits, prompt)

    def _rows(self, x, logits, prompt, out=None):
        """The layer of rows of one kind."""
        _, weights, plan = qlin.moe_route(logits, self.top_k, self.renormalize)
        h = self.product(x, 0, plan, prompt)
        return qlin.moe_combine(self.product(h, 1, plan, prompt), plan, weights, out)
