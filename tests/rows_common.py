"""Inputs and error bounds shared by the tests of layers whose rows choose
their weights."""

import numpy as np
import torch

from decode_nvfp4_rtn_amd import synth
from oracle import int4, nvfp4, rows
from oracle.gemm import TOL
from tests.gpu_common import dev_bf16, dev_f32, host_f64


def choices(seed, tokens, experts, top_k, idle=0.0, only=None):
    """int32 choices [tokens, top_k], no expert twice for a token; the share
    `idle` of tokens has none; only: the experts that are chosen from."""
    rng = np.random.default_rng([91, seed])
    among = np.arange(experts) if only is None else np.asarray(only)
    ids = np.stack([rng.permutation(among)[:top_k] for _ in range(tokens)]).astype(np.int32)
    ids = ids.reshape(tokens, top_k)
    ids[rng.random(tokens) < idle] = -1
    return ids


def bf16_rows(seed, count, cols):
    """bf16 bits of rows of uneven size with loud channels, and their values."""
    rng = np.random.default_rng([92, seed])
    x = rng.standard_normal((count, cols)).astype(np.float32)
    x *= np.where(rng.random(cols) < 0.02, 8.0, 1.0).astype(np.float32)
    x *= np.exp(0.4 * rng.standard_normal((count, 1))).astype(np.float32)
    bits = synth.to_bf16_bits(x)
    return bits, synth.bf16_bits_as_f32(bits)


class Stack:
    """Every expert's quantized weights: float64 values and the blobs."""

    def __init__(self, q, fmt, seed, experts, n, k, spare=0):
        rng = np.random.default_rng([93, seed])
        self.values, f = [], q.QL_INT4_G128 if fmt == "int4" else q.QL_NVFP4
        size = q.repack_weights_bytes(f, n, k)
        self.blobs = torch.full((experts, size + spare), 0xA5, dtype=torch.uint8, device="cuda")
        for e in range(experts):
            w = (rng.standard_normal((n, k)) * k ** -0.5).astype(np.float32)
            parts = int4.quantize(w) if fmt == "int4" else nvfp4.quantize(w)
            self.values.append(rows.weights_of(fmt, parts))
            on = [torch.from_numpy(np.ascontiguousarray(p).view(np.int16 if p.dtype == np.uint16 else p.dtype)).cuda()
                  for p in parts[:2]]
            if fmt != "int4":
                on.append(dev_f32(np.array([parts[2]])))
            q.repack_weights(f, n, k, *on, packed=self.blobs[e, :size])


def operand(q, fmt, bits):
    """(what the product takes of bf16 rows, their float64 values)."""
    if fmt == "int4":
        return (dev_bf16(bits),), synth.bf16_bits_as_f32(bits).astype(np.float64)
    parts = nvfp4.quantize(synth.bf16_bits_as_f32(bits))
    on = (torch.from_numpy(parts[0]).cuda(), torch.from_numpy(parts[1]).cuda(), dev_f32(np.array([parts[2]])))
    return on, nvfp4.dequantize(*parts)


def product(q, fmt, *args, **kw):
    return (q.moe_gemm_w4a16 if fmt == "int4" else q.moe_gemm_w4a4)(*args, **kw)


def half_step(v, dtype):
    """Half a step of the output's type at |v|, and of its least numbers."""
    return torch.finfo(dtype).eps / 2 * np.abs(v) + 2.0 ** -134


def product_bound(ref, dtype):
    """The library's rule for products (1e-3 of the RMS) and the output's rounding."""
    slack = TOL * np.sqrt(np.mean(ref ** 2)) if ref.size else 0.0
    return slack + half_step(np.abs(ref) + slack, dtype)


def silu_bound(gate, up, dtype):
    """The same for silu(gate) * up: |silu'| <= 1.1, each factor off by the rule's
    slack; the exponential, the division and two products round by 2^-20 at most."""
    h = rows.silu(gate) * up
    dg, du = (TOL * np.sqrt(np.mean(v ** 2)) if v.size else 0.0 for v in (gate, up))
    slack = 1.1 * dg * (np.abs(up) + du) + np.abs(rows.silu(gate)) * du + 2.0 ** -20 * np.abs(h)
    return h, slack + half_step(np.abs(h) + slack, dtype)


def check(got, want, bound, what=""):
    far = np.abs(host_f64(got) - want)
    bad = ~(far <= bound)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4].tolist(), float((far / bound).max()))
