"""The layer of decode_nvfp4_rtn_amd/attention.py: a prompt, drafted trees, their
commit and single tokens, each step against the float64 definition."""

import numpy as np
import pytest
import torch

from decode_nvfp4_rtn_amd import synth
from oracle import kvcache as kv
from tests.gpu_common import require_gpu, say
from tests.kv_common import FMTS

pytestmark = pytest.mark.gpu

HIDDEN, N_Q, N_KV, D, PAGE = 512, 4, 2, 128, 16


def _layer(q, fmt, seed=1):
    from decode_nvfp4_rtn_amd.attention import PagedAttention, rope_table
    cache = q.KVCache(FMTS[fmt], 24, PAGE, N_KV, D)
    w = [torch.from_numpy(synth.weights(1, seed + i, n, k)).cuda()
         for i, (n, k) in enumerate((((N_Q + 2 * N_KV) * D, HIDDEN), (HIDDEN, N_Q * D)))]
    wq, wk = (1 + 0.1 * torch.randn(D, generator=torch.Generator().manual_seed(i)) for i in (1, 2))
    return PagedAttention(cache, *w, N_Q, rope_table(256, D), wq.cuda(), wk.cuda())


def _x(tokens, seed):
    return torch.randn((tokens, HIDDEN), generator=torch.Generator().manual_seed(seed)).cuda().bfloat16()


class Mirror:
    """The layer's steps in float64, from the projections' own outputs."""

    def __init__(self, layer, fmt):
        self.layer, self.c = layer, kv.Cache(FMTS[fmt], 24, PAGE, N_KV, D)

    def step(self, x, step, seqs, p):
        qkv = self.layer.project(x, 0).double().cpu().numpy().reshape(x.shape[0], -1, D)
        pos, slots = step.positions.cpu().numpy(), step.slots.cpu().numpy()
        args = (1e-6, self.layer.rope.cpu().numpy(), pos, False)
        wq, wk = (w.double().cpu().numpy() for w in (self.layer.q_weight, self.layer.k_weight))
        qr = kv.norm_rope(qkv[:, :N_Q], wq, *args)
        self.c.write("k", kv.norm_rope(qkv[:, N_Q:N_Q + N_KV], wk, *args), slots)
        self.c.write("v", qkv[:, N_Q + N_KV:].astype(np.float32), slots)
        # the queries are rounded to bf16 (half a step 2^-9) before the products
        y, bound = np.zeros((x.shape[0], N_Q, D)), np.zeros((x.shape[0], N_Q, D))
        at, tree = 0, None if step.tree is None else step.tree.cpu().numpy().astype(np.uint64)
        for s, n in zip(seqs, step.nodes):
            length = p.lens[s] + n
            t = slice(at, at + n)
            here = np.arange(length)
            rows = np.array(p.pages[s])[here // PAGE] * PAGE + here % PAGE
            sees = kv.visible(n, length, None if tree is None else tree[t])
            y[t], mag, top, unit = kv.attention(qr[t], self.c.value["k"][rows], self.c.value["v"][rows],
                                                sees, D ** -0.5, self.c.exp["v"][rows])
            bound[t] = (2.0 ** -8 * np.abs(y[t]) + 2.0 ** -32 * unit +
                        (2.0 ** -10 + 4 * (2.0 ** -9 + D * 2.0 ** -24) * top[..., None]) * mag)
            at += n
        return y, bound


@pytest.mark.parametrize("fmt", list(FMTS))
def test_prompt_drafts_commit_decode(fmt):
    q = require_gpu()
    say("layer", fmt)
    from decode_nvfp4_rtn_amd.attention import PagedSequences
    layer, p = _layer(q, fmt), PagedSequences(24, PAGE)
    m = Mirror(layer, fmt)
    taken = []
    call = q.kv_attention

    def attention(*a, **k):
        taken.append(call(*a, **k))
        return taken[-1]

    def run(nodes, seed, tree=None):
        x = _x(sum(nodes), seed)
        step = p.step(seqs, nodes, tree)
        want, bound = m.step(x, step, seqs, p)
        q.kv_attention = attention
        try:
            out = layer.forward(x, step)
        finally:
            q.kv_attention = call
        got = taken[-1]
        assert np.all(np.abs(got.double().cpu().numpy() - want) <= bound)
        assert torch.equal(out, layer.project(got.flatten(1), 1)) and torch.isfinite(out).all()
        return step

    seqs = [p.add(), p.add()]
    run([70, 9], 1)                                         # prompts (W4A4 projections)
    p.settle(seqs, [70, 9])
    run([20, 30], 2)                                        # their second chunks
    p.settle(seqs, [20, 30])
    tree = [[1, 3, 5, 11, 19], [1, 2, 5, 13, 13 + 16]]
    step = run([5, 5], 3, tree)
    path = torch.tensor([[0, 1, 4], [0, 2, -1]], dtype=torch.int32, device="cuda")
    layer.commit(step, path)
    for b, (s, kept) in enumerate(zip(seqs, ([0, 1, 4], [0, 2]))):
        rows = step.slots.cpu().numpy()[5 * b:5 * b + 5]
        m.c.move([(rows[i], rows[j]) for j, i in enumerate(kept)])
    p.settle(seqs, [3, 2])
    for seed in (4, 5):                                     # single tokens over what was kept
        run([1, 1], seed)
        p.settle(seqs, [1, 1])
    assert p.lens == {seqs[0]: 95, seqs[1]: 43}
