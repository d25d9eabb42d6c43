"""Inputs and caches shared by the key/value-cache tests."""

import numpy as np
import torch

from decode_nvfp4_rtn_amd import synth
from oracle import kvcache as kv

FMTS = {"bf16": kv.BF16, "e4m3": kv.E4M3, "nvfp4": kv.NVFP4}


def rows(seed, tokens, heads, d, bf16=True):
    """float32 rows [tokens, heads, d] of uneven size with loud channels; bf16
    values if asked."""
    rng = np.random.default_rng([77, seed])
    x = rng.standard_normal((tokens, heads, d)).astype(np.float32)
    x *= np.where(rng.random((heads, d)) < 0.03, 8.0, 1.0).astype(np.float32)
    x *= np.exp(0.5 * rng.standard_normal((tokens, heads, 1))).astype(np.float32)
    return synth.bf16_bits_as_f32(synth.to_bf16_bits(x)).reshape(x.shape) if bf16 else x


def on_gpu(x, bf16=True):
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t.to(torch.bfloat16) if bf16 else t


def device_cache(qlin, c):
    """A KVCache holding the bytes of the oracle's Cache c."""
    return qlin.KVCache(c.fmt, c.n_pages, c.page, c.n_kv, c.d,
                        data=torch.from_numpy(c.bytes.copy()).cuda())


class Batch:
    """Sequences of given key counts and new tokens over shuffled pages, their
    rows written through the oracle; the rest of the cache holds `fill`."""

    def __init__(self, fmt, lens, nodes, n_q, n_kv, d, page=16, seed=0, fill=0xFF, spare=1,
                 scale_rows=None):
        rng = np.random.default_rng([78, seed])
        self.lens, self.nodes, self.n_q, self.n_kv, self.d = lens, nodes, n_q, n_kv, d
        need = [-(-n // page) for n in lens]
        pages = max(1, sum(need) + spare)
        perm = rng.permutation(pages)
        self.c = kv.Cache(fmt, pages, page, n_kv, d, fill)
        self.table = np.full((len(lens), max(need + [1]) + 2), -1, dtype=np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n]
            at += n
        for which in "kv":
            for b, n in enumerate(lens):
                x = rows(seed * 100 + b * 2 + (which == "v"), n, n_kv, d)
                if scale_rows is not None:
                    x = x * scale_rows(which, b, n).astype(np.float32)[:, None, None]
                self.c.write(which, x, self.slots(b, np.arange(n)))
        self.q = rows(seed + 5000, sum(nodes), n_q, d) * np.float32(0.5)
        self.cu = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)

    def slots(self, b, pos):
        pos = np.asarray(pos)
        return self.table[b, pos // self.c.page].astype(np.int64) * self.c.page + pos % self.c.page

    def reference(self, tree=None, scale=None, hidden=None):
        """(y, bound) [tokens, n_q, d]: the definition in float64 and how far a
        bf16 result computed as include/qlin.h says may be from it.

        bound: half a bf16 step of the result and of what it is rounded from
        (2^-8 |y|), the weights' rounding to 11 bits and the binary32 sums
        (2^-10 of the mean |v| under the weights), the scores' error: a
        binary32 sum of d products is off by at most d 2^-24 of the sum of
        their magnitudes, twice that relative in a weight and its normaliser,
        and in quantized rows the small weights' rounding to a multiple of
        2^-31 of the largest weight 2^e."""
        scale = self.d ** -0.5 if scale is None else scale
        y = np.zeros((sum(self.nodes), self.n_q, self.d))
        bound = np.zeros_like(y)
        for b, n in enumerate(self.lens):
            t = slice(self.cu[b], self.cu[b + 1])
            s = self.slots(b, np.arange(n))
            k, v = self.c.value["k"][s], self.c.value["v"][s]
            sees = kv.visible(self.nodes[b], n, None if tree is None else tree[t])
            if hidden is not None:
                sees = sees & ~hidden[b][None, :n]
            y[t], mag, top, unit = kv.attention(self.q[t].astype(np.float64), k, v, sees, scale,
                                                self.c.exp["v"][s])
            bound[t] = 2.0 ** -8 * np.abs(y[t]) + (2.0 ** -10 + 4 * self.d * 2.0 ** -24 * top[..., None]) * mag
            if self.c.fmt != kv.BF16:
                bound[t] += 2.0 ** -32 * unit
        return y, bound + 1e-35

    def run(self, qlin, tree=None, scale=None, max_q=None, max_kv=None, **kw):
        cache = device_cache(qlin, self.c)
        y = qlin.kv_attention(
            cache, on_gpu(self.q), torch.from_numpy(self.cu).cuda(),
            torch.tensor(self.lens, dtype=torch.int32, device="cuda"),
            torch.from_numpy(self.table).cuda(), max(self.nodes) if max_q is None else max_q,
            max(self.lens) if max_kv is None else max_kv,
            tree=None if tree is None else torch.tensor(
                [int(m) - (1 << 64) if int(m) >> 63 else int(m) for m in tree],
                dtype=torch.int64, device="cuda"), scale=scale, **kw)
        torch.cuda.synchronize()
        return y

    def check(self, y, tree=None, scale=None, hidden=None):
        want, bound = self.reference(tree, scale, hidden)
        got = y.float().cpu().numpy().astype(np.float64)
        assert np.all(np.isfinite(got))
        off = np.abs(got - want) / bound
        assert off.max() <= 1.0, (off.max(), np.unravel_index(off.argmax(), off.shape))


def random_tree(nodes, seed):
    """Ancestor masks of random trees, one after another for each count."""
    rng = np.random.default_rng([79, seed])
    out = []
    for n in nodes:
        m = []
        for j in range(n):
            parent = int(rng.integers(-1, j)) if j else -1
            m.append((m[parent] if parent >= 0 else 0) | 1 << j)
        out += m
    return np.array(out, dtype=object)
