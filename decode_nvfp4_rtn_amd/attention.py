"""A decoder layer's attention between its two quantized projections, with the
keys and values of many sequences in one paged cache.

``PagedSequences`` is the host's side: which pages each sequence holds, how many
of its tokens are settled, and the integer arrays that the calls of a step take.
``PagedAttention`` runs a step of one layer:

    qkv projection -> qkv_norm_rope_append -> kv_attention -> output projection

with NVFP4 W4A4 projections for prompts and INT4 weight-only ones for decoding,
as the pages split a model between prefill and decode (Disaggregated
Quantization).  A step's new tokens are a chain (a chunk of a prompt, one token
of decoding) or, for speculative decoding, a tree of drafts of which ``commit``
keeps a path.  Which weights a sequence's tokens meet goes by what they are, not
by how many sequences share the step.  Every kernel is the library's; this module holds the weights,
the cache and the order of the calls.
"""

from dataclasses import dataclass

import numpy as np
import torch

from . import qlin

DECODE_TOKENS = 32      # rows up to which ``project`` takes INT4 weights if not told


@dataclass
class Step:
    """One step's arrays: new tokens per sequence, and on the device where they
    start, the lengths with them, the pages, each token's slot and position and
    (a tree) which drafts it sees.  prompt: for each sequence, whether its new
    tokens are of its prompt (None: not said)."""
    nodes: list
    max_kv: int
    cu_q: torch.Tensor
    kv_lens: torch.Tensor
    block_table: torch.Tensor
    slots: torch.Tensor
    positions: torch.Tensor
    tree: torch.Tensor
    prompt: list = None


class PagedSequences:
    """Sequences over the pages of a cache.  A sequence keeps its pages until
    ``free``; drafts that were not accepted are overwritten by the next step."""

    def __init__(self, n_pages, page_size, device="cuda"):
        self.page_size, self.device = page_size, torch.device(device)
        self.unused = list(range(n_pages - 1, -1, -1))
        self.pages, self.lens = {}, {}
        self.next_id = 0

    def add(self):
        """A new, empty sequence's number."""
        s, self.next_id = self.next_id, self.next_id + 1
        self.pages[s], self.lens[s] = [], 0
        return s

    def free(self, s):
        self.unused += reversed(self.pages.pop(s))
        del self.lens[s]

    def step(self, seqs, nodes, tree=None, prompt=None):
        """Room for `nodes` new tokens of each of `seqs` (distinct) and the
        step's arrays.  tree: for each sequence its drafts' ancestor masks
        (integers, bit i of entry i set); None: chains.  prompt: for each
        sequence whether these are tokens of its prompt; None: those of chains
        that are longer than one token or begin a sequence."""
        if len(set(seqs)) != len(seqs) or len(nodes) != len(seqs) or min(nodes, default=1) < 0:
            raise ValueError("a step takes distinct sequences and a token count for each")
        if tree is not None and [len(m) for m in tree] != list(nodes):
            raise ValueError("a tree takes one mask for each new token")
        if prompt is not None and len(prompt) != len(seqs):
            raise ValueError("prompt takes a truth value for each sequence")
        if prompt is None:
            prompt = [tree is None and (n > 1 or self.lens[s] == 0) for s, n in zip(seqs, nodes)]
        total = [self.lens[s] + n for s, n in zip(seqs, nodes)]
        need = [max(0, -(-t // self.page_size) - len(self.pages[s])) for s, t in zip(seqs, total)]
        if sum(need) > len(self.unused):
            raise RuntimeError(f"{sum(need)} pages needed, {len(self.unused)} unused")
        for s, n in zip(seqs, need):
            self.pages[s] += [self.unused.pop() for _ in range(n)]
        table = np.full((len(seqs), max([len(self.pages[s]) for s in seqs] + [1])), -1, np.int32)
        slots, positions, masks = [], [], []
        for b, (s, n) in enumerate(zip(seqs, nodes)):
            table[b, :len(self.pages[s])] = self.pages[s]
            at = self.lens[s] + np.arange(n)
            slots.append(table[b, at // self.page_size].astype(np.int64) * self.page_size
                         + at % self.page_size)
            if tree is None:
                positions.append(at)
            else:     # a draft's depth: its ancestors
                depth = [bin(int(m)).count("1") - 1 for m in tree[b]]
                positions.append(self.lens[s] + np.array(depth, dtype=np.int64))
                masks += [int(m) - (1 << 64) if int(m) >> 63 else int(m) for m in tree[b]]

        def dev(x, dtype):
            return torch.from_numpy(np.ascontiguousarray(x, dtype=dtype)).to(self.device)
        return Step(list(nodes), max(total, default=0),
                    dev(np.concatenate([[0], np.cumsum(nodes)]), np.int32), dev(total, np.int32),
                    dev(table, np.int32), dev(np.concatenate(slots or [[]]), np.int64),
                    dev(np.concatenate(positions or [[]]), np.int32),
                    None if tree is None else dev(np.array(masks, dtype=np.int64), np.int64),
                    [bool(p) for p in prompt])

    def settle(self, seqs, counts):
        """`counts` of the last step's tokens now belong to each sequence."""
        for s, n in zip(seqs, counts):
            self.lens[s] += n


def rope_table(max_pos, rot, base=10000.0, device="cuda"):
    """[max_pos, rot]: cosines, then sines, of rot / 2 frequencies."""
    f = float(base) ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(max_pos, dtype=torch.float64)[:, None] * f
    return torch.cat((a.cos(), a.sin()), 1).float().to(device).contiguous()


class PagedAttention:
    """One layer.  wqkv fp32 [(n_q + 2 n_kv) * head_dim, hidden] and wo fp32
    [hidden, n_q * head_dim] on the GPU are quantized to INT4 group-128 (for
    decoding) and NVFP4 (for prompts); rope as
    qlin.qkv_norm_rope_append takes it, q_weight and k_weight fp32 [head_dim]
    or None."""

    def __init__(self, cache, wqkv, wo, n_q, rope, q_weight=None, k_weight=None, eps=1e-6,
                 interleaved=False):
        self.cache, self.n_q, self.rope, self.eps = cache, n_q, rope, eps
        self.q_weight, self.k_weight, self.interleaved = q_weight, k_weight, interleaved
        self.hidden = wqkv.shape[1]
        self.width = (n_q + 2 * cache.n_kv) * cache.head_dim
        if wqkv.shape[0] != self.width or wo.shape != (self.hidden, n_q * cache.head_dim):
            raise ValueError(f"wqkv must be [{self.width}, hidden] and wo [hidden, "
                             f"{n_q * cache.head_dim}], got {list(wqkv.shape)}, {list(wo.shape)}")
        self.weights = []
        for w in (wqkv, wo):
            n, k = w.shape
            few = qlin.repack_weights(qlin.QL_INT4_G128, n, k, *qlin.quantize_int4_g128(w))
            many = qlin.repack_weights(qlin.QL_NVFP4, n, k, *qlin.quantize_nvfp4(w))
            self.weights.append((few, many, n, k))

    def project(self, x, which, prompt=None, y=None):
        """Projection `which` (0 qkv, 1 output) of x's rows: of a prompt (NVFP4
        weights and activations, these under one tensor scale for all rows of
        the call) or of decoding (INT4 weights).  Not told: by their number."""
        few, many, n, k = self.weights[which]
        if x.shape[0] > DECODE_TOKENS if prompt is None else prompt:
            return qlin.quantize_gemm_w4a4(x, many, n, y, out_dtype=torch.bfloat16)[0]
        return qlin.gemm_w4a16(x, few, n, k, y)

    def project_step(self, x, which, step):
        """The same for a step's rows, each by its sequence's kind: one call for
        every run of sequences of one kind."""
        if step.prompt is None:
            return self.project(x, which)
        runs = []                                # [of a prompt, rows]
        for p, n in zip(step.prompt, step.nodes):
            if n and runs and runs[-1][0] == p:
                runs[-1][1] += n
            elif n:
                runs.append([p, n])
        if len(runs) < 2:
            return self.project(x, which, runs[0][0] if runs else False)
        y = torch.empty((x.shape[0], self.weights[which][2]), dtype=torch.bfloat16, device=x.device)
        at = 0
        for p, n in runs:
            self.project(x[at:at + n], which, p, y[at:at + n])
            at += n
        return y

    def forward(self, x, step):
        """x bf16 [tokens, hidden], the step's new tokens sequence after
        sequence -> the layer's output [tokens, hidden].  Their keys and values
        are in the cache afterwards."""
        qkv = self.project_step(x, 0, step)
        q = qlin.qkv_norm_rope_append(self.cache, qkv, self.n_q, step.slots, step.positions,
                                      self.rope, self.q_weight, self.k_weight, self.eps,
                                      self.interleaved)
        y = qlin.kv_attention(self.cache, q, step.cu_q, step.kv_lens, step.block_table,
                              max(step.nodes, default=0), step.max_kv, tree=step.tree)
        return self.project_step(y.flatten(1), 1, step)

    def commit(self, step, path):
        """After a tree's verification: path int32 [sequences, depth] on the
        device, accepted drafts root first, -1 past the end."""
        qlin.kv_commit(self.cache, step.cu_q, step.kv_lens, step.block_table, path)
