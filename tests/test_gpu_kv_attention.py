"""kv_attention against the float64 definition on the values the cache stands
for.  The bound on each element (tests/kv_common.py) follows from the roundings
include/qlin.h states; everything in the cache that no sequence owns is filled
with bytes that read as NaN."""

import numpy as np
import pytest
import torch

from oracle import kvcache as kv
from tests.gpu_common import require_gpu, say
from tests.kv_common import FMTS, Batch, device_cache, on_gpu, random_tree

pytestmark = pytest.mark.gpu

FD = [(f, d) for f in FMTS for d in (64, 128, 256)]


@pytest.mark.parametrize("fmt,d", FD)
@pytest.mark.parametrize("n_q,n_kv,page", [(4, 1, 16), (10, 2, 32), (3, 3, 128)])
def test_single_tokens(fmt, d, n_q, n_kv, page):
    """Ordinary decoding at lengths around blocks, tiles and pages."""
    q = require_gpu()
    lens = [1, 15, 16, 17, 31, 33, 64, 97, 129, 300]
    say("decode", fmt, d, n_q, n_kv, page)
    b = Batch(FMTS[fmt], lens, [1] * len(lens), n_q, n_kv, d, page, seed=1)
    b.check(b.run(q))


@pytest.mark.parametrize("fmt,d", FD)
def test_splits_and_wrong_hints(fmt, d):
    """Lengths past 512 are split and joined; max_kv is a hint only."""
    q = require_gpu()
    lens = [2100, 5, 700, 1]
    say("splits", fmt, d)
    b = Batch(FMTS[fmt], lens, [1, 2, 1, 1], 2, 1, d, 64, seed=2)
    ys = [b.run(q, max_kv=m) for m in (2100, 513, 16, 0, 100000)]
    for y in ys:
        b.check(y)
    assert torch.equal(ys[0], b.run(q, max_kv=2100))              # bit for bit again


@pytest.mark.parametrize("fmt,d", FD)
@pytest.mark.parametrize("n_q,n_kv", [(4, 2), (5, 1), (2, 2)])
def test_trees(fmt, d, n_q, n_kv):
    q = require_gpu()
    lens, nodes = [64, 100, 7, 40, 200], [64, 31, 7, 1, 9]
    say("trees", fmt, d, n_q, n_kv)
    b = Batch(FMTS[fmt], lens, nodes, n_q, n_kv, d, 16, seed=4)
    tree = random_tree(nodes, 4)
    b.check(b.run(q, tree), tree)


@pytest.mark.parametrize("fmt", list(FMTS))
def test_trees_over_splits(fmt):
    q = require_gpu()
    lens, nodes = [1500, 900, 33], [64, 3, 33]
    say("trees over splits", fmt)
    b = Batch(FMTS[fmt], lens, nodes, 4, 1, 128, 32, seed=6)
    tree = random_tree(nodes, 6)
    b.check(b.run(q, tree), tree)


@pytest.mark.parametrize("fmt,d", FD)
def test_long_chains(fmt, d):
    """A chunk of a prompt: causal over more tokens than a row block holds, with
    and without context, and over a split."""
    q = require_gpu()
    lens, nodes = [150, 333, 20, 700], [150, 90, 20, 65]
    say("chains", fmt, d)
    b = Batch(FMTS[fmt], lens, nodes, 2, 1, d, 64, seed=7)
    b.check(b.run(q))


@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("nodes", [1, 20])
def test_rows_that_see_nothing(fmt, nodes):
    """Empty masks, sequences without keys, without queries, and pages that are
    not there, give zeros."""
    q = require_gpu()
    say("nothing seen", fmt, nodes)
    lens = [nodes, 0, 40, nodes + 30]
    b = Batch(FMTS[fmt], lens, [nodes, 0, 0, nodes], 4, 2, 64, 16, seed=8)
    tree = np.array([0] * nodes + [1 << i for i in range(nodes)], dtype=object)
    y = b.run(q, tree, max_q=nodes)
    b.check(y, tree)
    assert torch.count_nonzero(y[:nodes]) == 0
    b.table[:] = -1
    assert torch.count_nonzero(b.run(q, tree, max_q=nodes)) == 0
    b.table[:] = b.c.n_pages                                     # past the last page
    assert torch.count_nonzero(b.run(q, tree, max_q=nodes)) == 0


@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("nodes", [1, 20])
def test_absent_pages_hide_their_tokens(fmt, nodes):
    q = require_gpu()
    say("absent pages", fmt, nodes)
    lens = [200, 130]
    b = Batch(FMTS[fmt], lens, [nodes, nodes], 4, 2, 128, 16, seed=9)
    hidden = []
    for s, gone in enumerate(([0, 3, 4, 5, 9], [2, 7])):
        h = np.zeros(max(lens), dtype=bool)
        for p in gone:
            h[16 * p:16 * p + 16] = True
        hidden.append(h)
    want = b.reference(hidden=hidden)
    for s, gone in enumerate(([0, 3, 4, 5, 9], [2, 7])):
        b.table[s, gone] = -1
    got = b.run(q).double().cpu().numpy()
    assert np.all(np.abs(got - want[0]) <= want[1])


@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("nodes", [2, 24])
def test_non_finite_rows_reach_only_who_sees_them(fmt, nodes):
    """A draft with a NaN key and one with a NaN value: the queries on other
    branches are as without them, those on their own are NaN."""
    q = require_gpu()
    say("hidden NaN", fmt, nodes)
    lens = [50 + nodes]
    b = Batch(FMTS[fmt], lens, [nodes], 4, 2, 128, 16, seed=10)
    tree = np.array([1 << i for i in range(nodes)], dtype=object)   # each sees only itself
    want, bound = b.reference(tree)
    cache = device_cache(q, b.c)
    for which, node in (("k", 0), ("v", nodes - 1)):
        slot = torch.tensor([b.slots(0, 50 + node)], device="cuda")
        k, v = q.kv_gather(cache, slot, out_dtype=torch.float32)
        (k if which == "k" else v)[0, :, 5] = float("nan")
        q.kv_append(cache, k, v, slot)
    y = q.kv_attention(cache, on_gpu(b.q), torch.from_numpy(b.cu).cuda(),
                       torch.tensor(lens, dtype=torch.int32, device="cuda"),
                       torch.from_numpy(b.table).cuda(), nodes, lens[0],
                       tree=torch.tensor([int(m) for m in tree], device="cuda"))
    got = y.double().cpu().numpy()
    assert np.isnan(got[0]).all()                                   # its key's score
    assert np.isnan(got[-1, :, 5]).all()
    assert np.all(np.abs(got - want)[1:-1] <= bound[1:-1])


@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("nodes", [1, 17])
def test_rows_of_very_different_size(fmt, nodes):
    """V rows 2^40 apart and K rows far from 1: the weights keep their relative
    precision, whichever rows are large."""
    q = require_gpu()
    say("row sizes", fmt, nodes)
    lens = [90, 600]

    def size(which, b, n):
        e = np.random.default_rng([5, b]).integers(-20, 21, n)
        return 2.0 ** (e if which == "v" else np.full(n, -30.0))
    b = Batch(FMTS[fmt], lens, [nodes] * 2, 4, 2, 128, 16, seed=11, scale_rows=size)
    b.check(b.run(q, scale=2.0 ** 29), scale=2.0 ** 29)


def test_zero_rows_and_zero_queries():
    q = require_gpu()
    for fmt in FMTS:
        say("zeros", fmt)
        b = Batch(FMTS[fmt], [40], [1], 4, 2, 64, 16, seed=12,
                  scale_rows=lambda w, s, n: (np.arange(n) % 3 > 0).astype(np.float64))
        b.q[:, 1] = 0
        b.check(b.run(q))


def test_strided_queries_other_stream_and_workspace():
    q = require_gpu()
    say("strides, stream")
    lens = [700, 90]
    b = Batch(kv.NVFP4, lens, [1, 2], 6, 2, 128, 32, seed=13)
    want = b.run(q)
    cache = device_cache(q, b.c)
    wide = torch.zeros((3, 10, 128), dtype=torch.bfloat16, device="cuda")
    wide[:, :6] = on_gpu(b.q)
    table = torch.full((2, 64), -1, dtype=torch.int32, device="cuda")
    table[:, :b.table.shape[1]] = torch.from_numpy(b.table).cuda()
    cu, ln = torch.from_numpy(b.cu).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y = q.kv_attention(cache, wide[:, :6], cu, ln, table[:, :40], 2, 700, stream=s)
    need = q.kv_attention_workspace(cache, 3, 6, 2, 2, 700)
    assert need > 0
    out = torch.empty((3, 6, 128), dtype=torch.bfloat16, device="cuda")
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    q.kv_attention(cache, wide[:, :6], cu, ln, table, 2, 700, y=out, workspace=ws, stream=s)
    s.synchronize()
    assert torch.equal(y, want) and torch.equal(out, want)
    with pytest.raises(q.QlinError) as e:
        q.kv_attention(cache, wide[:, :6], cu, ln, table, 2, 700, workspace=ws[:need - 16])
    assert e.value.status == q.QL_EWORKSPACE


def test_queries_past_max_q_are_left_alone():
    q = require_gpu()
    say("max_q")
    b = Batch(kv.E4M3, [40, 30], [8, 3], 2, 1, 64, 16, seed=14)
    full = b.run(q)
    y = torch.full((11, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    b.run(q, max_q=3, y=y)
    assert torch.equal(y[:3], full[:3]) and torch.equal(y[8:], full[8:])
    assert torch.all(y[3:8] == 7.0)


def test_refusals():
    q = require_gpu()
    b = Batch(kv.BF16, [20], [2], 4, 2, 64, 16, seed=15)
    cache = device_cache(q, b.c)
    qq, cu = on_gpu(b.q), torch.from_numpy(b.cu).cuda()
    ln, tb = torch.tensor([20], dtype=torch.int32, device="cuda"), torch.from_numpy(b.table).cuda()
    for bad in (lambda: q.kv_attention(cache, qq.float(), cu, ln, tb, 2, 20),
                lambda: q.kv_attention(cache, qq[..., :32], cu, ln, tb, 2, 20),
                lambda: q.kv_attention(cache, qq, cu.long(), ln, tb, 2, 20),
                lambda: q.kv_attention(cache, qq, cu, ln[:0], tb, 2, 20),
                lambda: q.kv_attention(cache, qq, cu, ln, tb.long(), 2, 20),
                lambda: q.kv_attention(cache, qq, cu, ln, tb, 2, 20, tree=cu),
                lambda: q.kv_attention(cache, qq, cu, ln, tb, 2, 20, y=qq.float())):
        with pytest.raises(ValueError):
            bad()
    for kw, status in ((dict(max_q=-1), q.QL_EINVAL), (dict(max_kv=-1), q.QL_EINVAL)):
        with pytest.raises(q.QlinError) as e:
            q.kv_attention(cache, qq, cu, ln, tb, **{"max_q": 2, "max_kv": 20, **kw})
        assert e.value.status == status
    tree = torch.zeros(2, dtype=torch.int64, device="cuda")
    with pytest.raises(q.QlinError) as e:
        q.kv_attention(cache, qq, cu, ln, tb, 65, 20, tree=tree)
    assert e.value.status == q.QL_ESHAPE
    with pytest.raises(q.QlinError) as e:                          # 3 query heads over 2
        q.kv_attention(cache, qq[:, :3].contiguous(), cu, ln, tb, 2, 20)
    assert e.value.status == q.QL_ESHAPE
    assert q.kv_attention(cache, qq[:0], cu[:1], ln[:0], tb[:0], 0, 0).shape == (0, 4, 64)


@pytest.mark.parametrize("fmt", list(FMTS))
def test_graph_replays_match_eager(fmt):
    """A decode step (norm + append + attention + commit) captured in a HIP graph
    and replayed, with eager work through the same workspace between replays."""
    q = require_gpu()
    say("graph", fmt)
    n_q, n_kv, d = 8, 2, 128
    b = Batch(FMTS[fmt], [900, 200], [4, 4], n_q, n_kv, d, 16, seed=16)
    lens = torch.tensor([900, 200], dtype=torch.int32, device="cuda")
    cu, tb = torch.from_numpy(b.cu).cuda(), torch.from_numpy(b.table).cuda()
    slots = torch.tensor(np.concatenate([b.slots(0, np.arange(896, 900)),
                                         b.slots(1, np.arange(196, 200))]), device="cuda")
    rng = torch.Generator(device="cuda").manual_seed(1)
    inputs = [torch.randn((8, (n_q + 2 * n_kv) * d), generator=rng, device="cuda").bfloat16()
              for _ in range(4)]
    rope = torch.randn((64, d), generator=rng, device="cuda")
    w = torch.ones(d, device="cuda")
    pos = torch.arange(8, device="cuda").int()
    path = torch.tensor([[0, 2, -1], [1, 3, -1]], dtype=torch.int32, device="cuda")
    start = torch.from_numpy(b.c.bytes).cuda()
    cache = q.KVCache(FMTS[fmt], b.c.n_pages, 16, n_kv, d, data=start.clone())
    x = torch.empty_like(inputs[0])
    qo = torch.empty((8, n_q, d), dtype=torch.bfloat16, device="cuda")
    y = torch.empty_like(qo)
    ws = torch.empty(q.kv_attention_workspace(cache, 8, n_q, 2, 4, 900), dtype=torch.uint8, device="cuda")
    assert ws.numel() > 0

    def step():
        q.qkv_norm_rope_append(cache, x, n_q, slots, pos, rope, w, w, q_out=qo)
        q.kv_attention(cache, qo, cu, lens, tb, 4, 900, y=y, workspace=ws)
        q.kv_commit(cache, cu, lens, tb, path)

    def eager(t):
        cache.data.copy_(start)
        x.copy_(t)
        step()
        return y.clone(), cache.data.clone()
    want = [eager(t) for t in inputs]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in (0, 1, 2, 3, 1, 0):
        cache.data.copy_(start)
        x.copy_(inputs[i])
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i][0]) and torch.equal(cache.data, want[i][1])
        eager(inputs[(i + 1) % 4])


@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("nodes", [4, 24])
def test_bytes_of_a_hidden_row_do_not_reach_its_neighbours(fmt, nodes):
    """A draft that was never written, between drafts that are seen."""
    q = require_gpu()
    say("hidden row", fmt, nodes)
    for gone in (0, 1, 2):
        b = Batch(FMTS[fmt], [48 + nodes], [nodes], 4, 2, 64, 16, seed=17)
        for which in "kv":
            for h in range(2):
                for p in b.c.places(which, b.slots(0, 48 + gone), h):
                    b.c.bytes[p] = 0xFF
        tree = np.array([int(m) & ~(1 << gone) for m in random_tree([nodes], 17)], dtype=object)
        b.check(b.run(q, tree), tree)


@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("nodes", [1, 17])
def test_many_uneven_sequences_share_the_parts(fmt, nodes):
    """More sequences than a wave has lanes, most of them short or empty, some
    long: parts go to the long ones."""
    q = require_gpu()
    say("uneven", fmt, nodes)
    lens = [nodes + (5 * i) % 40 for i in range(70)]
    lens[0] = lens[66] = 1900
    lens[69], lens[30] = 2700, 600
    count = [nodes if i % 9 else 0 for i in range(70)]
    lens[9] = lens[18] = 0
    b = Batch(FMTS[fmt], lens, count, 2, 1, 64, 32, seed=18)
    y = b.run(q)
    b.check(y)
    assert torch.equal(y, b.run(q)) and q.kv_attention_workspace(
        device_cache(q, b.c), sum(count), 2, 70, nodes, max(lens)) > 0


@pytest.mark.parametrize("fmt,d", FD)
@pytest.mark.parametrize("n_q,n_kv,nodes", [(4, 1, 5), (8, 1, 4), (3, 1, 11), (6, 2, 14), (1, 1, 48)])
def test_rows_around_the_blocks(fmt, d, n_q, n_kv, nodes):
    """20, 32, 33, 42 and 48 rows of a kv head: blocks of 16, 32 and 64 rows, the
    last one full or not."""
    q = require_gpu()
    say("row blocks", fmt, d, n_q, n_kv, nodes)
    lens = [nodes, nodes + 31, 640]
    b = Batch(FMTS[fmt], lens, [nodes] * 3, n_q, n_kv, d, 32, seed=19)
    tree = random_tree([nodes] * 3, 19)
    b.check(b.run(q, tree), tree)
    b.check(b.run(q))


def test_sequences_that_share_pages():
    """Two sequences with a common prompt's pages."""
    q = require_gpu()
    say("shared pages")
    b = Batch(kv.E4M3, [100, 90], [1, 1], 4, 2, 128, 16, seed=20)
    b.table[1, :5] = b.table[0, :5]
    b.check(b.run(q))


@pytest.mark.parametrize("n_kv,tokens", [(1, 65), (2, 300), (8, 700)])
def test_chunks_over_four_bits(n_kv, tokens):
    """A prompt's chunk over 4-bit 128-wide keys: few blocks and many."""
    q = require_gpu()
    say("4-bit chunk", n_kv, tokens)
    b = Batch(kv.NVFP4, [tokens + 40], [tokens], 4 * n_kv if n_kv < 8 else 8, n_kv, 128, 64, seed=21)
    b.check(b.run(q))
