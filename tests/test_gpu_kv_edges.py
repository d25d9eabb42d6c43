"""The key/value cache's calls at their edges: tables shorter than a length, values
that no rotation touches, roundings, rows far apart in size, sizes at the limits."""

import numpy as np
import pytest
import torch

from oracle import kvcache as kv
from tests.gpu_common import require_gpu, say
from tests.kv_common import FMTS, Batch, device_cache, on_gpu, random_tree, rows

pytestmark = pytest.mark.gpu

FD = [(f, d) for f in FMTS for d in (64, 128, 256)]


def _dev(x, dtype):
    return torch.tensor(x, dtype=dtype, device="cuda")


@pytest.mark.parametrize("fmt,d", FD)
@pytest.mark.parametrize("n_q,n_kv,nodes", [(4, 2, 1), (4, 2, 8), (4, 1, 8), (4, 1, 30)])
def test_tables_shorter_than_a_length(fmt, d, n_q, n_kv, nodes):
    """Positions past the table's last column are not read, and the new tokens
    stay the last ones of kv_lens: 2, 16, 32 and 120 rows, whole and split."""
    q = require_gpu()
    say("short table", fmt, d, n_q, n_kv, nodes)
    for lens, cols in (([100, 93], 6), ([100, 60], 5), ([1500, 1300], 81)):
        b = Batch(FMTS[fmt], lens, [nodes] * 2, n_q, n_kv, d, 16, seed=31)
        hidden = [np.arange(max(lens)) >= 16 * cols] * 2
        whole = b.table
        for tree in (None, random_tree([nodes] * 2, 31)):
            want, bound = b.reference(tree, hidden=hidden)
            for table in (whole[:, :cols], np.where(np.arange(whole.shape[1]) < cols, whole, -1).astype(np.int32)):
                b.table = table
                got = b.run(q, tree).double().cpu().numpy()
                b.table = whole
                assert np.all(np.abs(got - want) <= bound)


@pytest.mark.parametrize("fmt,d", FD)
@pytest.mark.parametrize("rot", [0, 16, 26])
@pytest.mark.parametrize("pairs", [False, True])
def test_elements_past_the_rotation_stay_as_they_are(fmt, d, rot, pairs):
    """Without norm weights, an infinity or a NaN past `rot` reaches no other
    element and stays what it is; a rotation by 0 changes nothing before it."""
    q = require_gpu()
    say("past the rotation", fmt, d, rot, pairs)
    n_q, n_kv, tokens = 3, 2, 6
    x = rows(41, tokens, n_q + 2 * n_kv, d)
    for t, at, value in ((0, rot, np.inf), (1, d - 1, -np.inf), (2, d // 2 + 1, np.nan), (3, rot + 1, np.nan)):
        x[t, :, at] = value
    x[4, :, rot:] = -0.0
    table = np.concatenate([np.ones((1, rot // 2)), np.zeros((1, rot // 2))], 1)
    slots = torch.arange(tokens, device="cuda")
    for bf16 in (True, False):
        got, want = (q.KVCache(FMTS[fmt], 1, 16, n_kv, d) for _ in range(2))
        qkv = on_gpu(x, bf16)
        queries = q.qkv_norm_rope_append(
            got, qkv.flatten(1), n_q, slots, slots.int() if rot else None,
            _dev(table, torch.float32) if rot else None, interleaved=pairs)
        q.kv_append(want, qkv[:, n_q:n_q + n_kv], qkv[:, n_q + n_kv:], slots)
        same = [(queries.float().cpu().numpy(), x[:, :n_q])]
        same += [(a.cpu().numpy(), b.cpu().numpy()) for a, b in
                 zip(q.kv_gather(got, slots, out_dtype=torch.float32),
                     q.kv_gather(want, slots, out_dtype=torch.float32))]
        for a, b in same:
            assert np.array_equal(a, b, equal_nan=True)
            real = ~np.isnan(b)
            assert np.array_equal(np.signbit(a)[real], np.signbit(b)[real])


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("part", [False, True])
def test_bf16_keys_are_rounded_once(d, pairs, part):
    """Keys 2^-40 to either side of the middle between two bf16 values, which
    binary32 does not hold."""
    q = require_gpu()
    say("bf16 keys", d, pairs, part)
    rot = 32 if part else d
    x = np.zeros((4, 3, d), dtype=np.float32)      # one query, key and value head
    a, b = (0, 1) if pairs else (0, rot // 2)
    x[:, 1, a] = 1 + np.array([1, 1, 3, 3]) / 256  # middles of 1, 1 + 2^-7, 1 + 2^-6
    x[:, 1, b] = 2.0 ** -20 * np.array([-1, 1, -1, 1])
    table = np.concatenate([np.ones((1, rot // 2)), np.full((1, rot // 2), 2.0 ** -20)], 1)
    cache = q.KVCache(q.QL_KV_BF16, 1, 16, 1, d)
    slots = torch.arange(4, device="cuda")
    q.qkv_norm_rope_append(cache, on_gpu(x, False).flatten(1), 1, slots, slots.int(),
                           _dev(table, torch.float32), interleaved=pairs)
    k, _ = q.kv_gather(cache, slots, out_dtype=torch.float32)
    assert k[:, 0, a].tolist() == [1 + 2.0 ** -7, 1.0, 1 + 2.0 ** -6, 1 + 2.0 ** -7]


@pytest.mark.parametrize("fmt,d", FD)
@pytest.mark.parametrize("size", [1e-34, 1e-30, 1e-22, 1e20, 1e30, 1e35])
def test_keys_are_normed_whatever_their_size(fmt, d, size):
    """The mean of their squares may lie outside of binary32's range; eps = 0."""
    q = require_gpu()
    say("key size", fmt, d, size)
    n_kv, slots = 2, np.arange(5)
    x = rows(51, 5, 1 + 2 * n_kv, d, bf16=False)
    x[:, 1:1 + n_kv] *= np.float32(size)
    w = np.linspace(0.5, 1.5, d).astype(np.float32)
    c = kv.Cache(FMTS[fmt], 1, 16, n_kv, d)
    c.write("k", kv.norm_rope(x[:, 1:1 + n_kv], w, 0.0, None, None, False), slots)
    c.write("v", x[:, 1 + n_kv:], slots)
    cache = q.KVCache(FMTS[fmt], 1, 16, n_kv, d,
                      data=torch.zeros(c.bytes.size, dtype=torch.uint8, device="cuda"))
    q.qkv_norm_rope_append(cache, on_gpu(x, False).flatten(1), 1, _dev(slots, torch.int64),
                           q_weight=_dev(w, torch.float32), k_weight=_dev(w, torch.float32), eps=0.0)
    assert np.array_equal(cache.data.cpu().numpy(), c.bytes)


@pytest.mark.parametrize("fmt", list(FMTS))
def test_norms_of_zero_and_infinite_rows(fmt):
    """x / sqrt(mean(x^2) + eps): an infinity gives NaN and makes the others 0, a
    row of zeros is zero, or NaN with eps = 0; queries and keys alike."""
    q = require_gpu()
    say("norm ends", fmt)
    d = 64
    x = rows(52, 3, 3, d, bf16=False)
    x[0, :, 5] = np.inf
    x[1] = x[2] = 0
    w = _dev(np.ones(d), torch.float32)
    cache = q.KVCache(FMTS[fmt], 1, 16, 1, d)
    for eps in (1e-6, 0.0):
        y = q.qkv_norm_rope_append(cache, on_gpu(x, False).flatten(1), 1, torch.arange(3, device="cuda"),
                                   q_weight=w, k_weight=w, eps=eps)
        k, _ = q.kv_gather(cache, torch.arange(3, device="cuda"), out_dtype=torch.float32)
        for got in (y[:, 0].float(), k[:, 0]):
            bad = torch.isnan(got[0]).nonzero().flatten().tolist()
            assert bad == (list(range(16)) if fmt == "nvfp4" and got.data_ptr() == k.data_ptr() else [5])
            assert not got[0].nan_to_num().any()
            assert torch.isnan(got[1:]).all() if eps == 0 else not got[1:].any()


@pytest.mark.parametrize("fmt,d", FD)
@pytest.mark.parametrize("nodes", [1, 20, 70])
@pytest.mark.parametrize("far", ["anywhere", "by tile", "by part"])
def test_value_rows_up_to_the_formats_ends(fmt, d, nodes, far):
    """V rows 2^190 apart, in any order, in tiles of one wave or in parts of their
    own: the small rows' weights stay in the sum of weights."""
    q = require_gpu()
    say("rows far apart", fmt, d, nodes, far)
    lens = [nodes + 40, nodes + 1500]

    def size(which, b, n):
        if which == "k":
            return np.ones(n)
        at = np.arange(n)
        big = {"anywhere": np.random.default_rng([6, b]).random(n) < 0.5,
               "by tile": at // 32 % 2 == 0, "by part": at < n // 2}[far]
        return 2.0 ** np.where(big, 95.0, -95.0)
    b = Batch(FMTS[fmt], lens, [nodes] * 2, 4, 2, d, 32, seed=61, scale_rows=size)
    b.check(b.run(q))


@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("nodes", [1, 20])
def test_a_large_row_of_little_weight(fmt, nodes):
    """The largest V row has 2^-90 of the weight: the others give the result."""
    q = require_gpu()
    say("large row of little weight", fmt, nodes)
    lens = [nodes + 90]
    b = Batch(FMTS[fmt], lens, [nodes], 2, 1, 64, 16, seed=62,
              scale_rows=lambda which, s, n: 2.0 ** np.where((np.arange(n) == 40) & (which == "v"), 60.0, -60.0)
              if which == "v" else np.ones(n))
    # one query direction: the large row's key lies against it
    b.q[:] = np.float32(0.5)
    k = rows(63, lens[0], 1, 64) * np.float32(0.05)
    k[40] = -2.0
    b.c.write("k", k, b.slots(0, np.arange(lens[0])))
    b.check(b.run(q, scale=1.0), scale=1.0)


@pytest.mark.parametrize("fmt,d", FD)
@pytest.mark.parametrize("nodes", [1, 20, 70])
def test_zero_rows_beside_small_ones(fmt, d, nodes):
    """A first key whose value is zero takes nearly all of the weight; the others'
    values are small.  What is left keeps its bits."""
    q = require_gpu()
    say("zero rows", fmt, d, nodes)
    lens = [nodes + 200]
    b = Batch(FMTS[fmt], lens, [nodes], 4, 2, d, 16, seed=71,
              scale_rows=lambda which, s, n: np.where(np.arange(n) == 0, 0.0, 2.0 ** -20)
              if which == "v" else np.ones(n))
    b.q[:] = np.abs(b.q)
    k = rows(72, lens[0], 2, d) * np.float32(2.0 ** -3)
    k[0] = 0.75
    at = b.slots(0, np.arange(lens[0]))
    b.c.write("k", k, at)
    cache, v = device_cache(q, b.c), np.zeros((1, 2, d), dtype=np.float32)
    q.kv_append(cache, on_gpu(k[:1], False), on_gpu(v, False), _dev(at[:1], torch.int64))
    y = q.kv_attention(cache, on_gpu(b.q), torch.from_numpy(b.cu).cuda(), _dev(lens, torch.int32),
                       torch.from_numpy(b.table).cuda(), nodes, lens[0])
    b.check(y)


@pytest.mark.parametrize("fmt", ["e4m3", "nvfp4"])
def test_a_row_of_zeros_takes_the_smallest_exponent(fmt):
    q = require_gpu()
    say("zero row bytes", fmt)
    c = kv.Cache(FMTS[fmt], 1, 16, 1, 64)
    x = np.zeros((2, 1, 64), dtype=np.float32)
    x[1, 0, ::2] = -0.0
    for which in "kv":
        c.write(which, x, [0, 1])
    assert c.exp["v"][0, 0] == kv.E_MIN and c.exp["k"][1, 0] == kv.E_MIN
    cache = q.KVCache(FMTS[fmt], 1, 16, 1, 64,
                      data=torch.zeros(c.bytes.size, dtype=torch.uint8, device="cuda"))
    q.kv_append(cache, on_gpu(x, False), on_gpu(x, False), _dev([0, 1], torch.int64))
    assert np.array_equal(cache.data.cpu().numpy(), c.bytes)


@pytest.mark.parametrize("fmt,d", [("nvfp4", 128), ("nvfp4", 256), ("e4m3", 128), ("bf16", 64)])
def test_prompt_chunks_that_fill_the_chip(fmt, d):
    """Chunks of prompts in blocks of 64 rows (4-bit 128-wide keys take 32 where
    the blocks of 64 would not fill a round), the last one not full, with and
    without context; a few of the sequences against the definition."""
    q = require_gpu()
    n_q, n_kv, seqs = 32, 4, 24
    nodes = [70 - (5 * i) % 13 for i in range(seqs)]
    lens = [n + (0, 33, 130, 7)[i % 4] for i, n in enumerate(nodes)]
    say("full chip", fmt, d)
    row_blocks = -(-max(nodes) * (n_q // n_kv) // 64)
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    assert max(nodes) > 64 and seqs * n_kv * row_blocks > 3 * cus
    b = Batch(FMTS[fmt], lens, nodes, n_q, n_kv, d, 32, seed=81)
    got = b.run(q).double().cpu().numpy()
    assert np.all(np.isfinite(got))
    for s in (0, 2, 13, 23):
        t = slice(b.cu[s], b.cu[s + 1])
        one = Batch.__new__(Batch)
        one.__dict__.update(b.__dict__, lens=[lens[s]], nodes=[nodes[s]], table=b.table[s:s + 1],
                            q=b.q[t], cu=np.array([0, nodes[s]], dtype=np.int32))
        want, bound = one.reference()
        assert np.all(np.abs(got[t] - want) <= bound)


def test_a_caches_buffer_is_fixed():
    """The calls take the buffer that the cache was made with: another one cannot
    be put in its place unnoticed."""
    q = require_gpu()
    say("cache buffer")
    cache = q.KVCache(q.QL_KV_E4M3, 2, 16, 2, 64)
    with pytest.raises(AttributeError):
        cache.data = torch.zeros_like(cache.data)
    for name in ("fmt", "n_pages", "page_size", "n_kv", "head_dim", "device"):
        with pytest.raises(AttributeError):
            setattr(cache, name, getattr(cache, name))


@pytest.mark.parametrize("n_q,d", [(1, 64), (33, 64), (33, 256)])
def test_the_longest_length(n_q, d):
    """2^31 - 16 positions, of which only the first and the last page are there."""
    q = require_gpu()
    say("longest", n_q, d)
    cols = (2 ** 31 - 1) // 16
    cache = q.KVCache(q.QL_KV_E4M3, 2, 16, 1, d)
    k, v = on_gpu(rows(91, 32, 1, d)), on_gpu(rows(92, 32, 1, d))
    q.kv_append(cache, k, v, torch.arange(32, device="cuda"))
    k, v = (t[:, 0].double() for t in q.kv_gather(cache, torch.arange(32, device="cuda"), out_dtype=torch.float32))
    table = torch.full((1, cols), -1, dtype=torch.int32, device="cuda")
    table[0, 0], table[0, -1] = 0, 1
    x = on_gpu(rows(93, 1, n_q, d))
    y = q.kv_attention(cache, x, _dev([0, 1], torch.int32), _dev([16 * cols], torch.int32), table, 1, 2 ** 30)
    want = torch.softmax(x[0].double() @ k.T * d ** -0.5, 1) @ v
    assert torch.allclose(y[0].double(), want, rtol=2.0 ** -7, atol=2.0 ** -7)


def test_tokens_past_a_grids_rows():
    """More tokens than one launch's grid holds: their last rows are written, normed
    and read back like the first."""
    q = require_gpu()
    say("many tokens")
    d, tokens = 64, (1 << 26) + 70
    cache = q.KVCache(q.QL_KV_E4M3, 8, 16, 1, d)
    slots = torch.full((tokens,), -1, dtype=torch.int64, device="cuda")
    some = torch.tensor([0, 5, (1 << 26) - 9, (1 << 26) - 1, 1 << 26, tokens - 1], device="cuda")
    slots[some] = torch.arange(6, device="cuda") * 3
    k = torch.empty((tokens, 1, d), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    k[some], v[some] = on_gpu(rows(95, 6, 1, d)), on_gpu(rows(96, 6, 1, d))
    q.kv_append(cache, k, v, slots)
    few = q.KVCache(q.QL_KV_E4M3, 8, 16, 1, d)
    q.kv_append(few, k[some], v[some], slots[some])
    want = q.kv_gather(few, slots[some])
    got = q.kv_gather(cache, slots[some])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    q.kv_gather(cache, slots, k=k, v=v)
    assert torch.equal(k[some], want[0]) and torch.equal(v[some], want[1])
    others = torch.ones(tokens, dtype=torch.bool, device="cuda")
    others[some] = False
    assert not k[others].any() and not v[others].any()
    del k, v, others
    qkv = torch.empty((tokens, 3 * d), dtype=torch.bfloat16, device="cuda")
    qkv[some] = on_gpu(rows(97, 6, 3, d)).flatten(1)
    out = q.qkv_norm_rope_append(cache, qkv, 1, slots)
    assert torch.equal(out[some], q.qkv_norm_rope_append(few, qkv[some], 1, slots[some]))
    got, want = q.kv_gather(cache, slots[some]), q.kv_gather(few, slots[some])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("d", [64, 256])
def test_more_blocks_than_a_grids_row(d):
    """Many sequences under a max_q that is far above their token counts, as one
    long chunk among them makes it: 2^24 thread blocks and more."""
    q = require_gpu()
    say("many blocks", d)
    seqs, n_q = 515, 32
    lens = [1 + (7 * i) % 40 for i in range(seqs)]
    b = Batch(kv.E4M3, lens, [1] * seqs, n_q, 1, d, 16, seed=99)
    most = 32768 if d == 64 else 65536
    x = torch.zeros((most, n_q, d), dtype=torch.bfloat16, device="cuda")
    x[:seqs] = on_gpu(b.q)
    y = torch.zeros_like(x)
    assert -(-most * n_q // (32 if d == 64 else 64)) * seqs > 1 << 24
    q.kv_attention(device_cache(q, b.c), x, torch.from_numpy(b.cu).cuda(), _dev(lens, torch.int32),
                   torch.from_numpy(b.table).cuda(), most, max(lens), y=y)
    b.check(y[:seqs])
    assert not y[seqs:].any()


@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("keys", [2, 64])
def test_infinities_that_are_seen(fmt, keys):
    """In V: infinite or NaN, or the value of the largest code; in K: a score of
    that sign."""
    q = require_gpu()
    say("infinities", fmt, keys)
    d = 64
    cache = q.KVCache(FMTS[fmt], 4, 16, 1, d)
    k = np.zeros((keys, 1, d), dtype=np.float32)
    v = np.ones((keys, 1, d), dtype=np.float32)
    v[0, 0, 3] = np.inf
    slots = torch.arange(keys, device="cuda")
    table, cu, lens = _dev([[0, 1, 2, 3]], torch.int32), _dev([0, 1], torch.int32), _dev([keys], torch.int32)

    def run(x):
        query = torch.full((1, 1, d), float(x), dtype=torch.bfloat16, device="cuda")
        return q.kv_attention(cache, query, cu, lens, table, 1, keys)[0, 0].double().cpu().numpy()
    q.kv_append(cache, on_gpu(k), on_gpu(v), slots)
    one = q.kv_gather(cache, slots[1:2])[1][0, 0, 0].item()       # 1 in this format
    y = run(1)
    if fmt == "bf16":
        assert not np.isfinite(y[3])
        assert np.isnan(y).all() or (np.delete(y, 3) == 1).all()
    else:
        # the other rows' weights are far below 2^-31 of that row's times 2^e, so
        # of the other elements nothing but their finiteness is stated
        assert y[3] == {"e4m3": 1.75, "nvfp4": 1.3125}[fmt] * 2.0 ** 128 / keys
        assert np.isfinite(y).all()
    k[0, 0, 7] = np.inf
    v[0, 0, 3] = 5
    q.kv_append(cache, on_gpu(k), on_gpu(v), slots)
    assert np.isnan(run(1)).all()
    assert (run(-1) == one).all()
