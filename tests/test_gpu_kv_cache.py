"""kv_append, kv_gather, qkv_norm_rope_append and kv_commit against the float64
definition: bytes and values of the cache exactly, queries within the rounding
of binary32 arithmetic and bf16."""

import numpy as np
import pytest
import torch

from oracle import kvcache as kv
from tests.gpu_common import require_gpu, say
from tests.kv_common import FMTS, Batch, device_cache, on_gpu, rows

pytestmark = pytest.mark.gpu

FD = [(f, d) for f in FMTS for d in (64, 128, 256)]


def _slots(rng, pages, page, tokens):
    return rng.permutation(pages * page)[:tokens].astype(np.int64)


def _dev(x, dtype):
    return torch.tensor(x, dtype=dtype, device="cuda")


@pytest.mark.parametrize("fmt,d", FD)
@pytest.mark.parametrize("n_kv,tokens,bf16", [(1, 1, True), (3, 37, False), (8, 70, True)])
def test_append_bytes_and_gather_values(fmt, d, n_kv, tokens, bf16):
    q = require_gpu()
    say("append", fmt, d, n_kv, tokens)
    rng = np.random.default_rng(5)
    c = kv.Cache(FMTS[fmt], 6, 16, n_kv, d, fill=0xA5)
    cache = device_cache(q, c)
    k, v = rows(1, tokens, n_kv, d, bf16), rows(2, tokens, n_kv, d, bf16)
    slots = _slots(rng, 6, 16, tokens)
    slots[tokens // 2] = -1 if tokens > 1 else slots[0]
    c.write("k", k, slots)
    c.write("v", v, slots)
    st = _dev(slots, torch.int64)
    q.kv_append(cache, on_gpu(k, bf16), on_gpu(v, bf16), st)
    torch.cuda.synchronize()
    assert np.array_equal(cache.data.cpu().numpy(), c.bytes)       # nothing else is touched
    ok = slots >= 0
    for dtype in (torch.float32, torch.bfloat16):
        gk, gv = q.kv_gather(cache, st, out_dtype=dtype)
        for got, which in ((gk, "k"), (gv, "v")):
            got = got.double().cpu().numpy()
            assert np.array_equal(got[ok], c.value[which][slots[ok]])
            assert np.all(got[~ok] == 0)


@pytest.mark.parametrize("fmt,d", FD)
@pytest.mark.parametrize("start", [0, 1, 6, 15])
def test_append_of_prompts_that_start_anywhere(fmt, d, start):
    """Consecutive slots (the quad path) from every alignment, over pages of 32,
    and from slices of a fused projection."""
    q = require_gpu()
    say("append prompt", fmt, d, start)
    n_q, n_kv, tokens = 2, 2, 45
    c = kv.Cache(FMTS[fmt], 3, 32, n_kv, d)
    qkv = rows(3, tokens, n_q + 2 * n_kv, d)
    slots = np.arange(start, start + tokens)
    slots = np.where(slots < 32, slots + 64, slots - 32)          # pages 2 and 0, 1
    c.write("k", qkv[:, n_q:n_q + n_kv], slots)
    c.write("v", qkv[:, n_q + n_kv:], slots)
    cache = q.KVCache(FMTS[fmt], 3, 32, n_kv, d,
                      data=torch.zeros(c.bytes.size, dtype=torch.uint8, device="cuda"))
    t = on_gpu(qkv)
    q.kv_append(cache, t[:, n_q:n_q + n_kv], t[:, n_q + n_kv:], _dev(slots, torch.int64))
    torch.cuda.synchronize()
    assert np.array_equal(cache.data.cpu().numpy(), c.bytes)


@pytest.mark.parametrize("fmt", ["e4m3", "nvfp4"])
def test_rows_of_extreme_values(fmt):
    """Zero rows, single elements, ties, values at the ends of the exponent's
    range, sizes 2^60 apart in one row, infinities and NaN."""
    q = require_gpu()
    say("extreme rows", fmt)
    d, top = 64, kv.TOP[FMTS[fmt]]
    x = np.zeros((12, 1, d), dtype=np.float32)
    x[1, 0, 7] = -3.0
    x[2, 0, :] = np.float32(top)                       # amax exactly Q: e = 0
    x[3, 0, 0] = np.nextafter(np.float32(top), np.float32(np.inf))
    x[4, 0, :] = np.linspace(-6, 6, d, dtype=np.float32)
    x[5, 0, :] = 2.0 ** np.arange(-60, 4, dtype=np.float32)
    x[6, 0, :] = np.float32(1e-38)                     # below the smallest exponent
    x[7, 0, :] = np.float32(3e38)
    x[8, 0, ::2] = np.float32(-0.0)
    x[9, 0, :] = np.float32(2.5) * 2.0 ** np.arange(d).astype(np.float32) % 7
    x[10, 0, 3] = np.inf
    x[10, 0, 4] = -1.0
    x[11, 0, 20] = np.nan
    x[11, 0, 40] = 5.0
    c = kv.Cache(FMTS[fmt], 1, 16, 1, d)
    finite = list(range(10))
    c.write("k", x[:10], finite)
    c.write("v", x[:10], finite)
    cache = q.KVCache(FMTS[fmt], 1, 16, 1, d,
                      data=torch.zeros(c.bytes.size, dtype=torch.uint8, device="cuda"))
    slots = _dev(np.arange(12), torch.int64)
    q.kv_append(cache, on_gpu(x, False), on_gpu(x, False), slots)
    gk, gv = (t.double().cpu().numpy() for t in q.kv_gather(cache, slots, out_dtype=torch.float32))
    for got, which in ((gk, "k"), (gv, "v")):
        assert np.array_equal(got[:10], c.value[which][:10])
        # the largest code under the exponent of 2^128, which passes binary32
        assert got[10, 0, 3] == np.inf and np.count_nonzero(got[10]) == 1
        bad = np.isnan(got[11, 0])
        rest = kv.quantize(FMTS[fmt], np.nan_to_num(x[11]))["value"]      # as if it were zero
        assert bad[20] and not bad[40] and got[11, 0, 40] == rest[0, 40]
        assert bad.sum() == (1 if fmt == "e4m3" else 16)


def _norm_case(fmt, tokens, n_q, n_kv, d, rot, pairs, norm=True, bf16=True, seed=0):
    qkv = rows(10 + seed, tokens, n_q + 2 * n_kv, d, bf16)
    rng = np.random.default_rng([80, seed])
    wq = (1 + 0.2 * rng.standard_normal(d)).astype(np.float32) if norm else None
    wk = (1 + 0.2 * rng.standard_normal(d)).astype(np.float32) if norm else None
    a = rng.standard_normal((50, rot // 2)) * 3
    table = np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)
    pos = rng.integers(0, 50, tokens).astype(np.int32)
    return qkv, wq, wk, table, pos


@pytest.mark.parametrize("fmt,d", FD)
@pytest.mark.parametrize("tokens,n_q,n_kv,rot,pairs,norm,bf16", [
    (1, 2, 1, None, False, True, True),
    (7, 6, 2, None, True, True, False),
    (13, 5, 1, 16, False, True, True),
    (6, 4, 2, 26, True, True, True),
    (9, 3, 3, 30, False, True, False),
    (5, 4, 4, None, False, False, True),
    (4, 2, 2, 0, False, True, True),
    (33, 12, 4, None, False, True, True)])
def test_norm_rope_append(fmt, d, tokens, n_q, n_kv, rot, pairs, norm, bf16):
    q = require_gpu()
    say("norm rope", fmt, d, tokens, n_q, n_kv, rot, pairs, norm)
    rot = d if rot is None else rot
    qkv, wq, wk, table, pos = _norm_case(fmt, tokens, n_q, n_kv, d, rot, pairs, norm, bf16)
    rng = np.random.default_rng(81)
    slots = _slots(rng, 4, 16, tokens)
    if tokens > 4:
        slots[3] = -7
    cache = q.KVCache(FMTS[fmt], 4, 16, n_kv, d, data=torch.zeros(
        q.kv_cache_bytes(FMTS[fmt], 4, 16, n_kv, d), dtype=torch.uint8, device="cuda"))
    t = on_gpu(qkv, bf16).flatten(1)
    wide = torch.empty((tokens, t.shape[1] + 16), dtype=t.dtype, device="cuda")
    wide[:, :t.shape[1]] = t                                      # rows with a longer stride
    got = q.qkv_norm_rope_append(
        cache, wide[:, :t.shape[1]], n_q, _dev(slots, torch.int64),
        _dev(pos, torch.int32) if rot else None, _dev(table, torch.float32) if rot else None,
        None if wq is None else _dev(wq, torch.float32),
        None if wk is None else _dev(wk, torch.float32), eps=1e-5, interleaved=pairs)
    torch.cuda.synchronize()
    want = kv.norm_rope(qkv[:, :n_q], wq, 1e-5, table, pos, pairs)
    # before rounding to bf16 (2^-9 of the result): eight binary32 roundings of
    # terms no larger than the row's largest normed value, and the sum of
    # squares' of half of d 2^-24 (plus the reciprocal root's last bits)
    normed = np.abs(kv.norm_rope(qkv[:, :n_q], wq, 1e-5, None, pos, pairs)).max(-1, keepdims=True)
    bound = 2.0 ** -8 * np.abs(want) + (8 + d / 2 + 4) * 2.0 ** -24 * 2 * normed
    assert np.all(np.abs(got.double().cpu().numpy() - want) <= bound)
    # keys: binary64 up to the roundings of the format
    c = kv.Cache(FMTS[fmt], 4, 16, n_kv, d)
    keys = kv.norm_rope(qkv[:, n_q:n_q + n_kv], wk, 1e-5, table, pos, pairs)
    c.write("k", keys, slots)
    c.write("v", qkv[:, n_q + n_kv:], slots)
    assert np.array_equal(cache.data.cpu().numpy(), c.bytes)


def test_norm_rope_positions_are_clamped():
    q = require_gpu()
    say("norm rope positions")
    qkv, wq, wk, table, _ = _norm_case("bf16", 3, 2, 1, 64, 64, False)
    cache = q.KVCache(q.QL_KV_BF16, 1, 16, 1, 64)
    slots = _dev([0, 1, 2], torch.int64)

    def run(pos):
        return q.qkv_norm_rope_append(cache, on_gpu(qkv).flatten(1), 2, slots,
                                      _dev(pos, torch.int32), _dev(table, torch.float32),
                                      _dev(wq, torch.float32), _dev(wk, torch.float32))
    assert torch.equal(run([-5, 50, 2 ** 31 - 1]), run([0, 49, 49]))


@pytest.mark.parametrize("fmt,d", FD)
def test_commit_moves_rows(fmt, d):
    q = require_gpu()
    say("commit", fmt, d)
    lens, nodes, n_kv = [40, 9, 70, 5, 3], [16, 9, 64, 2, 3], 2
    b = Batch(FMTS[fmt], lens, nodes, n_kv, n_kv, d, page=16, seed=3)
    path = np.full((5, 20), -1, dtype=np.int32)
    path[0, :5] = [0, 2, 5, 6, 15]           # sources and targets overlap
    path[1, :4] = [0, 1, 2, 3]               # nothing to move
    path[2, :20] = np.arange(1, 64, 3)[:20]  # across pages
    path[3, :3] = [1, 7, -5]                 # an index that is no node
    path[4, :3] = [2, 0, 1]                  # not ascending: all sources first
    cache = device_cache(q, b.c)
    q.kv_commit(cache, torch.from_numpy(b.cu).cuda(), _dev(lens, torch.int32),
                torch.from_numpy(b.table).cuda(), torch.from_numpy(path).cuda())
    torch.cuda.synchronize()
    for s in range(5):
        ctx = lens[s] - nodes[s]
        pairs = [(ctx + p, ctx + j) for j, p in enumerate(path[s]) if 0 <= p < nodes[s] and p != j]
        b.c.move([(b.slots(s, x), b.slots(s, y)) for x, y in pairs])
    assert np.array_equal(cache.data.cpu().numpy(), b.c.bytes)


@pytest.mark.parametrize("fmt", list(FMTS))
def test_commit_leaves_rows_of_absent_pages(fmt):
    q = require_gpu()
    say("commit absent pages", fmt)
    lens, nodes = [40, 40], [30, 30]                  # drafts at 10..39, over three pages
    b = Batch(FMTS[fmt], lens, nodes, 2, 2, 64, page=16, seed=4)
    path = np.array([[3, 8, 20, 25]] * 2, dtype=np.int32)
    gone = b.table.copy()
    gone[0, 1], gone[1, 0] = -1, b.c.n_pages          # sources 13, 18, 30, 35
    cache = device_cache(q, b.c)
    q.kv_commit(cache, torch.from_numpy(b.cu).cuda(), _dev(lens, torch.int32),
                torch.from_numpy(gone).cuda(), torch.from_numpy(path).cuda())
    torch.cuda.synchronize()
    # of the first sequence only sources on pages 0 and 2 move, of the second
    # none: all targets (10..13) lie on its page 0
    at = b.slots(0, [13, 35, 10, 13])
    b.c.move([(at[0], at[2]), (at[1], at[3])])
    assert np.array_equal(cache.data.cpu().numpy(), b.c.bytes)


def test_reads_back_what_a_reappend_keeps():
    """E4M3 rows survive reading back and appending again unchanged."""
    q = require_gpu()
    say("reappend")
    cache = q.KVCache(q.QL_KV_E4M3, 4, 16, 2, 128)
    slots = torch.arange(50, device="cuda")
    q.kv_append(cache, on_gpu(rows(1, 50, 2, 128)), on_gpu(rows(2, 50, 2, 128)), slots)
    k, v = q.kv_gather(cache, slots, out_dtype=torch.float32)
    q.kv_append(cache, k, v, slots)
    k2, v2 = q.kv_gather(cache, slots, out_dtype=torch.float32)
    assert torch.equal(k, k2) and torch.equal(v, v2)


def test_offsets_past_32_bits():
    """Slots whose bytes lie past 4 GiB, and block indices in the last page."""
    q = require_gpu()
    say("large cache")
    pages, page, d = 1100, 4096, 256
    cache = q.KVCache(q.QL_KV_BF16, pages, page, 1, d)            # 4.6 GB
    slots = _dev([pages * page - 1, pages * page - 2, 17, 4_400_000], torch.int64)
    k, v = on_gpu(rows(1, 4, 1, d)), on_gpu(rows(2, 4, 1, d))
    q.kv_append(cache, k, v, slots)
    gk, gv = q.kv_gather(cache, slots)
    assert torch.equal(gk, k) and torch.equal(gv, v)
    # one sequence whose four tokens' pages are the last ones
    table = _dev([[pages - 1]], torch.int32)
    tail = torch.arange(4, device="cuda") + (pages - 1) * page
    q.kv_append(cache, k, v, tail)
    cu, lens = _dev([0, 1], torch.int32), _dev([4], torch.int32)
    y = q.kv_attention(cache, k[:1], cu, lens, table, 1, 4)
    s = (k[:, 0].double() @ k[0, 0].double()) * d ** -0.5
    want = torch.softmax(s, 0) @ v[:, 0].double()
    assert torch.allclose(y[0, 0].double(), want, rtol=2.0 ** -7, atol=2.0 ** -7)


def test_refusals():
    q = require_gpu()
    cache = q.KVCache(q.QL_KV_E4M3, 2, 16, 2, 64)
    k = torch.zeros((3, 2, 64), dtype=torch.bfloat16, device="cuda")
    slots = torch.arange(3, device="cuda")
    for bad in (lambda: q.KVCache(3, 2, 16, 2, 64), lambda: q.KVCache(1, 2, 24, 2, 64),
                lambda: q.KVCache(1, 2, 16, 2, 96), lambda: q.KVCache(1, 0, 16, 2, 64),
                lambda: q.KVCache(1, 2, 16, 2, 64, data=torch.zeros(64, dtype=torch.uint8, device="cuda")),
                lambda: q.kv_append(cache, k[:, :1], k, slots),
                lambda: q.kv_append(cache, k.half(), k.half(), slots),
                lambda: q.kv_append(cache, k.float(), k, slots),
                lambda: q.kv_append(cache, k, k, slots.int()),
                lambda: q.kv_append(cache, k, k, slots[:2]),
                lambda: q.kv_append(cache, k.cpu(), k, slots),
                lambda: q.kv_append(cache, k.transpose(0, 1).contiguous().transpose(0, 1), k, slots),
                lambda: q.kv_gather(cache, slots, k=k[:2]),
                lambda: q.kv_gather(cache, slots, out_dtype=torch.float16),
                lambda: q.qkv_norm_rope_append(cache, k.flatten(1), 2, slots),
                lambda: q.qkv_norm_rope_append(cache, torch.zeros((3, 384), device="cuda"), 2, slots,
                                               rope=torch.zeros((4, 64), device="cuda")),
                lambda: q.kv_commit(cache, slots, slots.int(), slots.int()[None], slots.int()[None])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(q.QlinError):                              # rot odd: refused by the library
        q.qkv_norm_rope_append(cache, torch.zeros((3, 384), device="cuda"), 2, slots, slots.int(),
                               torch.zeros((4, 33), device="cuda"))
    wide = torch.zeros((3, 2 * 64 + 1), dtype=torch.bfloat16, device="cuda")
    odd = wide[:, :128].unflatten(1, (2, 64))                     # rows not on 16 bytes
    with pytest.raises(q.QlinError) as e:
        q.kv_append(cache, odd, odd, slots)
    assert e.value.status == q.QL_EALIGN
