"""Low-rank adapters against the oracle, and beside the projections of a layer."""

import numpy as np
import pytest
import torch

from oracle import rows
from decode_nvfp4_rtn_amd import synth
from tests.gpu_common import require_gpu, say, dev_bf16, host_f64
from tests.rows_common import bf16_rows, half_step

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def adapters_of(seed, count, rank, n, k):
    rng = np.random.default_rng([97, seed])
    a = synth.bf16_bits_as_f32(synth.to_bf16_bits((rng.standard_normal((count * rank, k)) * k ** -0.5)
                                                  .astype(np.float32))).reshape(count, rank, k)
    b = synth.bf16_bits_as_f32(synth.to_bf16_bits((rng.standard_normal((count * n, rank)) * rank ** -0.5)
                                                  .astype(np.float32))).reshape(count, n, rank)
    return a, b, (2 * rng.random(count)).astype(np.float32)


def on(v, dtype=BF):
    return torch.from_numpy(np.ascontiguousarray(v)).cuda().to(dtype)


def bound_of(y, x, a, b, scale, ids, dtype):
    """(reference, bound).  A x: k binary32 steps of at most 2^-23 each, at
    least 16 bits kept of the result (24 beside binary32 rows); B u: a step for
    each of the rank and of up to three terms; the last sum rounds by 2^-24 of
    its terms; then the output's rounding."""
    rank, k = a.shape[1:]
    want, mid, far = rows.lora(y, x.astype(np.float64), a.astype(np.float64), b.astype(np.float64),
                               scale.astype(np.float64), ids)
    kept = 2.0 ** -16 if dtype == BF else 2.0 ** -23
    slack = k * 2.0 ** -23 * far + (kept + (3 * rank + 2) * 2.0 ** -23) * mid + 2.0 ** -23 * np.abs(want)
    slack[(np.asarray(ids) < 0) | (np.asarray(ids) >= a.shape[0])] = 0
    return want, slack + half_step(np.abs(want) + slack, dtype)


CASES = [(1, 1, 8, 16, 128, BF), (1, 3, 16, 48, 256, F32), (7, 2, 24, 144, 128, BF), (16, 4, 32, 256, 640, F32),
         (50, 40, 16, 512, 1024, BF), (64, 2, 40, 528, 384, F32), (200, 3, 64, 320, 256, BF),
         (200, 2, 128, 160, 384, BF), (33, 2, 128, 96, 256, F32), (130, 1, 104, 64, 128, F32),
         (1000, 3, 16, 64, 128, BF), (300, 1000, 8, 32, 128, F32), (20, 2, 72, 16, 5120, BF)]


@pytest.mark.parametrize("tokens,count,rank,n,k,dtype", CASES)
def test_lora(tokens, count, rank, n, k, dtype):
    q = require_gpu()
    rng = np.random.default_rng([98, tokens, count])
    ids = rng.integers(-1, count, tokens).astype(np.int32)
    bits, x = bf16_rows(tokens, tokens, k)
    y = synth.bf16_bits_as_f32(synth.to_bf16_bits(rng.standard_normal((tokens, n)).astype(np.float32)))
    a, b, scale = adapters_of(tokens, count, rank, n, k)
    say("lora", tokens, count, rank, n, k, dtype)
    plan = q.group_rows(torch.from_numpy(ids).cuda(), count)
    args = (on(a), on(b), plan)
    yt = on(y, dtype)
    out = torch.full((tokens, n), float("nan"), dtype=dtype, device="cuda")
    assert q.lora_add(yt, dev_bf16(bits), *args, scale=on(scale, F32), out=out) is out
    want, bound = bound_of(y, x, a, b, scale, ids, dtype)
    far = np.abs(host_f64(out) - want)
    assert np.all(far <= bound), float((far / bound).max())
    assert torch.equal(yt, on(y, dtype))
    bare = torch.from_numpy(ids < 0).cuda()
    assert torch.equal(out[bare], yt[bare])
    # in place, and without scales
    assert q.lora_add(yt, dev_bf16(bits), *args, scale=on(scale, F32)) is yt
    assert torch.equal(yt, out)
    one = q.lora_add(on(y, dtype), dev_bf16(bits), *args)
    want, bound = bound_of(y, x, a, b, np.ones(count, np.float32), ids, dtype)
    assert np.all(np.abs(host_f64(one) - want) <= bound)


@pytest.mark.parametrize("rows_each", [15, 16, 17, 47, 48, 49, 63, 64, 65, 129])
@pytest.mark.parametrize("rank", [16, 128])
def test_run_lengths(rows_each, rank):
    q = require_gpu()
    ids = np.repeat([1, 0, -1], rows_each).astype(np.int32)
    n, k = 144, 256
    bits, x = bf16_rows(rows_each, ids.size, k)
    y = synth.bf16_bits_as_f32(bf16_rows(rows_each + 1, ids.size, n)[0])
    a, b, scale = adapters_of(rows_each, 2, rank, n, k)
    say("lora runs", rows_each, rank)
    plan = q.group_rows(torch.from_numpy(ids).cuda(), 2)
    out = q.lora_add(on(y), dev_bf16(bits), on(a), on(b), plan, scale=on(scale, F32))
    want, bound = bound_of(y, x, a, b, scale, ids, BF)
    assert np.all(np.abs(host_f64(out) - want) <= bound)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_slices_of_a_fused_projection(dtype):
    """Adapters of the middle third of a projection, x a slice too; what lies
    around them stays."""
    q = require_gpu()
    ids = np.array([0, 1, -1, 1, 0, 2, 2, 9], dtype=np.int32)
    n, k = 48, 128
    bits, x = bf16_rows(1, 8, k)
    y = synth.bf16_bits_as_f32(bf16_rows(2, 8, n)[0])
    a, b, scale = adapters_of(1, 3, 16, n, k)
    wide = torch.full((8, 3 * n), 5.0, dtype=dtype, device="cuda")
    wide[:, n:2 * n] = on(y, dtype)
    xw = torch.full((8, k + 64), float("nan"), dtype=BF, device="cuda")
    xw[:, 64:] = dev_bf16(bits)
    say("slices", dtype)
    plan = q.group_rows(torch.from_numpy(ids).cuda(), 3)
    q.lora_add(wide[:, n:2 * n], xw[:, 64:], on(a), on(b), plan, scale=on(scale, F32))
    want, bound = bound_of(y, x, a, b, scale, ids, dtype)
    assert np.all(np.abs(host_f64(wide[:, n:2 * n]) - want) <= bound)
    assert (wide[:, :n] == 5).all() and (wide[:, 2 * n:] == 5).all()


def test_a_row_meets_its_own_adapter_alone():
    """NaN in an adapter, or in a row, stays with the rows of that adapter, or
    with that row."""
    q = require_gpu()
    ids = np.array([0, 1, 2, -1, 1, 0], dtype=np.int32)
    n, k = 64, 256
    bits, x = bf16_rows(3, 6, k)
    y = bf16_rows(4, 6, n)[1]
    a, b, scale = adapters_of(2, 3, 16, n, k)
    say("own adapter")
    plan = q.group_rows(torch.from_numpy(ids).cuda(), 3)
    good = q.lora_add(on(y), dev_bf16(bits), on(a), on(b), plan, scale=on(scale, F32))
    at, xt = on(a), dev_bf16(bits)
    at[1] = float("nan")
    xt[5] = float("inf")
    out = q.lora_add(on(y), xt, at, on(b), plan, scale=on(scale, F32))
    assert out[1].isnan().all() and out[4].isnan().all() and not out[5].isfinite().any()
    for t in (0, 2, 3):
        assert torch.equal(out[t], good[t])


def test_all_bare_and_no_rows():
    q = require_gpu()
    a, b, _ = (on(v) for v in adapters_of(2, 3, 16, 64, 256))
    y = torch.randn((70, 64), device="cuda")
    x = torch.full((70, 256), float("nan"), dtype=BF, device="cuda")
    say("bare")
    plan = q.group_rows(torch.full((70,), -1, dtype=torch.int32, device="cuda"), 3)
    out = torch.empty_like(y)
    assert torch.equal(q.lora_add(y, x, a, b, plan, out=out), y)
    before = y.clone()
    q.lora_add(y, x, a, b, plan)
    assert torch.equal(y, before)
    none = q.group_rows(torch.zeros(0, dtype=torch.int32, device="cuda"), 3)
    assert q.lora_add(y[:0], x[:0], a, b, none).shape == (0, 64)


def test_plan_out_of_range_is_held():
    q = require_gpu()
    a, b, _ = (on(v) for v in adapters_of(2, 3, 16, 64, 256))
    x = torch.zeros((30, 256), dtype=BF, device="cuda")
    room = torch.zeros((64 + 30 + 64, 64), device="cuda")
    plan = q.group_rows(torch.zeros(30, dtype=torch.int32, device="cuda"), 3)
    say("bad plan")
    for bad in ([0, 40, 5, 30], [-9, 2 ** 31 - 1, 0, -2 ** 31], [0, 30, 0, 30]):
        plan.offsets.copy_(torch.tensor(bad))
        plan.order.copy_(torch.arange(30) * 71000003 - 77)
        q.lora_add(torch.ones((30, 64), device="cuda"), x, a, b, plan, out=room[64:94])
        assert not room[:64].any() and not room[94:].any()


def test_past_31_bits():
    """y, x and out of more than 2^31 elements."""
    q = require_gpu()
    n, k, tokens = 2048, 128, 1100000
    a, b, scale = adapters_of(5, 2, 16, n, k)
    bits, x = bf16_rows(6, 1000, k)
    ids = np.zeros(tokens, dtype=np.int32)
    ids[-500:] = 1
    ids[::7] = -1
    say("past 31 bits")
    y = torch.full((tokens, n), 0.25, dtype=BF, device="cuda")
    plan = q.group_rows(torch.from_numpy(ids).cuda(), 2)
    q.lora_add(y, dev_bf16(bits).repeat(tokens // 1000, 1), on(a), on(b), plan, scale=on(scale, F32))
    for first in (0, tokens - 1000, tokens - 200):
        at = np.arange(first, first + 200)
        want, bound = bound_of(np.full((200, n), 0.25), x[at % 1000], a, b, scale, ids[at], BF)
        assert np.all(np.abs(host_f64(y[first:first + 200]) - want) <= bound), first


def test_graph_replays_with_other_adapters():
    q = require_gpu()
    count, rank, n, k, tokens = 5, 16, 256, 512, 90
    a, b, scale = adapters_of(7, count, rank, n, k)
    at, bt, st = on(a), on(b), on(scale, F32)
    ids = torch.zeros(tokens, dtype=torch.int32, device="cuda")
    x = torch.zeros((tokens, k), dtype=BF, device="cuda")
    y = torch.zeros((tokens, n), dtype=BF, device="cuda")
    say("graph")

    def go(ids, x, y):
        return q.lora_add(y, x, at, bt, q.group_rows(ids, count), scale=st, out=torch.empty_like(y))
    go(ids, x, y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = go(ids, x, y)
    for i in range(5):
        g = torch.Generator(device="cuda").manual_seed(i)
        ids.copy_(torch.randint(-1, count, (tokens,), generator=g, device="cuda"))
        x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        y.copy_(torch.randn(y.shape, generator=g, device="cuda"))
        want = go(ids.clone(), x.clone(), y.clone())
        out.fill_(9)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), i


def test_beside_a_layers_projections():
    """PagedAttention with adapters: the plain layer's calls with lora_add
    between them, and the plain layer where no row has an adapter."""
    q = require_gpu()
    from decode_nvfp4_rtn_amd.attention import PagedAttention, PagedSequences, rope_table
    n_q, n_kv, d, hidden, count, rank = 4, 2, 64, 256, 3, 16
    g = torch.Generator(device="cuda").manual_seed(3)

    def rand(*shape):
        return torch.randn(shape, generator=g, device="cuda")
    width = (n_q + 2 * n_kv) * d
    wqkv, wo = rand(width, hidden) / 16, rand(hidden, n_q * d) / 16
    pairs = [((rand(count, rank, kk) / 16).to(BF), (rand(count, nn, rank) / 4).to(BF), rand(count).abs())
             for nn, kk in ((width, hidden), (hidden, n_q * d))]
    say("layer")

    def layer():
        return PagedAttention(q.KVCache(q.QL_KV_BF16, 8, 16, n_kv, d), wqkv, wo, n_q, rope_table(64, d))
    outs = []
    for adapted in (False, True, None):
        lay, seqs = layer(), PagedSequences(8, 16)
        if adapted is not False:
            lay.set_adapters(qkv=pairs[0], out=pairs[1])
        ids = torch.tensor([0] * 20 + [2] * 7, dtype=torch.int32, device="cuda")
        if adapted is None:
            ids.fill_(-1)
        s = [seqs.add(), seqs.add()]
        step = seqs.step(s, [20, 7])
        gx = torch.Generator(device="cuda").manual_seed(4)
        x = torch.randn((27, hidden), generator=gx, device="cuda").to(BF)
        plan = q.group_rows(ids, count) if adapted is not False else None
        outs.append(lay.forward(x, step, plan))
        if adapted:     # the same by hand
            by, qkv = layer(), None
            qkv = q.lora_add(by.project_step(x, 0, step), x, *pairs[0][:2], plan, scale=pairs[0][2])
            qq = q.qkv_norm_rope_append(by.cache, qkv, n_q, step.slots, step.positions, by.rope)
            y = q.kv_attention(by.cache, qq, step.cu_q, step.kv_lens, step.block_table, 20, step.max_kv).flatten(1)
            assert torch.equal(outs[-1], q.lora_add(by.project_step(y, 1, step), y, *pairs[1][:2], plan,
                                                    scale=pairs[1][2]))
    assert torch.equal(outs[0], outs[2]) and not torch.equal(outs[0], outs[1])
    with pytest.raises(ValueError):
        layer().set_adapters(qkv=pairs[1])


def test_refusals():
    q = require_gpu()
    a, b, scale = (on(v, t) for v, t in zip(adapters_of(2, 3, 16, 64, 256), (BF, BF, F32)))
    y, x = torch.zeros((6, 64), device="cuda"), torch.zeros((6, 256), dtype=BF, device="cuda")
    plan = q.group_rows(torch.zeros(6, dtype=torch.int32, device="cuda"), 3)
    pairs = q.group_rows(torch.zeros((6, 2), dtype=torch.int32, device="cuda"), 3)
    say("refusals")
    for call in (lambda: q.lora_add(y[:5], x, a, b, plan), lambda: q.lora_add(y, x.float(), a, b, plan),
                 lambda: q.lora_add(y.half(), x, a, b, plan), lambda: q.lora_add(y, x, a[:2], b, plan),
                 lambda: q.lora_add(y, x, a, b[:, :48], plan), lambda: q.lora_add(y, x, a.float(), b, plan),
                 lambda: q.lora_add(y, x[:, :128], a, b, plan), lambda: q.lora_add(y, x, a, b, pairs),
                 lambda: q.lora_add(y, x, a, b, plan, scale=scale[:2]),
                 lambda: q.lora_add(y, x, a, b, plan, scale=scale.cpu()),
                 lambda: q.lora_add(y, x, a, b, plan, out=torch.zeros((6, 48), device="cuda")),
                 lambda: q.lora_add(y, x, a, b, plan, out=y.to(BF)),
                 lambda: q.lora_add(y, x, a, b, plan, workspace=torch.zeros(64, dtype=torch.uint8)),
                 lambda: q.lora_add(torch.zeros((64, 6), device="cuda").t(), x, a, b, plan)):
        with pytest.raises(ValueError):
            call()
    many = q.group_rows(torch.zeros(200, dtype=torch.int32, device="cuda"), 3)
    assert q.lora_add_workspace(200, 3, 16, 256) > 16
    for call in (lambda: q.lora_add(torch.zeros((200, 64), device="cuda"), x[:1].repeat(200, 1), a, b, many,
                                    workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
                 lambda: q.lora_add(y, x, a[:, :12].contiguous(), b[:, :, :12].contiguous(), plan),
                 lambda: q.lora_add(torch.zeros((6, 66), device="cuda")[:, :64], x, a, b, plan)):
        with pytest.raises(q.QlinError):
            call()


def test_x_and_y_of_one_buffer():
    """Slices side by side; an output that would be x is refused, since blocks
    read rows of x that others have written."""
    q = require_gpu()
    for rows in (5, 300):
        ids = np.arange(rows, dtype=np.int32) % 4 - 1
        n, k = 128, 128
        bits, x = bf16_rows(1, rows, k)
        y = synth.bf16_bits_as_f32(bf16_rows(2, rows, n)[0])
        a, b, scale = adapters_of(1, 3, 16, n, k)
        both = torch.cat((dev_bf16(bits), on(y)), 1)
        say("one buffer", rows)
        plan = q.group_rows(torch.from_numpy(ids).cuda(), 3)
        q.lora_add(both[:, k:], both[:, :k], on(a), on(b), plan, scale=on(scale, F32))
        want, bound = bound_of(y, x, a, b, scale, ids, BF)
        assert np.all(np.abs(host_f64(both[:, k:]) - want) <= bound)
        assert torch.equal(both[:, :k], dev_bf16(bits))
        for out, z in ((both[:, :n], both[:, :k]), (both[:, 64:64 + n], both[:, :k])):
            with pytest.raises(q.QlinError):
                q.lora_add(out, z, on(a), on(b), plan)
