"""The experts' products and the layer that runs them, against the oracle in
float64 on exactly dequantized operands."""

import numpy as np
import pytest
import torch

from oracle import nvfp4, rows
from decode_nvfp4_rtn_amd import synth
from tests.gpu_common import require_gpu, say, dev_bf16, host_f64
from tests.rows_common import (Stack, bf16_rows, check, choices, half_step, operand, product, product_bound,
                               silu_bound)

pytestmark = pytest.mark.gpu


def run(fmt, tokens, experts, top_k, n, k, gather, silu, dtype, idle=0.0, only=None, spare=0, seed=0):
    q = require_gpu()
    ids = choices(seed + tokens, tokens, experts, top_k, idle, only)
    order, where, offsets = rows.plan(ids, experts)
    stack = Stack(q, fmt, seed + n, experts, n, k, spare)
    bits, _ = bf16_rows(seed + k, tokens if gather else tokens * top_k, k)
    x, values = operand(q, fmt, bits)
    say(fmt, tokens, experts, top_k, n, k, gather, silu, dtype)
    plan = q.group_rows(torch.from_numpy(ids).cuda(), experts)
    y = torch.full((tokens * top_k, n // 2 if silu else n), float("nan"), dtype=dtype, device="cuda")
    product(q, fmt, *x, stack.blobs, plan, n, k, gather=gather, silu_mul=silu, y=y)
    ref = rows.experts_product(values, stack.values, order, offsets, top_k, gather)
    if silu:
        check(y, *silu_bound(ref[:, :n // 2], ref[:, n // 2:], dtype))
    else:
        check(y, ref, product_bound(ref, dtype))
    assert not host_f64(y)[offsets[-1]:].any()
    again = product(q, fmt, *x, stack.blobs, plan, n, k, gather=gather, silu_mul=silu, out_dtype=dtype)
    assert torch.equal(y, again)


BF, F32 = torch.bfloat16, torch.float32
# tokens, experts, top_k, n, k, gather, silu, type, more
CASES = [(1, 1, 1, 32, 128, True, False, F32, {}),
         (1, 8, 2, 64, 256, True, True, BF, {}),
         (5, 3, 1, 48, 128, False, False, BF, {}),                  # an odd number of weight tiles
         (17, 4, 2, 96, 384, True, True, F32, {}),
         (16, 1, 1, 272, 640, True, False, BF, {}),
         (33, 2, 2, 544, 256, False, True, BF, {}),                 # tiles past 256 weight rows
         (64, 16, 4, 128, 896, True, False, F32, dict(idle=0.3)),
         (64, 70, 4, 128, 128, False, True, BF, dict(idle=0.3)),    # most experts meet nothing
         (40, 6, 2, 64, 256, True, False, BF, dict(only=[2, 3])),   # runs between empty experts
         (40, 6, 1, 64, 256, True, True, BF, dict(only=[5])),
         (20, 5, 2, 64, 256, True, False, F32, dict(idle=1.0)),     # no expert at all
         (257, 2, 1, 288, 384, True, False, BF, dict(only=[1])),    # one place past a tile
         (600, 3, 2, 320, 256, False, True, F32, {}),
         (300, 1000, 3, 32, 128, True, False, BF, {}),
         (130, 2, 1, 64, 1408, True, True, BF, dict(spare=48)),     # blobs with room between them
         (3, 2, 1, 32, 8192, True, False, F32, {}),                 # x in pieces
         (100, 2, 2, 64, 4224, True, True, BF, {}),
         (12, 2, 1, 32, 8192, False, False, BF, {}),
         (3, 2, 1, 32, 20480, True, False, BF, {}),
         (1, 8, 2, 64, 1024, True, True, BF, {}),                   # k shared by 2, 4, 8 waves
         (1, 8, 3, 64, 2048, True, False, F32, {}),
         (4, 9, 3, 96, 4096, True, True, BF, {}),
         (2, 5, 2, 48, 4096, True, False, BF, {}),
         (1200, 3, 1, 4096, 128, True, False, BF, {}),              # tiles in halves, and whole
         (1200, 3, 1, 4096, 128, True, True, F32, {}),
         (1300, 3, 1, 8192, 128, False, False, BF, dict(idle=0.2))]


@pytest.mark.parametrize("fmt", ["int4", "nvfp4"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:5])))
def test_product(fmt, case):
    run(fmt, *case[:8], **case[8])


@pytest.mark.parametrize("fmt", ["int4", "nvfp4"])
@pytest.mark.parametrize("rows_each", [1, 4, 15, 16, 17, 31, 32, 33, 48, 49, 63, 64, 65, 127, 129, 191, 192, 193, 255,
                                       256, 257])
def test_run_lengths(fmt, rows_each):
    """Two experts' runs of each length around the tiles' borders."""
    run(fmt, rows_each, 3, 2, 64, 256, True, rows_each % 2 == 0, BF, only=[0, 2])


@pytest.mark.parametrize("fmt", ["int4", "nvfp4"])
@pytest.mark.parametrize("tokens", [3, 50])
def test_an_expert_chosen_twice(fmt, tokens):
    """All choices of every token are one expert: its run holds every row top_k times."""
    q = require_gpu()
    ids = np.full((tokens, 8), 2, dtype=np.int32)
    order, where, offsets = rows.plan(ids, 4)
    stack = Stack(q, fmt, 5, 4, 64, 1024)
    x, values = operand(q, fmt, bf16_rows(tokens, tokens, 1024)[0])
    say("chosen twice", fmt, tokens)
    plan = q.group_rows(torch.from_numpy(ids).cuda(), 4)
    y = product(q, fmt, *x, stack.blobs, plan, 64, 1024)
    ref = rows.experts_product(values, stack.values, order, offsets, 8, True)
    check(y, ref, product_bound(ref, BF))


@pytest.mark.parametrize("fmt", ["int4", "nvfp4"])
def test_a_foreign_blob_leaves_its_rows(fmt):
    q = require_gpu()
    ids = np.array([[0], [1], [2], [1]], dtype=np.int32)
    stack = Stack(q, fmt, 5, 3, 64, 256)
    other = Stack(q, "nvfp4" if fmt == "int4" else "int4", 5, 1, 64, 256)
    size = min(other.blobs.shape[1], stack.blobs.shape[1])
    stack.blobs[1, :size] = other.blobs[0, :size]
    bits, _ = bf16_rows(4, 4, 256)
    x, _ = operand(q, fmt, bits)
    say("foreign blob", fmt)
    plan = q.group_rows(torch.from_numpy(ids).cuda(), 3)
    y = torch.full((4, 64), 7.0, device="cuda")
    product(q, fmt, *x, stack.blobs, plan, 64, 256, y=y)
    assert (y[1:3] == 7).all() and not (y[0] == 7).any() and not (y[3] == 7).any()


@pytest.mark.parametrize("fmt", ["int4", "nvfp4"])
def test_no_tokens(fmt):
    q = require_gpu()
    stack = Stack(q, fmt, 5, 3, 64, 256)
    plan = q.group_rows(torch.zeros((0, 2), dtype=torch.int32, device="cuda"), 3)
    x, _ = operand(q, fmt, bf16_rows(4, 4, 256)[0])
    x = tuple(t[:0] if t.dim() == 2 else t for t in x)
    assert product(q, fmt, *x, stack.blobs, plan, 64, 256).shape == (0, 64)


@pytest.mark.parametrize("fmt", ["int4", "nvfp4"])
def test_offsets_out_of_range_are_held(fmt):
    """Contents that no plan has: the calls stay in their buffers."""
    q = require_gpu()
    stack = Stack(q, fmt, 6, 4, 64, 256)
    x, _ = operand(q, fmt, bf16_rows(4, 30, 256)[0])
    plan = q.group_rows(torch.from_numpy(choices(1, 30, 4, 2)).cuda(), 4)
    good = product(q, fmt, *x, stack.blobs, plan, 64, 256)
    say("bad plan", fmt)
    order, offsets = plan.order.clone(), plan.offsets.clone()
    room = torch.zeros((64 + 60 + 64, 64), dtype=BF, device="cuda")
    for bad in ([0, 10, 5, 70, 60], [-9, 2 ** 31 - 1, 0, -2 ** 31, 7], [100] * 5, [0, 60, 0, 60, 0]):
        plan.offsets.copy_(torch.tensor(bad))
        plan.order.copy_(order.flip(0) * 1000003 - 77)
        product(q, fmt, *x, stack.blobs, plan, 64, 256, y=room[64:124])
        assert not room[:64].any() and not room[124:].any()
    plan.order.copy_(order)
    plan.offsets.copy_(offsets)
    assert torch.equal(product(q, fmt, *x, stack.blobs, plan, 64, 256), good)


def test_rows_past_31_bits():
    """y of more than 2^31 elements: the last rows are right."""
    q = require_gpu()
    n, k, tokens = 2048, 128, 1100000
    stack = Stack(q, "int4", 8, 2, n, k)
    bits, values = bf16_rows(3, 1000, k)
    x = dev_bf16(bits).repeat(tokens // 1000, 1)
    ids = torch.zeros(tokens, dtype=torch.int32, device="cuda")
    ids[-500:] = 1
    say("past 31 bits")
    plan = q.group_rows(ids, 2)
    y = q.moe_gemm_w4a16(x, stack.blobs, plan, n, k)
    assert y.numel() > 2 ** 31
    for first, e in ((0, 0), (tokens - 1000, 0), (tokens - 300, 1)):
        at = np.arange(first, first + 200)
        ref = values.astype(np.float64)[at % 1000] @ stack.values[e].T
        check(y[first:first + 200], ref, product_bound(ref, BF), first)
    out = q.moe_combine(y, plan, torch.full((tokens, 1), 0.5, device="cuda"))
    assert torch.equal(out[-1000:].float(), y[-1000:].float() * 0.5)


def weights_of(seed, experts, inter, hidden):
    rng = np.random.default_rng([96, seed])
    up = (rng.standard_normal((experts, 2 * inter, hidden)) * hidden ** -0.5).astype(np.float32)
    down = (rng.standard_normal((experts, hidden, inter)) * inter ** -0.5).astype(np.float32)
    return up, down


@pytest.mark.parametrize("tokens,prompt", [(1, None), (5, None), (40, False), (40, None), (5, True), (300, True)])
def test_layer_step_by_step(tokens, prompt):
    """RoutedExperts against the oracle, each call on the one before's outputs."""
    q = require_gpu()
    from decode_nvfp4_rtn_amd.experts import RoutedExperts
    from oracle import int4
    experts, inter, hidden, top_k = 6, 128, 256, 3
    up, down = weights_of(tokens, experts, inter, hidden)
    layer = RoutedExperts(torch.from_numpy(up).cuda(), torch.from_numpy(down).cuda(), top_k)
    bits, values = bf16_rows(tokens, tokens, hidden)
    logits = np.random.default_rng(tokens).standard_normal((tokens, experts)).astype(np.float32)
    logits[tokens // 2] = -np.inf
    say("layer", tokens, prompt)
    x, l = dev_bf16(bits), torch.from_numpy(logits).cuda()
    out = layer.forward(x, l, prompt)
    ids, weights, plan = q.moe_route(l, top_k)
    many = tokens > 32 if prompt is None else prompt
    fmt = "nvfp4" if many else "int4"
    quantize = nvfp4.quantize if many else int4.quantize
    h = layer.product(x, 0, plan, many)
    y = layer.product(h, 1, plan, many)
    assert torch.equal(out, q.moe_combine(y, plan, weights))
    want, w = rows.route(logits, top_k, True)
    order, where, offsets = rows.plan(want, experts)
    assert np.array_equal(ids.cpu().numpy(), want)
    for got, given, ws, gather in ((h, values, up, True), (y, host_f64(h).astype(np.float32), down, False)):
        v = nvfp4.dequantize(*nvfp4.quantize(given)) if many else given.astype(np.float64)
        ref = rows.experts_product(v, [rows.weights_of(fmt, quantize(e)) for e in ws], order, offsets, top_k, gather)
        if gather:
            check(got, *silu_bound(ref[:, :inter], ref[:, inter:], BF))
        else:
            check(got, ref, product_bound(ref, BF))
    yv = host_f64(y)
    ref = rows.combine(yv, where.reshape(want.shape), offsets, w)
    slack = (top_k + 80) * 2.0 ** -24 * rows.combine(np.abs(yv), where.reshape(want.shape), offsets, w)
    check(out, ref, slack + half_step(np.abs(ref) + slack, BF))
    assert not out[tokens // 2].any()


@pytest.mark.parametrize("prompt", [None, False, True])
def test_layer_of_no_tokens(prompt):
    require_gpu()
    from decode_nvfp4_rtn_amd.experts import RoutedExperts
    up, down = weights_of(1, 4, 128, 256)
    layer = RoutedExperts(torch.from_numpy(up).cuda(), torch.from_numpy(down).cuda(), 2)
    say("layer of no tokens", prompt)
    out = layer.forward(torch.zeros((0, 256), dtype=BF, device="cuda"), torch.zeros((0, 4), device="cuda"), prompt)
    assert out.shape == (0, 256)


def test_graph_replays_on_other_choices():
    """One captured layer, replayed with other tokens and other experts'
    sizes; eager work through the same memory between the replays."""
    q = require_gpu()
    from decode_nvfp4_rtn_amd.experts import RoutedExperts
    experts, inter, hidden, top_k, tokens = 12, 128, 256, 3, 200
    up, down = weights_of(1, experts, inter, hidden)
    layer = RoutedExperts(torch.from_numpy(up).cuda(), torch.from_numpy(down).cuda(), top_k)
    say("graph")
    for prompt in (False, True):
        x = torch.zeros((tokens, hidden), dtype=BF, device="cuda")
        logits = torch.zeros((tokens, experts), device="cuda")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            layer.forward(x, logits, prompt)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = layer.forward(x, logits, prompt)
        for i in range(5):
            g = torch.Generator(device="cuda").manual_seed(i)
            x.copy_(torch.randn((tokens, hidden), generator=g, device="cuda"))
            logits.copy_(torch.randn((tokens, experts), generator=g, device="cuda") * (1 + 3 * i))
            if i == 3:
                logits[:, 2:] = float("-inf")
            want = layer.forward(x.clone(), logits.clone(), prompt)
            out.fill_(9)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want), (prompt, i)


def test_on_another_stream():
    """A chain of calls on a stream of its own, while another runs on the current one."""
    q = require_gpu()
    stack = Stack(q, "int4", 9, 8, 128, 256)
    bits, _ = bf16_rows(4, 50, 256)
    x, w = dev_bf16(bits), torch.ones((50, 2), device="cuda")
    say("stream")

    def chain(ids, stream=None):
        plan = q.group_rows(ids, 8, stream=stream)
        y = q.moe_gemm_w4a16(x, stack.blobs, plan, 128, 256, stream=stream)
        return y, q.moe_combine(y, plan, w, stream=stream)
    two = [torch.from_numpy(choices(i, 50, 8, 2)).cuda() for i in (5, 6)]
    want = [chain(ids) for ids in two]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = chain(two[0], s), chain(two[1])
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_refusals():
    q = require_gpu()
    stack = Stack(q, "int4", 9, 4, 64, 256)
    four = Stack(q, "nvfp4", 9, 4, 64, 256)
    plan = q.group_rows(torch.zeros((6, 2), dtype=torch.int32, device="cuda"), 4)
    x = torch.zeros((6, 256), dtype=BF, device="cuda")
    c, s, t = q.quantize_nvfp4(x)
    say("refusals")
    for call in (lambda: q.moe_gemm_w4a16(x, stack.blobs, plan, 64, 256, gather=False),
                 lambda: q.moe_gemm_w4a16(x.float(), stack.blobs, plan, 64, 256),
                 lambda: q.moe_gemm_w4a16(x.t().contiguous().t(), stack.blobs, plan, 64, 256),
                 lambda: q.moe_gemm_w4a16(x, stack.blobs[:3], plan, 64, 256),
                 lambda: q.moe_gemm_w4a16(x, stack.blobs[:, :-256], plan, 64, 256),
                 lambda: q.moe_gemm_w4a16(x, stack.blobs.cpu(), plan, 64, 256),
                 lambda: q.moe_gemm_w4a16(x, stack.blobs, plan, 64, 128),
                 lambda: q.moe_gemm_w4a16(x, stack.blobs, plan, 64.0, 256),
                 lambda: q.moe_gemm_w4a16(x, stack.blobs, plan, 64, 256, out_dtype=torch.float16),
                 lambda: q.moe_gemm_w4a16(x, stack.blobs, plan, 64, 256, y=torch.zeros((12, 32), device="cuda")),
                 lambda: q.moe_gemm_w4a4(c[:5], s, t, four.blobs, plan, 64, 256),
                 lambda: q.moe_gemm_w4a4(c, s[:, :8], t, four.blobs, plan, 64, 256),
                 lambda: q.moe_gemm_w4a4(c, s, t.cpu(), four.blobs, plan, 64, 256),
                 lambda: q.moe_gemm_w4a4(c, s, t, stack.blobs, plan, 64, 256)):
        with pytest.raises(ValueError):
            call()
    wide = torch.zeros((4, stack.blobs.shape[1] + 8), dtype=torch.uint8, device="cuda")
    with pytest.raises(q.QlinError):      # blobs 8 bytes off
        q.moe_gemm_w4a16(x, wide[:, :stack.blobs.shape[1]], plan, 64, 256)
