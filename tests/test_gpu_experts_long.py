"""moe_gemm_w4a4 above 256 rows of an expert on average (tiles of 256 places), and
the accuracy of moe_gemm_w4a16's binary32 results."""

import functools

import numpy as np
import pytest
import torch

from decode_nvfp4_rtn_amd import synth
from oracle import nvfp4, rows
from tests.gpu_common import require_gpu, say, dev_bf16, host_f64
from tests.rows_common import Stack, bf16_rows, check, choices, operand, product_bound, silu_bound
from tests.test_gpu_experts import weights_of

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def product_of(values, weights, order, offsets, top_k, gather):
    """rows.experts_product, a run at a time."""
    out = np.zeros((order.size, weights[0].shape[0]))
    for e, w in enumerate(weights):
        at = slice(offsets[e], offsets[e + 1])
        out[at] = values[order[at] // top_k if gather else np.arange(order.size)[at]] @ w.T
    return out


# What is left of each of four experts' runs after whole tiles of 256 places, rows
# without an expert, k.  With 16 tiles along the weights and 256 CUs: one round of
# tiles; a rest cut into four; a rest cut in two; a rest that is left whole.
WIDE = 4064      # the last tile is not full
RUNS = [([3 * 256 + 64, 3 * 256 + 129, 3 * 256 + 193, 2 * 256 + 1], 70, 1152),
        ([3 * 256 + 1, 4 * 256 + 65, 4 * 256 + 128, 4 * 256 + 255], 0, 1408),
        ([4 * 256 + 1, 4 * 256 + 64, 4 * 256 + 192, 4 * 256 + 255], 300, 1280),
        ([5 * 256 + 65, 6 * 256 + 128, 6 * 256 + 193, 5 * 256], 5, 1024)]


@functools.lru_cache(maxsize=1)
def long_case(i):
    lengths, idle, k = RUNS[i]
    q = require_gpu()
    ids = np.random.default_rng(i).permutation(np.repeat(np.arange(5), [*lengths, idle])).astype(np.int32)
    ids[ids == 4] = -1
    stack = Stack(q, "nvfp4", 40 + i, 4, WIDE, k)
    x, values = operand(q, "nvfp4", bf16_rows(i, ids.size, k)[0])
    order, where, offsets = rows.plan(ids, 4)
    ref = product_of(values, stack.values, order, offsets, 1, True)
    stack.values = None
    return ids[:, None], stack, x, offsets, ref


@pytest.mark.parametrize("i,silu,dtype", [(i, silu, dtype) for i in range(len(RUNS)) for silu in (True, False)
                                          for dtype in (BF, F32)])
def test_long_runs(i, silu, dtype):
    q = require_gpu()
    ids, stack, x, offsets, ref = long_case(i)
    assert ids.size > 256 * 4
    say("long runs", RUNS[i], silu, dtype)
    plan = q.group_rows(torch.from_numpy(ids).cuda(), 4)
    h = WIDE // 2
    y = torch.full((ids.size, h if silu else WIDE), float("nan"), dtype=dtype, device="cuda")
    q.moe_gemm_w4a4(*x, stack.blobs, plan, WIDE, RUNS[i][2], silu_mul=silu, y=y)
    if silu:
        check(y, *silu_bound(ref[:, :h], ref[:, h:], dtype))
    else:
        check(y, ref, product_bound(ref, dtype))
    assert not y[int(offsets[-1]):].any()
    assert torch.equal(y, q.moe_gemm_w4a4(*x, stack.blobs, plan, WIDE, RUNS[i][2], silu_mul=silu, out_dtype=dtype))


@pytest.mark.parametrize("tokens", [257, 700])
def test_long_prompt_through_the_layer(tokens):
    """RoutedExperts with more than 256 rows of an expert, each call on the one
    before's outputs."""
    q = require_gpu()
    from decode_nvfp4_rtn_amd.experts import RoutedExperts
    experts, inter, hidden, top_k = 2, 1280, 1152, 2
    up, down = weights_of(tokens, experts, inter, hidden)
    layer = RoutedExperts(torch.from_numpy(up).cuda(), torch.from_numpy(down).cuda(), top_k)
    bits, values = bf16_rows(tokens, tokens, hidden)
    logits = np.random.default_rng(tokens).standard_normal((tokens, experts)).astype(np.float32)
    logits[::9] = -np.inf
    logits[1::9, 0] = -np.inf
    say("long layer", tokens)
    x, l = dev_bf16(bits), torch.from_numpy(logits).cuda()
    out = layer.forward(x, l, True)
    ids, weights, plan = q.moe_route(l, top_k)
    h = layer.product(x, 0, plan, True)
    y = layer.product(h, 1, plan, True)
    assert torch.equal(out, q.moe_combine(y, plan, weights))
    want = rows.route(logits, top_k, True)[0]
    order, where, offsets = rows.plan(want, experts)
    assert tokens * top_k > 256 * experts and np.array_equal(ids.cpu().numpy(), want)
    for got, given, ws, gather in ((h, values, up, True), (y, host_f64(h).astype(np.float32), down, False)):
        v = nvfp4.dequantize(*nvfp4.quantize(given))
        ref = product_of(v, [rows.weights_of("nvfp4", nvfp4.quantize(e)) for e in ws], order, offsets, top_k, gather)
        if gather:
            check(got, *silu_bound(ref[:, :inter], ref[:, inter:], BF))
        else:
            check(got, ref, product_bound(ref, BF))
    assert not out[::9].any()


def test_offsets_out_of_range_are_held():
    """Contents that no plan has, with tiles of 256 places: the calls stay in their buffers."""
    q = require_gpu()
    tokens = 550
    stack = Stack(q, "nvfp4", 6, 4, 64, 256)
    x, _ = operand(q, "nvfp4", bf16_rows(4, tokens, 256)[0])
    plan = q.group_rows(torch.from_numpy(choices(1, tokens, 4, 2)).cuda(), 4)
    pairs = 2 * tokens
    good = q.moe_gemm_w4a4(*x, stack.blobs, plan, 64, 256)
    say("bad plan, long")
    order, offsets = plan.order.clone(), plan.offsets.clone()
    room = torch.zeros((300 + pairs + 300, 64), dtype=BF, device="cuda")
    for bad in ([0, 10, 5, pairs + 9, pairs], [-9, 2 ** 31 - 1, 0, -2 ** 31, 7], [5000] * 5, [0, pairs, 0, pairs, 0]):
        plan.offsets.copy_(torch.tensor(bad))
        plan.order.copy_(order.flip(0) * 1000003 - 77)
        q.moe_gemm_w4a4(*x, stack.blobs, plan, 64, 256, y=room[300:300 + pairs])
        assert not room[:300].any() and not room[300 + pairs:].any()
    plan.order.copy_(order)
    plan.offsets.copy_(offsets)
    assert torch.equal(q.moe_gemm_w4a4(*x, stack.blobs, plan, 64, 256), good)


def whole_rows(seed, count, k):
    """bf16 rows of whole numbers, in every group of 128: 64 of 2048 .. 4096 in
    steps of 32 and 64 of 1 .. 3, so that a group's sum times 31 is below 2^23.
    Then each product of a group with the operands 16 + u, u in 0 .. 15, their sums
    in any order and those less 24 times the sum of the row are whole numbers below
    2^24, which binary32 holds exactly.  128 + u would pass 2^25 and round."""
    rng = np.random.default_rng([91, seed])
    x = np.empty((count, k // 128, 128))
    x[..., :64] = 32 * rng.integers(64, 128, (count, k // 128, 64))
    x[..., 64:] = rng.integers(1, 4, (count, k // 128, 64))
    assert x.sum(2).max() * 31 < 2 ** 23 and x.sum(2).min() * 128 > 2 ** 24
    x = rng.permuted(x, axis=2).reshape(count, k)
    bits = synth.to_bf16_bits(x.astype(np.float32))
    assert np.array_equal(synth.bf16_bits_as_f32(bits), x)
    return bits, x


@pytest.mark.parametrize("k", [128, 1024])
@pytest.mark.parametrize("tokens", [1, 5, 20, 160])
def test_w4a16_sums_within_a_group_are_exact(tokens, k):
    """binary32 results round once for each group (its sum times the group's scale,
    added up), and where waves share k once more for each of at most 8 of them."""
    q = require_gpu()
    experts, top_k, n = 4, 2, 96
    stack = Stack(q, "int4", tokens + k, experts, n, k)
    bits, x = whole_rows(tokens, tokens, k)
    order, where, offsets = rows.plan(choices(tokens, tokens, experts, top_k), experts)
    say("exact sums", tokens, k)
    plan = q.group_rows(torch.from_numpy(choices(tokens, tokens, experts, top_k)).cuda(), experts)
    y = q.moe_gemm_w4a16(dev_bf16(bits), stack.blobs, plan, n, k, out_dtype=F32)
    groups = k // 128
    ref, size = np.zeros((order.size, n)), np.zeros((order.size, n))
    for g in range(groups):
        at = slice(128 * g, 128 * g + 128)
        part = product_of(x[:, at], [w[:, at] for w in stack.values], order, offsets, top_k, True)
        ref += part
        size += np.abs(part)
    steps = 1 if groups == 1 else groups + 8
    check(y, ref, steps * 2.0 ** -24 * size)


def test_as_many_tiles_as_a_launch_has():
    """2^21 tiles of 256 x 256, an output of 128 GiB: its first, middle and last rows."""
    q = require_gpu()
    n, k, pairs, base = 32768, 128, 1 << 22, 1024
    if torch.cuda.mem_get_info()[0] < 140 << 30:
        pytest.skip("needs 140 GiB of GPU memory")
    stack = Stack(q, "nvfp4", 12, 2, n, k)
    (codes, scales, ts), values = operand(q, "nvfp4", bf16_rows(5, base, k)[0])
    ids = torch.zeros(pairs, dtype=torch.int32, device="cuda")
    ids[-500:] = 1
    say("128 GiB")
    plan = q.group_rows(ids, 2)
    y = q.moe_gemm_w4a4(codes.repeat(pairs // base, 1), scales.repeat(pairs // base, 1), ts, stack.blobs, plan, n, k,
                        silu_mul=True)
    assert y.numel() == 1 << 36
    for first, e in ((0, 0), (pairs // 2 + 77, 0), (pairs - 700, 0), (pairs - 100, 1)):
        at = np.arange(first, first + 100)
        ref = values[at % base] @ stack.values[e].T
        check(y[first:first + 100], *silu_bound(ref[:, :n // 2], ref[:, n // 2:], BF), first)
    del y
    torch.cuda.empty_cache()
