"""Plans, a router's choice and the sum over a token's experts against the
oracle: whole numbers equal, weights and sums within bounds of their roundings."""

import numpy as np
import pytest
import torch

from oracle import rows
from tests.gpu_common import require_gpu, say, dev_bf16, host_f64
from tests.rows_common import bf16_rows, choices, half_step
from decode_nvfp4_rtn_amd import synth

pytestmark = pytest.mark.gpu


def same_plan(plan, ids, groups):
    order, where, offsets = rows.plan(ids, groups)
    assert np.array_equal(plan.order.cpu().numpy(), order)
    assert np.array_equal(plan.where.cpu().numpy().ravel(), where)
    assert np.array_equal(plan.offsets.cpu().numpy(), offsets)


@pytest.mark.parametrize("count,groups", [(0, 3), (1, 1), (2, 1024), (63, 5), (64, 5), (511, 64), (1024, 63), (1025, 65),
                                          (4097, 1), (20000, 1000), (140001, 7), (300000, 1024)])
def test_group_rows(count, groups):
    q = require_gpu()
    rng = np.random.default_rng([94, count])
    ids = rng.integers(-2, groups + 2, count).astype(np.int32)
    if count:
        ids[rng.integers(0, count)] = np.iinfo(np.int32).min
        ids[rng.integers(0, count)] = np.iinfo(np.int32).max
    say("group rows", count, groups)
    same_plan(q.group_rows(torch.from_numpy(ids).cuda(), groups), ids, groups)


@pytest.mark.parametrize("value", [0, 5, -1])
def test_one_group_takes_all(value):
    q = require_gpu()
    ids = np.full(5000, value, dtype=np.int32)
    say("one group", value)
    same_plan(q.group_rows(torch.from_numpy(ids).cuda(), 6), ids, 6)


def test_group_rows_of_pairs_and_into_a_plan():
    q = require_gpu()
    ids = choices(1, 700, 60, 6, idle=0.2)
    say("pairs")
    plan = q.group_rows(torch.from_numpy(ids).cuda(), 60)
    same_plan(plan, ids, 60)
    assert plan.where.shape == (700, 6) and plan.top_k == 6 and plan.tokens == 700
    other = choices(2, 700, 60, 6)
    assert q.group_rows(torch.from_numpy(other).cuda(), 60, plan=plan) is plan
    same_plan(plan, other, 60)


def logits_of(seed, tokens, experts, bf16, masked):
    rng = np.random.default_rng([95, seed])
    x = (2 * rng.standard_normal((tokens, experts))).astype(np.float32)
    if masked:
        x[rng.random(x.shape) < 0.3] = -np.inf
        x[rng.random(x.shape) < 0.02] = np.nan
        x[rng.random(x.shape) < 0.01] = np.inf
        x[rng.random(tokens) < 0.2] = -np.inf
    if bf16:      # few values: ties
        x = np.round(x * 4) / 4
    t = torch.from_numpy(x).cuda()
    return (t.to(torch.bfloat16) if bf16 else t), x


ROUTES = [(1, 1, 1), (1, 8, 8), (3, 60, 4), (64, 128, 8), (65, 128, 8), (33, 64, 7), (700, 256, 6), (300, 1000, 64),
          (50, 1024, 1), (5000, 130, 2), (40000, 65, 4), (7, 512, 32)]


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("bf16,masked", [(False, False), (False, True), (True, False), (True, True)])
@pytest.mark.parametrize("tokens,experts,top_k", ROUTES)
def test_route(tokens, experts, top_k, bf16, masked, renormalize):
    q = require_gpu()
    t, x = logits_of(tokens + experts, tokens, experts, bf16, masked)
    say("route", tokens, experts, top_k, bf16, masked, renormalize)
    ids, weights, plan = q.moe_route(t, top_k, renormalize=renormalize)
    want, w = rows.route(x, top_k, renormalize)
    assert np.array_equal(ids.cpu().numpy(), want)
    same_plan(plan, want, experts)
    # an exponent is off by half a step of l - max (at most 20 here), the
    # exponential by 2 steps, the sum by its 22 additions, the quotient by one
    tol = 2.0 ** -24 * (2 * 20 + 4 + 22 + 2)
    assert np.all(np.abs(weights.cpu().numpy() - w) <= tol * w + 2.0 ** -149)


def test_route_ties_zeros_and_masks():
    q = require_gpu()
    inf, nan = np.inf, np.nan
    x = np.array([[1.0, 1.0, 1.0, 1.0], [-inf, 2.0, -inf, nan], [-inf, -inf, nan, -inf], [inf, 0.0, inf, 1.0],
                  [0.0, -0.0, -1.0, 0.0], [3.4e38, -3.4e38, 3.4e38, 1e-45], [-1e-45, 1e-45, 0.0, -0.0]],
                 dtype=np.float32)
    say("ties")
    ids, weights, plan = q.moe_route(torch.from_numpy(x).cuda(), 3, renormalize=False)
    want, w = rows.route(x, 3, False)
    assert np.array_equal(ids.cpu().numpy(), want)
    assert np.allclose(weights.cpu().numpy(), w, rtol=1e-6, atol=1e-38)
    same_plan(plan, want, 4)


def test_route_strided_logits_and_no_tokens():
    q = require_gpu()
    t, x = logits_of(9, 200, 96, False, False)
    say("strided")
    wide = torch.full((200, 130), 9.0, device="cuda")
    wide[:, 7:103] = t
    ids, weights, plan = q.moe_route(wide[:, 7:103], 5)
    assert np.array_equal(ids.cpu().numpy(), rows.route(x, 5, True)[0])
    ids, weights, plan = q.moe_route(t[:0], 5)
    assert ids.shape == (0, 5) and not plan.offsets.any()


@pytest.mark.parametrize("bf16_in", [True, False])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tokens,experts,top_k,n", [(1, 4, 1, 8), (5, 9, 2, 24), (48, 32, 8, 2048), (3, 20, 13, 4104),
                                                    (300, 8, 3, 264)])
def test_combine(tokens, experts, top_k, n, bf16_in, out_dtype):
    q = require_gpu()
    ids = choices(tokens, tokens, experts, top_k, idle=0.2)
    bits, values = bf16_rows(tokens, tokens * top_k, n)
    if not bf16_in:
        values = (values * np.float32(1.0009765)).astype(np.float32)
    w = np.random.default_rng(tokens).random((tokens, top_k)).astype(np.float32)
    say("combine", tokens, experts, top_k, n, bf16_in, out_dtype)
    plan = q.group_rows(torch.from_numpy(ids).cuda(), experts)
    _, where, offsets = rows.plan(ids, experts)
    x = dev_bf16(bits) if bf16_in else torch.from_numpy(values).cuda()
    x[int(offsets[-1]):] = float("nan")       # rows of no expert are not read
    out = q.moe_combine(x, plan, torch.from_numpy(w).cuda(), out_dtype=out_dtype)
    v = values.astype(np.float64)
    want = rows.combine(v, where.reshape(ids.shape), offsets, w.astype(np.float64))
    size = rows.combine(np.abs(v), where.reshape(ids.shape), offsets, w.astype(np.float64))
    slack = top_k * 2.0 ** -24 * size          # each fused step rounds once
    assert np.all(np.abs(host_f64(out) - want) <= slack + half_step(np.abs(want) + slack, out_dtype))


def test_plan_arrays_out_of_range_are_held():
    """Contents that no plan has: the calls stay in their buffers."""
    q = require_gpu()
    ids = choices(3, 40, 6, 2)
    plan = q.group_rows(torch.from_numpy(ids).cuda(), 6)
    say("bad plan")
    plan.where.fill_(2 ** 31 - 1)
    w = torch.ones((40, 2), device="cuda")
    x = torch.ones((80, 64), dtype=torch.bfloat16, device="cuda")
    assert not q.moe_combine(x, plan, w).any()
    plan.where.fill_(-5)
    assert not q.moe_combine(x, plan, w).any()


def test_refusals():
    q = require_gpu()
    t = torch.zeros((4, 8), device="cuda")
    plan = q.moe_route(t, 2)[2]
    other = q.moe_route(t, 3)[2]
    say("refusals")
    for call in (lambda: q.moe_route(t, 9), lambda: q.moe_route(t, 0), lambda: q.moe_route(t, 2.0),
                 lambda: q.moe_route(t, True), lambda: q.moe_route(t.cpu(), 2), lambda: q.moe_route(t.half(), 2),
                 lambda: q.moe_route(t[0], 2), lambda: q.moe_route(t.t(), 2), lambda: q.moe_route(t, 2, plan=other),
                 lambda: q.moe_route(t, 2, ids=torch.zeros((4, 2), dtype=torch.int64, device="cuda")),
                 lambda: q.moe_route(t, 2, weights=torch.zeros((4, 3), device="cuda")),
                 lambda: q.group_rows(torch.zeros(4, device="cuda"), 3),
                 lambda: q.group_rows(torch.zeros(4, dtype=torch.int32), 3),
                 lambda: q.group_rows(torch.zeros(4, dtype=torch.int32, device="cuda"), 0),
                 lambda: q.group_rows(torch.zeros(4, dtype=torch.int32, device="cuda"), 1025),
                 lambda: q.group_rows(torch.zeros((4, 65), dtype=torch.int32, device="cuda"), 3),
                 lambda: q.group_rows(torch.zeros((8, 2), dtype=torch.int32, device="cuda")[::2, 0], 3),
                 lambda: q.moe_combine(torch.zeros((7, 8), device="cuda"), plan, torch.zeros((4, 2), device="cuda")),
                 lambda: q.moe_combine(torch.zeros((8, 8), device="cuda"), plan, torch.zeros((4, 3), device="cuda")),
                 lambda: q.moe_combine(torch.zeros((8, 8), device="cuda").half(), plan,
                                       torch.zeros((4, 2), device="cuda")),
                 lambda: q.moe_combine(torch.zeros((8, 8), device="cuda"), plan, torch.zeros((4, 2), device="cuda"),
                                       out=torch.zeros((4, 9), device="cuda"))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(q.QlinError):       # 12 columns
        q.moe_combine(torch.zeros((8, 12), device="cuda"), plan, torch.zeros((4, 2), device="cuda"))
    with pytest.raises(q.QlinError):       # a workspace that is too small
        q.group_rows(torch.zeros(2000, dtype=torch.int32, device="cuda"), 3,
                     workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
