"""Plans and adapters at sizes that take the kernels' other ways: more choices to a
block than it holds, and ranks of 24 and 32 over long runs."""

import numpy as np
import pytest
import torch

from decode_nvfp4_rtn_amd import synth
from oracle import rows
from tests.gpu_common import require_gpu, say, dev_bf16, host_f64
from tests.rows_common import bf16_rows
from tests.test_gpu_lora import adapters_of, bound_of, on
from tests.test_gpu_rows_plan import logits_of, same_plan

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("bf16,masked,renormalize", [(False, False, True), (True, True, False)])
@pytest.mark.parametrize("tokens,experts,top_k", [(40000, 65, 8), (5000, 70, 64)])
def test_route_of_more_choices_than_a_block_holds(tokens, experts, top_k, bf16, masked, renormalize):
    """256 blocks of more than 1024 choices each."""
    q = require_gpu()
    assert tokens * top_k > 256 * 1024
    t, x = logits_of(tokens + experts, tokens, experts, bf16, masked)
    say("route", tokens, experts, top_k, bf16, masked, renormalize)
    ids, weights, plan = q.moe_route(t, top_k, renormalize=renormalize)
    want, w = rows.route(x, top_k, renormalize)
    assert np.array_equal(ids.cpu().numpy(), want)
    same_plan(plan, want, experts)
    # half a step of l - max (at most 20), the exponential's 2 steps, the sum's
    # additions (at most 2 logits a lane and 6 across lanes), the quotient's one
    tol = 2.0 ** -24 * (2 * 20 + 4 + 22 + 2)
    assert np.all(np.abs(weights.cpu().numpy() - w) <= tol * w + 2.0 ** -149)


@pytest.mark.parametrize("rank", [24, 32])
@pytest.mark.parametrize("tokens,count,n,k", [(200, 2, 320, 128), (130, 2, 144, 1280), (1000, 3, 528, 2048)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_ranks_up_to_32_over_long_runs(rank, tokens, count, n, k, dtype):
    q = require_gpu()
    assert tokens >= 48 * count
    rng = np.random.default_rng([98, tokens, rank])
    ids = rng.integers(-1, count, tokens).astype(np.int32)
    bits, x = bf16_rows(tokens, tokens, k)
    y = synth.bf16_bits_as_f32(synth.to_bf16_bits(rng.standard_normal((tokens, n)).astype(np.float32)))
    a, b, scale = adapters_of(tokens, count, rank, n, k)
    say("lora", tokens, count, rank, n, k, dtype)
    plan = q.group_rows(torch.from_numpy(ids).cuda(), count)
    out = q.lora_add(on(y, dtype), dev_bf16(bits), on(a), on(b), plan, scale=on(scale, F32))
    want, bound = bound_of(y, x, a, b, scale, ids, dtype)
    far = np.abs(host_f64(out) - want)
    assert np.all(far <= bound), float((far / bound).max())
