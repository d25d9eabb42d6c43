"""RoutedExperts on a step's tokens: each sequence meets the weights of its kind,
whoever shares the step."""

import pytest
import torch

from tests.gpu_common import require_gpu, say
from tests.test_gpu_experts import weights_of

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
HIDDEN, EXPERTS = 256, 6


def layer_and_step(nodes, settled, prompt=None, tree=None):
    require_gpu()
    from decode_nvfp4_rtn_amd.attention import PagedSequences
    from decode_nvfp4_rtn_amd.experts import RoutedExperts
    up, down = weights_of(7, EXPERTS, 128, HIDDEN)
    layer = RoutedExperts(torch.from_numpy(up).cuda(), torch.from_numpy(down).cuda(), 2)
    p = PagedSequences(64, 16)
    seqs = [p.add() for _ in nodes]
    p.settle(seqs, settled)
    g = torch.Generator(device="cuda").manual_seed(sum(nodes))
    x = torch.randn((sum(nodes), HIDDEN), generator=g, device="cuda").to(BF)
    logits = torch.randn((sum(nodes), EXPERTS), generator=g, device="cuda")
    return layer, p.step(seqs, nodes, prompt=prompt, tree=tree), x, logits


def test_a_decode_batch_of_any_size():
    """40 sequences' single tokens are decoding, as each of them alone is."""
    layer, step, x, logits = layer_and_step([1] * 40, [5] * 40)
    say("decode batch")
    out = layer.forward(x, logits, step=step)
    assert torch.equal(out, layer.forward(x, logits, False)) and out.any()
    assert not torch.equal(out, layer.forward(x, logits, True))


def test_a_short_prompt():
    layer, step, x, logits = layer_and_step([7], [0])
    say("short prompt")
    assert torch.equal(layer.forward(x, logits, step=step), layer.forward(x, logits, True))


def test_a_mixed_step():
    """Rows of a chunk are what the chunk alone gives, the others what they give
    without it."""
    layer, step, x, logits = layer_and_step([1, 1, 30, 5, 0, 1], [9, 9, 9, 0, 9, 9])
    say("mixed step")
    out = layer.forward(x, logits, step=step)
    for at, prompt in ((slice(0, 2), False), (slice(2, 37), True), (slice(37, 38), False)):
        assert torch.equal(out[at], layer.forward(x[at], logits[at], prompt)), at


def test_drafts_and_no_tokens():
    layer, step, x, logits = layer_and_step([20, 20], [9, 9], tree=[[1] * 20] * 2)
    say("drafts")
    assert torch.equal(layer.forward(x, logits, step=step), layer.forward(x, logits, False))
    layer, step, x, logits = layer_and_step([0, 0], [9, 9])
    assert layer.forward(x, logits, step=step).shape == (0, HIDDEN)


def test_a_step_that_does_not_say():
    layer, step, x, logits = layer_and_step([1] * 40, [5] * 40)
    step.prompt = None
    say("not said")
    assert torch.equal(layer.forward(x, logits, step=step), layer.forward(x, logits))


def test_refusals():
    layer, step, x, logits = layer_and_step([1, 4], [5, 5])
    for call in (lambda: layer.forward(x, logits, True, step=step),
                 lambda: layer.forward(x[:4], logits[:4], step=step), lambda: layer.forward(x, logits[:4])):
        with pytest.raises(ValueError):
            call()


def test_tokens_without_experts_may_hold_anything_when_decoding():
    """Masked tokens' rows of NaN and infinities reach no other token."""
    layer, step, x, logits = layer_and_step([1] * 40, [5] * 40)
    say("masked rows")
    masked = torch.arange(40, device="cuda") % 3 == 1
    logits[masked] = float("-inf")
    want = layer.forward(x, logits, step=step)
    x[masked] = float("nan")
    x[1] = float("inf")
    out = layer.forward(x, logits, step=step)
    assert torch.equal(out, want) and not out[masked].any() and out[~masked].any(1).all()
