"""Which weights the layer of decode_nvfp4_rtn_amd/attention.py takes: by what a
sequence's new tokens are, whoever shares the step."""

import pytest
import torch

from tests.gpu_common import require_gpu, say
from tests.test_gpu_paged_attention import HIDDEN, N_Q, _layer, _x

pytestmark = pytest.mark.gpu


@pytest.fixture
def calls(monkeypatch):
    """(weights, rows) of each projection, and the attentions' outputs."""
    q = require_gpu()
    made, outs = [], []

    def wrap(name, note):
        call = getattr(q, name)

        def wrapped(*a, **k):
            r = call(*a, **k)
            note(a, r)
            return r
        monkeypatch.setattr(q, name, wrapped)
    wrap("gemm_w4a16", lambda a, r: made.append(("int4", a[0].shape[0])))
    wrap("quantize_gemm_w4a4", lambda a, r: made.append(("nvfp4", a[0].shape[0])))
    wrap("kv_attention", lambda a, r: outs.append(r))
    return q, made, outs


def _forward(layer, calls, x, step):
    _, made, outs = calls
    made.clear()
    y = layer.forward(x, step)
    assert y.shape == (x.shape[0], HIDDEN) and outs[-1].shape[:2] == (x.shape[0], N_Q)
    assert torch.isfinite(y).all()
    used = list(made)
    assert used[:len(used) // 2] == used[len(used) // 2:]       # both projections alike
    return y, used[:len(used) // 2]


def test_decoding_and_prompts_of_any_number(calls):
    from decode_nvfp4_rtn_amd.attention import PagedSequences
    say("layer weights")
    layer, p = _layer(calls[0], "e4m3"), PagedSequences(24, 16)
    seqs = [p.add() for _ in range(23)]
    _, used = _forward(layer, calls, _x(20, 1), p.step(seqs[:1], [20]))
    assert used == [("nvfp4", 20)]                              # a short prompt
    p.settle(seqs[:1], [20])
    _, used = _forward(layer, calls, _x(22, 6), p.step(seqs[1:], [1] * 22))
    assert used == [("nvfp4", 22)]                              # prompts of one token
    p.settle(seqs[1:], [1] * 22)
    step = p.step(seqs, [2] * 23, tree=[[1, 3]] * 23)
    _, used = _forward(layer, calls, _x(46, 2), step)
    assert used == [("int4", 46)]                               # many drafts


def test_a_chunk_beside_decoding(calls):
    """Each part's rows are what its own weights give."""
    from decode_nvfp4_rtn_amd.attention import PagedSequences
    q, _, outs = calls
    say("layer weights, mixed")
    layer, p = _layer(q, "bf16"), PagedSequences(24, 16)
    seqs = [p.add() for _ in range(4)]
    x = _x(63, 3)
    _forward(layer, calls, x, p.step(seqs[:3], [40, 20, 3]))
    p.settle(seqs[:3], [40, 20, 3])
    x = _x(44, 4)
    step = p.step(seqs, [1, 1, 32, 10])                         # two decode, a chunk, a new prompt
    y, used = _forward(layer, calls, x, step)
    assert used == [("int4", 2), ("nvfp4", 42)]
    a = outs[-1].flatten(1)
    assert torch.equal(y[:2], layer.project(a[:2], 1, False)) and torch.equal(y[2:], layer.project(a[2:], 1, True))
    # the two sequences' keys and values are those of a step of their own
    at = step.slots[:2]
    kept = q.kv_gather(layer.cache, at)
    q.kv_append(layer.cache, torch.zeros_like(kept[0]), torch.zeros_like(kept[1]), at)
    layer.forward(x[:2], p.step(seqs[:2], [1, 1]))
    again = q.kv_gather(layer.cache, at)
    assert torch.equal(kept[0], again[0]) and torch.equal(kept[1], again[1])
    step = p.step(seqs, [1, 30, 1, 1], prompt=[False, True, False, False])
    _, used = _forward(layer, calls, _x(33, 5), step)
    assert used == [("int4", 1), ("nvfp4", 30), ("int4", 2)]
