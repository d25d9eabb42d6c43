"""Host bookkeeping of decode_nvfp4_rtn_amd/attention.py: no GPU needed."""

import pytest
import torch

from decode_nvfp4_rtn_amd.attention import PagedSequences, rope_table


def test_steps_pages_and_slots():
    p = PagedSequences(6, 16, device="cpu")
    a, b = p.add(), p.add()
    s = p.step([a, b], [20, 3])
    assert s.cu_q.tolist() == [0, 20, 23] and s.kv_lens.tolist() == [20, 3] and s.max_kv == 20
    assert s.block_table.tolist() == [[0, 1], [2, -1]]
    assert s.slots.tolist() == list(range(20)) + [32, 33, 34]
    assert s.positions.tolist() == list(range(20)) + [0, 1, 2] and s.tree is None
    p.settle([a, b], [20, 3])
    s = p.step([b, a], [1, 4], tree=[[1], [1, 3, 5, 7]])
    assert s.slots.tolist() == [35, 20, 21, 22, 23]
    assert s.positions.tolist() == [3, 20, 21, 21, 22]          # by depth
    assert s.tree.tolist() == [1, 1, 3, 5, 7] and s.tree.dtype == torch.int64
    p.settle([b, a], [1, 2])
    assert p.lens == {a: 22, b: 4}
    # rejected drafts' places are taken again
    assert p.step([a], [1]).slots.tolist() == [22]
    p.free(b)
    c = p.add()
    assert p.step([c], [16]).block_table.tolist() == [[2]]
    assert p.step([], []).slots.numel() == 0


def test_masks_of_64_drafts():
    p = PagedSequences(8, 16, device="cpu")
    chain = [(2 << i) - 1 for i in range(64)]
    s = p.step([p.add()], [64], tree=[chain])
    assert s.tree[63].item() == -1 and s.tree[62].item() == (1 << 63) - 1
    assert s.positions.tolist() == list(range(64))


def test_refusals():
    p = PagedSequences(2, 16, device="cpu")
    a = p.add()
    with pytest.raises(RuntimeError):
        p.step([a], [33])
    assert p.pages[a] == [] and len(p.unused) == 2              # nothing was taken
    for bad in (lambda: p.step([a, a], [1, 1]), lambda: p.step([a], [1, 2]), lambda: p.step([a], [-1]),
                lambda: p.step([a], [2], tree=[[1]])):
        with pytest.raises(ValueError):
            bad()


def test_rope_table():
    t = rope_table(5, 8, device="cpu")
    assert t.shape == (5, 8) and t.is_contiguous()
    assert torch.equal(t[0], torch.tensor([1.0] * 4 + [0.0] * 4))
    assert torch.allclose(t[:, :4] ** 2 + t[:, 4:] ** 2, torch.ones(5, 4))
