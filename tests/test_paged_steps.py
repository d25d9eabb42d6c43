"""What a step says of its sequences' new tokens (decode_nvfp4_rtn_amd/attention.py):
no GPU needed."""

import pytest

from decode_nvfp4_rtn_amd.attention import PagedSequences


def test_kind_of_a_steps_tokens():
    p = PagedSequences(40, 16, device="cpu")
    a, b, c = p.add(), p.add(), p.add()
    assert p.step([a, b, c], [20, 1, 40]).prompt == [True, True, True]    # a prompt of one token too
    p.settle([a, b, c], [20, 1, 40])
    assert p.step([a, b, c], [1, 7, 0]).prompt == [False, True, False]    # a chunk beside decoding
    assert p.step([a, b], [3, 1], tree=[[1, 3, 5], [1]]).prompt == [False, False]
    assert p.step([a, b], [3, 1], prompt=[0, 1]).prompt == [False, True]  # as told
    with pytest.raises(ValueError):
        p.step([a, b], [3, 1], prompt=[True])
    assert p.step([], []).prompt == []
