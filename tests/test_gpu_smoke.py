"""The figures that smoke() prints are those of its checks."""

import re

import pytest

from oracle import gemm
from tests.gpu_common import require_gpu, say

pytestmark = pytest.mark.gpu


def test_printed_figures_are_the_checked_ones(capsys):
    require_gpu()
    import __graft_entry__
    say("smoke")
    __graft_entry__.smoke()
    line = capsys.readouterr().out.split("smoke ok:")[1]
    errors = {name.strip(): float(v) for name, v in re.findall(r"([^,]+?) err ([0-9.e+-]+)", line)}
    assert {"w4a4", "fused quantize + w4a4", "w4a16", "w4a16 2:4", "lut2", "experts", "adapter"} == set(errors)
    assert all(0 < v <= gemm.TOL for v in errors.values()), errors
    assert 0 < float(re.search(r"attention ([0-9.]+) of its error bound", line)[1]) <= 1
