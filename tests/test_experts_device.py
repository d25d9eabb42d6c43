"""RoutedExperts works on its tensors' device, whichever is current: no GPU needed,
the calls are recorded."""

from types import SimpleNamespace

import pytest
import torch

from decode_nvfp4_rtn_amd import experts, qlin


@pytest.fixture
def current(monkeypatch):
    """The current device's number, and the device of each library call."""
    at, seen = [0], []

    class Device:
        def __init__(self, device):
            self.index = device if isinstance(device, int) else device.index

        def __enter__(self):
            self.before, at[0] = at[0], self.index

        def __exit__(self, *a):
            at[0] = self.before
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: at[0], raising=False)

    def note(name, result):
        monkeypatch.setattr(qlin, name, lambda *a, **k: seen.append((name, at[0])) or result)
    note("moe_route", (None, None, None))
    for name in ("quantize_nvfp4", "quantize_int4_g128"):
        note(name, (None, None, None))
    for name in ("moe_gemm_w4a4", "moe_gemm_w4a16", "moe_combine", "repack_weights"):
        note(name, "out")
    return at, seen


class Weights:
    """A stack of zeros that says it lies on cuda:1."""

    def __init__(self, *shape):
        self.shape, self.device = shape, torch.device("cuda", 1)

    def __iter__(self):
        return iter([torch.zeros(self.shape[1:])] * self.shape[0])


def test_calls_go_to_the_tensors_device(current, monkeypatch):
    at, seen = current
    monkeypatch.setattr(experts.torch, "empty", lambda *a, **k: [None] * 3)
    layer = experts.RoutedExperts(Weights(3, 256, 128), Weights(3, 128, 128), 2)
    assert {d for _, d in seen} == {1} and len(seen) > 8
    seen.clear()
    x, logits = (SimpleNamespace(shape=s, device=torch.device("cuda", 1)) for s in ((40, 128), (40, 3)))
    for prompt in (True, False, None):
        assert layer.forward(x, logits, prompt) == "out"
    assert {d for _, d in seen} == {1} and {"quantize_nvfp4", "moe_route", "moe_combine"} <= {n for n, _ in seen}
    assert at == [0]
