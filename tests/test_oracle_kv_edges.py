"""Pins of oracle/kvcache.py where a rounding could go wrong."""

import numpy as np

from oracle import kvcache as kv


def test_bf16_rows_of_binary64_values_are_rounded_once():
    """Values around the middles between bf16 values, nearer to them than
    binary32 can tell: the nearest of the two, the even one at the middle."""
    lo = np.float64(1 + np.arange(128) / 128)
    lo = np.concatenate([lo, -lo]) * 2.0 ** 3
    step = np.sign(lo) * 2.0 ** -7 * 2.0 ** 3
    for off, up in ((0.0, np.arange(256) % 2 == 1), (2.0 ** -44, np.ones(256, bool)), (-2.0 ** -44, np.zeros(256, bool))):
        x = lo + step * (0.5 + off)
        got = kv.quantize(kv.BF16, x.reshape(4, 64))["value"].ravel()
        assert np.array_equal(got, np.where(up, lo + step, lo))
    # binary32 rows are as ever
    y = np.random.default_rng(1).standard_normal((3, 64)).astype(np.float32)
    assert np.array_equal(kv.quantize(kv.BF16, y)["value"], kv.quantize(kv.BF16, y.astype(np.float64))["value"])
