"""Pins of oracle/kvcache.py: closed forms, torch's conversions, brute force."""

import math

import numpy as np
import pytest
import torch

from oracle import kvcache as kv, nvfp4
from tests.kv_common import random_tree, rows


def test_row_exponent_is_the_smallest_that_fits():
    for top in (448.0, 2688.0):
        for a in (1e-45, 1e-31, 0.1, 1.0, 447.0, 448.0, 448.5, 2688.0, 2689.0, 3e38):
            e = int(kv.row_exponent(np.array(a), top))
            assert a <= top * 2.0 ** e and (e == kv.E_MIN or a > top * 2.0 ** (e - 1))
        assert int(kv.row_exponent(np.array(0.0), top)) == 0


def test_e4m3_rows_are_torchs_casts():
    x = rows(1, 20, 1, 64, bf16=False)[:, 0]
    q = kv.quantize(kv.E4M3, x)
    e = q["exp"].astype(int) - 127
    y = torch.from_numpy(np.ldexp(x, -e[:, None]))
    assert np.array_equal(y.to(torch.float8_e4m3fn).view(torch.uint8).numpy(), q["row"])


def test_nvfp4_rows_are_nvfp4_with_a_power_of_two_tensor_scale():
    x = rows(2, 12, 1, 128)[:, 0]
    q = kv.quantize(kv.NVFP4, x)
    for i in range(12):
        s = np.float32(2.0 ** (int(q["exp"][i]) - 127))
        codes, scales, _ = nvfp4.quantize(x[i:i + 1], s)
        assert np.array_equal(codes[0], q["row"][i]) and np.array_equal(scales[0], q["scales"][i])
        assert np.array_equal(nvfp4.dequantize(codes, scales, s)[0], q["value"][i])


@pytest.mark.parametrize("fmt", [kv.BF16, kv.E4M3, kv.NVFP4])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_layout_uses_every_byte_once(fmt, d):
    off = kv.offsets(fmt, d)
    codes = np.concatenate([off["k"].ravel(), off["v"].ravel()])
    assert np.array_equal(np.sort(codes), np.arange(32 * kv.row_bytes(fmt, d)))
    if fmt == kv.NVFP4:
        sc = np.concatenate([off[n].ravel() for n in ("ks", "vs", "ke", "ve")])
        assert np.array_equal(np.sort(sc), np.arange(kv.scale_bytes(fmt, d)))
    elif fmt == kv.E4M3:
        assert np.array_equal(np.sort(np.concatenate([off["ke"], off["ve"]])), np.arange(32))


def test_norm_and_rotation_closed_forms():
    x = rows(3, 4, 2, 64).astype(np.float64)
    y = kv.norm_rope(x, np.full(64, 2.0), 0.0, None, None, False)
    assert np.allclose((y ** 2).mean(-1), 4.0)
    a = np.random.default_rng(1).standard_normal((9, 16))
    table = np.concatenate([np.cos(a), np.sin(a)], 1)
    pos = np.array([0, 8, 3, 20])
    for pairs in (False, True):
        z = kv.norm_rope(x, None, 0.0, table, pos, pairs)
        assert np.array_equal(z[..., 32:], x[..., 32:])            # past rot: as it was
        first, second = (np.arange(0, 32, 2), np.arange(1, 32, 2)) if pairs else (np.arange(16), np.arange(16, 32))
        c = x[..., first] + 1j * x[..., second]
        turn = np.exp(1j * a[np.minimum(pos, 8)])[:, None]
        assert np.allclose(z[..., first] + 1j * z[..., second], c * turn)


def test_attention_is_softmax_and_trees_are_chains_when_they_are():
    rng = np.random.default_rng(4)
    q, k, v = (rng.standard_normal(s) for s in ((3, 4, 8), (10, 2, 8), (10, 2, 8)))
    chain = np.array([1, 3, 7], dtype=object)
    sees = kv.visible(3, 10, chain)
    assert np.array_equal(sees, kv.visible(3, 10))
    y, mag, top, unit = kv.attention(q, k, v, sees, 0.3)
    for i in range(3):
        for h in range(4):
            s = [0.3 * math.fsum(q[i, h] * k[p, h // 2]) for p in range(8 + i)]
            w = np.exp(np.array(s) - max(s))
            assert np.allclose(y[i, h], (w[:, None] * v[:8 + i, h // 2]).sum(0) / w.sum())
    assert np.all(np.abs(y) <= mag + 1e-12) and np.all(top > 0) and np.all(unit + 1e-12 >= mag)
    y, _, _, _ = kv.attention(q, k, v, np.zeros((3, 10), dtype=bool), 0.3)
    assert not y.any()


def test_random_trees_are_closed_under_ancestors():
    for n in (1, 2, 40, 64):
        m = random_tree([n], n)
        for j in range(n):
            assert m[j] >> j & 1 and m[j] < 1 << j + 1
            for i in range(j):
                if m[j] >> i & 1:
                    assert m[i] & m[j] == m[i]
