"""Pins of oracle/rows.py: plans, choices and products against other
definitions of the same."""

import numpy as np
import pytest
import torch

from oracle import rows


def test_plan_is_a_stable_sort():
    rng = np.random.default_rng(3)
    for groups in (1, 5, 40):
        ids = rng.integers(-2, groups + 2, 300)
        order, where, offsets = rows.plan(ids, groups)
        key = np.where((ids >= 0) & (ids < groups), ids, groups)
        assert np.array_equal(order, np.argsort(key, kind="stable"))
        assert np.array_equal(where[order], np.arange(300))
        assert np.array_equal(np.diff(offsets), np.bincount(key, minlength=groups + 1)[:groups])


def test_plan_by_hand():
    order, where, offsets = rows.plan([2, -1, 0, 2, 7, 0], 3)
    assert order.tolist() == [2, 5, 0, 3, 1, 4] and offsets.tolist() == [0, 2, 2, 4]
    assert where.tolist() == [2, 4, 0, 3, 5, 1]


@pytest.mark.parametrize("renormalize", [True, False])
def test_route_against_softmax(renormalize):
    x = torch.randn(50, 24, dtype=torch.float64, generator=torch.Generator().manual_seed(1))
    ids, w = rows.route(x.numpy(), 5, renormalize)
    p = x.softmax(1)
    values, at = p.topk(5, 1)
    if renormalize:
        values = values / values.sum(1, keepdim=True)
    assert np.array_equal(ids, at.numpy())
    assert np.allclose(w, values.numpy(), rtol=1e-13, atol=0)


def test_route_masks_and_ties():
    inf, nan = np.inf, np.nan
    x = np.array([[1.0, 1.0, 1.0, 1.0], [-inf, 2.0, -inf, nan], [-inf, -inf, nan, -inf], [inf, 0.0, inf, 1.0],
                  [0.0, -0.0, -1.0, 0.0]])
    ids, w = rows.route(x, 3, False)
    assert ids.tolist() == [[0, 1, 2], [1, -1, -1], [-1, -1, -1], [0, 2, 3], [0, 1, 3]]
    assert w[0].tolist() == [0.25] * 3 and w[1].tolist() == [1, 0, 0] and not w[2].any()
    assert w[3].tolist() == [0.5, 0.5, 0]


def test_products_and_sum_against_a_dense_mixture():
    """Every token times every expert, masked by the choices."""
    rng = np.random.default_rng(5)
    t, e, k, n, top_k = 9, 6, 7, 4, 3
    x, w = rng.standard_normal((t, k)), rng.standard_normal((e, n, k))
    ids, weights = rows.route(rng.standard_normal((t, e)), top_k, True)
    ids[4], weights[4] = -1, 0
    order, where, offsets = rows.plan(ids, e)
    y = rows.experts_product(x, list(w), order, offsets, top_k, True)
    out = rows.combine(y, where.reshape(t, top_k), offsets, weights)
    gate = np.zeros((t, e + 1))
    for i in range(t):
        gate[i, ids[i]] += weights[i]
    assert np.allclose(out, np.einsum("te,enk,tk->tn", gate[:, :e], w, x), atol=1e-12)
    assert not y[offsets[-1]:].any() and not out[4].any()
    again = rows.experts_product(y[:, :k] if n >= k else np.pad(y, ((0, 0), (0, k - n))), list(w), order, offsets,
                                 top_k, False)
    assert np.allclose(again[offsets[-1] - 1], w[ids[ids >= 0].max()][:, :n] @ y[offsets[-1] - 1])


def test_silu():
    g = torch.linspace(-20, 20, 101, dtype=torch.float64)
    assert np.allclose(rows.silu(g.numpy()), torch.nn.functional.silu(g).numpy(), rtol=1e-12, atol=0)


def test_lora_is_a_merged_weight():
    rng = np.random.default_rng(6)
    x, y = rng.standard_normal((5, 8)), rng.standard_normal((5, 6))
    a, b = rng.standard_normal((2, 3, 8)), rng.standard_normal((2, 6, 3))
    scale = np.array([0.5, -2.0])
    out, mid, far = rows.lora(y, x, a, b, scale, [1, -1, 0, 2, 1])
    for t, i in ((0, 1), (2, 0), (4, 1)):
        assert np.allclose(out[t], y[t] + (scale[i] * b[i] @ a[i]) @ x[t])
    assert np.array_equal(out[[1, 3]], y[[1, 3]]) and not mid[1].any()
    assert (np.abs(out - y) <= mid + 1e-12).all() and (mid <= far + 1e-12).all()
