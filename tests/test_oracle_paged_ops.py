"""Pins of the oracle of the operators around the paged cache."""

import numpy as np
import pytest

from oracle import decode as od
from oracle import paged_ops as op

FREQ = 10000.0 ** (-np.arange(8) / 8.0)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_norms_and_composes(interleaved):
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 2, 24))
    a, b = rng.integers(0, 1000, 5), rng.integers(0, 1000, 5)
    y = op.rotate(x, a, FREQ, interleaved)
    assert np.allclose((y[..., :16] ** 2).sum(-1), (x[..., :16] ** 2).sum(-1), rtol=1e-13)
    assert (y[..., 16:] == x[..., 16:]).all()
    assert np.allclose(op.rotate(y, b, FREQ, interleaved), op.rotate(x, a + b, FREQ, interleaved),
                       atol=1e-12)
    assert np.allclose(op.rotate(x, np.zeros(5), FREQ, interleaved), x)


@pytest.mark.parametrize("interleaved", [False, True])
def test_products_depend_on_the_distance_only(interleaved):
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((1, 1, 16)), rng.standard_normal((1, 1, 16))

    def dot(m, n):
        return (op.rotate(q, np.array([m]), FREQ, interleaved)
                * op.rotate(k, np.array([n]), FREQ, interleaved)).sum()

    assert abs(dot(70, 20) - dot(5050, 5000)) < 1e-9


def test_the_layouts_are_permutations_of_each_other():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((3, 2, 16))
    perm = np.concatenate([np.arange(0, 16, 2), np.arange(1, 16, 2)])
    pos = np.array([3, 1, 900])
    assert np.allclose(op.rotate(x, pos, FREQ, True)[..., perm],
                       op.rotate(x[..., perm], pos, FREQ, False), atol=1e-14)


def test_page_scores_bound_every_logit():
    rng = np.random.default_rng(3)
    k = rng.standard_normal((4, 16, 2, 8))
    bounds = op.page_bounds(k, np.array([[2, 0, 3]]), np.array([47]), None,
                            np.zeros((4, 2, 2, 8)), 16)
    assert (bounds[3] == 0).all() and (bounds[1] == 0).all()      # incomplete; not in the table
    q = rng.standard_normal((6, 8))
    s = op.page_scores(q, bounds, np.array([2, 0]))
    for kv in range(2):
        for p, blk in enumerate((2, 0)):
            logits = k[blk, :, kv] @ q[kv * 3:(kv + 1) * 3].T
            assert s[kv, p] >= logits.max() - 1e-12


def test_selection_ties_go_to_the_lower_page():
    assert op.select_pages(np.zeros(10), 5, 1, 1).tolist() == [0, 1, 2, 3, 9]
    assert op.select_pages(np.arange(10.0), 5, 1, 1).tolist() == [0, 6, 7, 8, 9]
    assert op.select_pages(np.zeros(3), 5, 1, 1).tolist() == [0, 1, 2, -1, -1]
    assert op.select_pages(np.zeros(9), 3, 1, 2).tolist() == [0, 7, 8]


def test_with_every_page_it_is_decode_attention():
    rng = np.random.default_rng(4)
    k, v = rng.standard_normal((9, 16, 2, 8)), rng.standard_normal((9, 16, 2, 8))
    q = rng.standard_normal((3, 4, 8))
    table = np.array([[0, 3, 5], [1, -1, -1], [-1, -1, -1]])
    lengths = np.array([40, 7, 0])
    out, mag = op.dense_attention(q, k, v, table, lengths, 0.4, 16)
    assert np.allclose(out, od.decode_attention(q, k, v, table, lengths, 0.4, 16), atol=1e-14)
    assert (np.abs(out) <= mag + 1e-14).all()
