"""Pins of the gate and int8-product oracles that do not reuse their formulas (CPU)."""
import itertools

import numpy as np
import pytest
import torch

from oracle import gate as ogate
from oracle import int8 as oint8
from oracle import moe as omoe


def test_plain_softmax_gate_is_the_layers_gate():
    rng = np.random.default_rng(0)
    x, wr, b = rng.standard_normal((40, 16)), rng.standard_normal((7, 16)), rng.standard_normal(7)
    for K in (1, 2, 5):
        ids, w, _ = ogate.route(x, wr, b, K)
        rid, rw, _ = omoe.route(x, wr, b, K)
        assert np.array_equal(ids, rid) and np.allclose(w, rw, rtol=1e-12)


def test_scores_against_torch():
    l = np.random.default_rng(1).standard_normal((5, 9)) * 20
    assert np.allclose(ogate.scores(l, False), torch.softmax(torch.from_numpy(l), 1).numpy(), rtol=1e-12, atol=0)
    assert np.allclose(ogate.scores(l, True), torch.sigmoid(torch.from_numpy(l)).numpy(), rtol=1e-12, atol=0)


@pytest.mark.parametrize("top2", [False, True])
def test_groups_by_brute_force(top2):
    """The kept groups are the subset with the largest total of group values, the experts the best of their subset."""
    rng = np.random.default_rng(2)
    for _ in range(30):
        G, n = rng.integers(2, 5), rng.integers(2, 5)
        gk = rng.integers(1, G + 1)
        K = rng.integers(1, gk * n + 1)
        s = rng.random(G * n)
        b = rng.standard_normal(G * n) * 0.3
        ids, w = ogate.choose(s, K, b, groups=G, group_topk=gk, top2=top2, renorm=False)
        c = (s + b).reshape(G, n)
        val = np.sort(c, 1)[:, -2:].sum(1) if top2 else c.max(1)
        best = max(itertools.combinations(range(G), gk), key=lambda k: val[list(k)].sum())
        allowed = [g * n + i for g in best for i in range(n)]
        chosen = max(itertools.combinations(allowed, K), key=lambda k: (s + b)[list(k)].sum())
        assert sorted(ids) == sorted(chosen)
        assert (np.diff((s + b)[ids]) <= 0).all() and np.array_equal(w, s[ids])


def test_ties_disabled_experts_and_weights():
    assert ogate.choose([0.5, 0.5, 0.5], 2)[0] == [0, 1]
    assert ogate.choose([0.2, 0.2, 0.2, 0.2], 1, groups=2, group_topk=1)[0] == [0]
    inf = float("inf")
    ids, w = ogate.choose([0.5, 0.25, 0.125], 3, [-inf, 0, float("nan")], scale=2.0)
    assert ids == [1, -1, -1] and w == [2.0, 0.0, 0.0]
    assert ogate.choose([0.0, 0.0], 2) == ([0, 1], [0.0, 0.0])          # a sum of zero
    assert ogate.choose([0.1, 0.9], 2, [5.0, 0.0], renorm=False) == ([0, 1], [0.1, 0.9])


def test_product_against_integer_loops():
    rng = np.random.default_rng(3)
    a, w = rng.integers(-127, 128, (4, 6)), rng.integers(-127, 128, (2, 3, 6))
    a_s, w_s = rng.random(4), rng.random((2, 3))
    off, rows = [0, 1, 3], [2, 0, 3, 1]
    got = oint8.grouped_product(a, a_s, w, w_s, off, rows)
    for r, e in ((0, 0), (1, 1), (2, 1)):
        for n in range(3):
            p = sum(int(a[rows[r], k]) * int(w[e, n, k]) for k in range(6))
            assert got[r, n] == pytest.approx(p * a_s[rows[r]] * w_s[e, n], rel=1e-14)
    assert np.isnan(got[3]).all()
    two = oint8.grouped_product(a, a_s, w, w_s, off, rows, w, w_s)
    g = torch.from_numpy(got[:3])
    assert np.allclose(two[:3], (torch.nn.functional.silu(g) * g).numpy(), rtol=1e-12)
