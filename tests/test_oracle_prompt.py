"""Pins of the 64-bit oracle of the operators of a long prompt (oracle/serving.py)."""
import math

import numpy as np
import torch

from oracle import serving as O


def test_attention_mass_is_the_softmax_summed_over_rows():
    g = np.random.default_rng(1)
    q, k, v = g.standard_normal((5, 4, 8)), g.standard_normal((9, 2, 8)), g.standard_normal((9, 2, 8))
    limits = [5, 6, 7, 8, 9]
    _, lse, _ = O.attend(q, k, v, 0.3, limits)
    mass = O.attention_mass(q, k, lse, 0.3, limits)
    want = np.zeros((2, 9))
    for i in range(5):
        for h in range(4):
            s = torch.from_numpy(0.3 * k[:limits[i], h // 2] @ q[i, h])
            want[h // 2, :limits[i]] += torch.softmax(s, 0).numpy()
    assert np.allclose(mass, want, rtol=1e-12, atol=1e-15)
    assert np.allclose(mass.sum(1), 10.0)            # five rows, two heads: each adds one
    assert not O.attention_mass(q, k, lse, 0.3, [0] * 5).any()


def test_evict_hand_worked():
    m = np.array([0.1, 0.5, 0.5, 0.0, 0.9, 0.2])
    assert O.evict(m, 6, 2, 0, 0) == [1, 4]                # of the equals the lower position
    assert O.evict(m, 6, 3, 0, 0) == [1, 2, 4]
    assert O.evict(m, 6, 3, 1, 1) == [0, 4, 5]
    assert O.evict(m, 6, 2, 3, 3) == [0, 1]                # more protected than kept
    assert O.evict(m, 4, 9, 0, 0) == [0, 1, 2, 3]
    assert O.evict(m, 6, 0, 1, 1) == [] and O.evict(m, 6, -2, 1, 1) == []
    m[4] = math.nan
    assert O.evict(m, 6, 5, 0, 0) == [0, 1, 2, 3, 5]       # NaN comes last
    assert O.evict(np.array([0.0, -0.0, -1.0, -math.inf]), 4, 2, 0, 0) == [0, 1]


def test_evict_against_a_sort():
    g = np.random.default_rng(2)
    for _ in range(50):
        n = int(g.integers(1, 60))
        m = g.integers(0, 6, n).astype(float)
        keep, sink, recent = (int(x) for x in g.integers(0, n + 3, 3))
        w = m.copy()
        w[:sink] = np.inf
        w[max(0, n - recent):] = np.inf
        order = np.argsort(-w, kind="stable")[:min(keep, n)]
        assert O.evict(m, n, keep, sink, recent) == sorted(order.tolist())


def test_score_against_torch():
    g = np.random.default_rng(3)
    z = g.standard_normal(50) * 3
    z[7] = -math.inf
    for T in (0.5, 1.0, 2.0):
        lp = torch.log_softmax(torch.from_numpy(z / T), 0).numpy()
        p = np.exp(lp)
        lp11, rank, ent, ids, tops = O.score(z, T, 11, 6)
        assert math.isclose(lp11, lp[11], rel_tol=1e-12)
        assert math.isclose(ent, -float((p[p > 0] * lp[p > 0]).sum()), rel_tol=1e-12)
        order = np.argsort(-z, kind="stable")
        assert rank == list(order).index(11) and ids == order[:6].tolist() and np.allclose(tops, lp[order[:6]])
    assert O.score(z, 1.0, 7, 0)[:2] == (-math.inf, 49)
    assert O.score(z, 1.0, -1, 60)[:2] == (0.0, -1) and len(O.score(z, 1.0, -1, 60)[3]) == 49
    assert O.score(np.array([1.0, 2.0, 2.0]), 1.0, 2, 3)[1:4:2] == (1, [1, 2, 0])        # ties: the lower index
    for bad in ([-math.inf] * 3, [0.0, math.nan], [0.0, math.inf]):
        assert O.score(np.array(bad), 1.0, 0, 1) is None
