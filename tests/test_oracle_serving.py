"""Pins of the serving oracle (oracle/serving.py) against torch and closed forms."""
import math

import numpy as np
import pytest
import torch

from oracle import serving as O


def test_rotation_is_a_rotation_and_relative():
    g = np.random.default_rng(0)
    f, mag = O.rope_freqs(32, 1e4)
    assert mag == 1.0 and f[0] == 1.0 and np.all(np.diff(f) < 0)
    x = g.standard_normal((3, 2, 48))
    for inter in (False, True):
        y = O.rotate(x, [0, 5, 70000], f, 1.0, inter)
        assert np.array_equal(y[0], x[0])                      # position 0
        assert np.array_equal(y[..., 32:], x[..., 32:])        # past rot_dim
        assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
        q, k = x[:1], x[1:2]
        dots = [(O.rotate(q, [s + 3], f, 1.0, inter) * O.rotate(k, [s], f, 1.0, inter)).sum()
                for s in (0, 11, 1000)]
        assert np.allclose(dots, dots[0])


def test_half_and_interleaved_are_the_same_up_to_order():
    g = np.random.default_rng(1)
    x = g.standard_normal((4, 1, 16))
    f, _ = O.rope_freqs(16, 1e4)
    perm = np.r_[np.arange(0, 16, 2), np.arange(1, 16, 2)]
    a = O.rotate(x, np.arange(4), f, 1.0, True)[..., perm]
    b = O.rotate(x[..., perm], np.arange(4), f, 1.0, False)
    assert np.allclose(a, b)


def test_scaled_frequencies():
    f, _ = O.rope_freqs(64, 1e6)
    assert np.allclose(O.rope_freqs(64, 1e6, "linear", 4.0)[0] * 4.0, f)
    ntk = O.rope_freqs(64, 1e6, "ntk", 4.0)[0]
    assert ntk[0] == 1.0 and math.isclose(ntk[-1] * 4.0, f[-1], rel_tol=1e-9)  # slowest pair: / factor
    y, mag = O.rope_freqs(64, 1e6, "yarn", 4.0, 32768)
    assert math.isclose(mag, 0.1 * math.log(4.0) + 1.0)
    assert np.allclose(y[0], f[0]) and np.allclose(y[-1], f[-1] / 4.0)
    assert np.all(y <= f * (1 + 1e-12)) and np.all(y >= f / 4.0 * (1 - 1e-12))


@pytest.mark.parametrize("causal", [False, True])
def test_attend_against_sdpa(causal):
    g = torch.Generator().manual_seed(2)
    q, k, v = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((5, 4, 16), (9, 2, 16), (9, 2, 16)))
    limits = [9 - 5 + i + 1 for i in range(5)] if causal else [9] * 5
    out, lse, _ = O.attend(q.numpy(), k.numpy(), v.numpy(), 0.25, limits)
    mask = torch.arange(9)[None] < torch.tensor(limits)[:, None]
    kk, vv = (t.repeat_interleave(2, 1).transpose(0, 1) for t in (k, v))
    ref = torch.nn.functional.scaled_dot_product_attention(q.transpose(0, 1), kk, vv, attn_mask=mask, scale=0.25)
    assert np.allclose(out, ref.transpose(0, 1).numpy())
    s = torch.where(mask, 0.25 * (q.transpose(0, 1) @ kk.transpose(1, 2)), -math.inf)
    assert np.allclose(lse, torch.logsumexp(s, -1).T.numpy())


def test_attend_empty_rows():
    out, lse, _ = O.attend(np.ones((2, 1, 4)), np.ones((3, 1, 4)), np.ones((3, 1, 4)), 1.0, [0, -2])
    assert not out.any() and np.all(lse == -np.inf)


def test_sample_hand_worked():
    z = np.log(np.array([0.1, 0.4, 0.2, 0.3]))
    assert O.sample(z, 1.0, 0, 1.0, 0.0, 0.05)[:2] == (0, 4)
    assert O.sample(z, 1.0, 0, 1.0, 0.0, 0.2)[0] == 1
    assert O.sample(z, 1.0, 2, 1.0, 0.0, 0.5)[:2] == (1, 2)       # {1, 3}: 4/7, 3/7
    assert O.sample(z, 1.0, 2, 1.0, 0.0, 0.6)[0] == 3
    assert O.sample(z, 1.0, 0, 0.65, 0.0, 0.9)[:2] == (3, 2)      # 0.4 + 0.3 >= 0.65
    assert O.sample(z, 1.0, 3, 0.75, 0.0, 0.0)[1] == 2            # of K's mass 0.9: 0.675 <= 0.7
    assert O.sample(z, 1.0, 0, 1.0, 0.6, 0.0)[1] == 2             # ratio to 0.4: 0.75 stays, 0.5 not
    assert O.sample(z, 0.0, 0, 1.0, 0.0, 0.9)[:3] == (1, 1, 0.0)
    assert O.sample(z, 1.0, 0, 0.0, 0.0, 0.9)[:2] == (1, 1)
    t = O.sample(z, 1.0, 0, 1.0, 0.0, 0.2)
    assert math.isclose(t[2], math.log(0.4))


def test_sample_ties_and_masks():
    z = np.array([1.0, 2.0, 2.0, 2.0, -np.inf])
    assert O.sample(z, 1.0, 2, 1.0, 0.0, 0.99)[:2] == (2, 2)      # lowest indices of the tie
    assert O.sample(z, 1.0, 0, 1.0, 0.0, 0.9999)[1] == 4
    assert O.sample(np.full(3, -np.inf), 1.0, 0, 1.0, 0.0, 0.5)[0] == -1
    assert O.sample(np.array([0.0, np.nan]), 1.0, 0, 1.0, 0.0, 0.5)[0] == -1


def test_sample_frequencies():
    g = np.random.default_rng(3)
    z = g.standard_normal(6)
    w = np.exp(z / 0.7)
    top = np.argsort(-z)[:4]
    p = np.where(np.isin(np.arange(6), top), w, 0.0)
    p /= p.sum()
    n = 4000
    hits = np.bincount([O.sample(z, 0.7, 4, 1.0, 0.0, (i + 0.5) / n)[0] for i in range(n)], minlength=6)
    assert np.abs(hits / n - p).max() <= 1.0 / n
