"""Pins for the oracle of the paged cache, drafted trees and sampling: worked
rotations of both layouts and scalings, attention cases with closed forms, a
worked sampling row for every limit and every tie, and a worked tree."""
import math

import numpy as np
import pytest

import oracle


def test_rope_pairs_hand_worked():
    turns = np.array([0.25, 0.125])  # a quarter and an eighth of a turn per position
    x = np.array([[[1.0, 2.0, 3.0, 4.0, 5.0]]])
    r = math.sqrt(0.5)
    # halves: pairs (1, 3) and (2, 4); the fifth element passes through
    assert np.allclose(oracle.rope_pairs(x, [1], turns)[0, 0], [-3, (2 - 4) * r, 1, (4 + 2) * r, 5], atol=1e-15)
    # neighbours: pairs (1, 2) and (3, 4)
    assert np.allclose(oracle.rope_pairs(x, [1], turns, True)[0, 0], [-2, 1, (3 - 4) * r, (4 + 3) * r, 5], atol=1e-15)
    assert np.allclose(oracle.rope_pairs(x, [2], turns, True, 2.0)[0, 0], [-2, -4, -8, 6, 5], atol=1e-14)
    # the contiguous cache's rotation is the half layout of the whole head
    g = np.random.default_rng(1)
    y = g.standard_normal((1, 3, 64))
    assert np.allclose(oracle.rope_pairs(y, [37], oracle.rope_turns(64)), oracle.rope(y.ravel(), 37, 64).reshape(1, 3, 64),
                       atol=1e-12)


def test_rope_turns_scalings():
    f = oracle.rope_turns(8, 10000.0)
    assert np.allclose(f * 2 * np.pi, [1, 0.1, 0.01, 0.001], rtol=1e-14)
    assert np.allclose(oracle.rope_turns(8, 10000.0, factor=4.0), f / 4, rtol=1e-14)
    # by parts over 628.3 positions: 100, 10, 1, 0.1 turns; 2 .. 18 is the ramp
    part = oracle.rope_turns(8, 10000.0, factor=4.0, orig_len=628, alpha=2.0, beta=18.0)
    r = 628 * f
    c = (r[1] - 2) / 16
    assert np.allclose(part, [f[0], f[1] * (c + (1 - c) / 4), f[2] / 4, f[3] / 4], rtol=1e-14)
    assert 0.49 < c < 0.51


def test_tree_attention_closed_forms():
    d = 4
    k = np.zeros((3, 1, d))
    v = np.arange(12.0).reshape(3, 1, d)
    q = np.zeros((3, 2, d))
    sees = np.array([[1, 0, 0], [1, 0, 1], [0, 0, 0]], bool)
    a, A = oracle.tree_attention(q, k, v, sees)
    assert np.allclose(a[0, 0], v[0, 0]) and np.allclose(a[1, 1], (v[0, 0] + v[2, 0]) / 2)
    assert not a[2].any() and not A[2].any()
    v[1] = np.nan  # a row that nobody sees
    assert np.isfinite(oracle.tree_attention(q, k, v, sees)[0]).all()
    # scores ln 3 and 0 weigh 3/4 and 1/4
    q[0, 0, 0] = k[0, 0, 0] = math.sqrt(math.log(3) * math.sqrt(d))
    a, _ = oracle.tree_attention(q[:1, :1], k[::2], v[::2], np.ones((1, 2), bool))
    assert np.allclose(a[0, 0], 0.75 * v[0, 0] + 0.25 * v[2, 0])


def test_tree_sees():
    want = [[1, 0, 0, 0], [1, 1, 0, 0], [1, 0, 1, 0], [1, 1, 0, 1]]
    assert np.array_equal(oracle.tree_sees([-1, 0, 0, 1]), np.array(want, bool))


# weights 4, 2, 1, 1 (of 8) at indices 2, 0, 1, 4
ROW = [math.log(2), 0.0, math.log(4), -np.inf, 0.0]


@pytest.mark.parametrize("kw,want", [
    (dict(u=0.0), (2, 4 / 8)), (dict(u=0.49), (2, 4 / 8)), (dict(u=0.51), (0, 2 / 8)), (dict(u=0.76), (1, 1 / 8)),
    (dict(u=0.9999), (4, 1 / 8)), (dict(), (2, 1.0)), (dict(u=0.9, temperature=0.0), (2, 1.0)),
    (dict(u=0.9, top_k=1), (2, 1.0)), (dict(u=0.7, top_k=2), (0, 2 / 6)), (dict(u=0.99, top_k=3), (1, 1 / 7)),
    (dict(u=0.99, top_p=0.49), (2, 1.0)), (dict(u=0.99, top_p=0.51), (0, 2 / 6)), (dict(u=0.99, top_p=0.0), (2, 1.0)),
    (dict(u=0.99, top_k=2, top_p=0.65), (2, 1.0)),      # 4 of the first two's 6 come to it
    (dict(u=0.99, min_p=0.3), (0, 2 / 6)), (dict(u=0.99, min_p=2.0), (2, 1.0)),
    (dict(u=0.6, temperature=0.5), (2, 16 / 22)), (dict(u=0.9, temperature=0.5), (0, 4 / 22))])
def test_sample_worked(kw, want):
    tok, p = oracle.sample(ROW, **kw)
    assert tok == want[0] and abs(p - want[1]) < 1e-12


def test_sample_edges():
    assert oracle.sample([-np.inf, np.nan], u=0.5) == (-1, 0.0)
    assert oracle.sample([np.nan, -3.0], u=0.5) == (1, 1.0)
    assert oracle.sample([1.0, np.inf, 5.0, np.inf], u=0.6) == (3, 0.5)
    assert oracle.sample([0.0] * 4, u=0.5, top_p=0.5)[0] == 1  # two of four equal ones come to half; u is past the first


def test_tree_path():
    #        0: root; 1, 2, 3 continue it; 4, 5 continue 2; 6 continues 5
    parents = [-1, 0, 0, 0, 2, 2, 5]
    draft = [9, 1, 2, 2, 7, 8, 5]
    assert oracle.tree_path(draft, parents, [2, 0, 8, 0, 0, 5, 1]) == [0, 2, 5, 6]
    assert oracle.tree_path(draft, parents, [4, 0, 8, 0, 0, 5, 1]) == [0]
    assert oracle.tree_path(draft, parents, [2, 0, -1, 0, 0, 5, 1]) == [0, 2]
    assert oracle.tree_path([], [], []) == []
