"""Pins of the fp64 definitions for drafted trees (CPU only): against the single-token step, which is
itself pinned by brute force, and against what speculative sampling promises -- the emitted tokens
are distributed as samples of the target, whatever the draft."""

import numpy as np
import pytest

from oracle import favor, features, speculative


def problem(T, d=8, m=24, seed=0, prior=5):
    g = np.random.default_rng(seed)
    W = features.draw_W(3, m, d)
    Q, K, V = (g.standard_normal((T, d)) for _ in range(3))
    S, z = np.zeros((m, d)), np.zeros(m)
    for _ in range(prior):
        _, S, z = favor.decode_step(S, z, *g.standard_normal((3, d)), W)
    return S, z, Q, K, V, W


@pytest.mark.parametrize("prior", [0, 5])
def test_chain_is_the_single_token_step(prior):
    S, z, Q, K, V, W = problem(9, prior=prior)
    out = speculative.decode_tree(S, z, Q, K, V, W, list(range(-1, 8)))
    for t in range(9):
        o, S, z = favor.decode_step(S, z, Q[t], K[t], V[t], W)
        assert np.allclose(out[t], o, rtol=1e-12, atol=1e-13)


def test_every_path_of_a_tree_is_a_chain():
    parents = [-1, 0, 0, 1, 1, 2, 3, -1, 7]
    S, z, Q, K, V, W = problem(len(parents))
    out = speculative.decode_tree(S, z, Q, K, V, W, parents)
    for i in range(len(parents)):
        Si, zi = S, z
        for j in reversed(speculative.ancestors(parents, i)):
            o, Si, zi = favor.decode_step(Si, zi, Q[j], K[j], V[j], W)
        assert np.allclose(out[i], o, rtol=1e-12, atol=1e-13)


def test_extend_is_repeated_steps_in_any_order():
    S, z, Q, K, V, W = problem(7)
    S1, z1 = speculative.decode_extend(S, z, K, V, W, [4, 2, 2, 6])
    for j in (2, 6, 4, 2):
        _, S, z = favor.decode_step(S, z, Q[j], K[j], V[j], W)
    assert np.allclose(S1, S, rtol=1e-12) and np.allclose(z1, z, rtol=1e-12)


def _emitted(dense, n=60000):
    """First emitted token of a walk over a root with three drafted children, many times over."""
    g = np.random.default_rng(1)
    V = 5
    target, draft = np.array([0.35, 0.05, 0.3, 0.1, 0.2]), np.array([0.1, 0.4, 0.2, 0.25, 0.05])
    parents = [-1, 0, 0, 0]
    p = np.tile(target, (4, 1))
    hist = np.zeros(V)
    for _ in range(n):
        drafted = g.choice(V, 3, p=draft) if dense else g.choice(V, 3, replace=False)
        tokens = [0, *drafted]
        path, nxt = speculative.verify(parents, tokens, p, np.tile(draft, (4, 1)) if dense else None, g.random(4),
                                       g.random())
        hist[tokens[path[1]] if len(path) > 1 else nxt] += 1
    return hist / n, target


@pytest.mark.parametrize("dense", [True, False])
def test_emitted_tokens_follow_the_target(dense):
    n = 60000
    hist, target = _emitted(dense, n)
    # binomial standard deviations; 4.5 of them over ten comparisons
    assert (np.abs(hist - target) <= 4.5 * np.sqrt(target * (1 - target) / n)).all()


def test_walk_by_hand():
    p = np.array([[0.5, 0.3, 0.2], [0.1, 0.1, 0.8], [0.25, 0.25, 0.5]])
    q = np.array([[0.2, 0.7, 0.1], [0.3, 0.3, 0.4], [1.0, 0.0, 0.0]])
    parents, tokens = [-1, 0, 0], [9, 1, 0]
    # node 1 (token 1): 0.5 * 0.7 >= 0.3, rejected; residual [0.3, 0, 0.1], Z = 0.4; node 2 (token 0):
    # u 0.4 0.2 < 0.3 for every u in [0, 1): accepted; its row decides the next token
    assert speculative.verify(parents, tokens, p, q, [0, 0.5, 0.99], 0.49) == ([0, 2], 1)
    # point masses: node 1 rejected (0.5 >= 0.3), residual [0.5, 0, 0.2], Z = 0.7; node 2: 0.8 * 0.7 >= 0.5
    assert speculative.verify(parents, tokens, p, None, [0, 0.5, 0.8], 0.0) == ([0], 2)
    # a draft equal to the target: nothing left after a rejection, the target's own row is sampled
    same = np.tile(p[0], (3, 1))
    assert speculative.verify([-1, 0], [9, 2], same[:2], same[:2], [0, 1.0], 0.6) == ([0], 1)
    assert speculative.verify([-1], [9], np.zeros((1, 3)), None, [0], 0.5) == ([0], -1)
