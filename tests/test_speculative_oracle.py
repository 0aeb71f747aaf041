"""Pins of the speculative step's oracle: hand values, closed forms and a distribution that has to come out."""
import math

import numpy as np

from oracle import speculative as sp


def test_rotation_by_hand():
    x = np.zeros((1, 1, 128), np.float32)
    x[0, 0, 0], x[0, 0, 64] = 3.0, 4.0
    y = sp.qk_norm_rope(x, [1])                       # pair 0 turns by one radian
    assert math.isclose(y[0, 0, 0], 3 * math.cos(1) - 4 * math.sin(1))
    assert math.isclose(y[0, 0, 64], 4 * math.cos(1) + 3 * math.sin(1))
    x = np.zeros((1, 1, 128), np.float32)
    x[0, 0, 2], x[0, 0, 3], x[0, 0, 40] = 1.0, 2.0, 7.0
    y = sp.qk_norm_rope(x, [5], rot=4, theta=100.0, interleaved=True)   # pair 1 of two: 5 * 100^(-1/2)
    assert math.isclose(y[0, 0, 2], math.cos(0.5) - 2 * math.sin(0.5))
    assert math.isclose(y[0, 0, 3], 2 * math.cos(0.5) + math.sin(0.5))
    assert y[0, 0, 40] == 7.0


def test_norm_gives_unit_mean_square():
    x = np.random.default_rng(1).standard_normal((2, 3, 128)).astype(np.float32) * 5
    y = sp.qk_norm_rope(x, [7, 9], eps=0.0, norm=True)
    np.testing.assert_allclose((y * y).mean(-1), 1.0, rtol=1e-12)   # the rotation keeps lengths


def test_scores_depend_on_the_distance_alone():
    rng = np.random.default_rng(2)
    q, k = rng.standard_normal((2, 1, 1, 128)).astype(np.float32)
    dots = [(sp.qk_norm_rope(q, [a]) * sp.qk_norm_rope(k, [a - 11])).sum() for a in (11, 500, 100000)]
    np.testing.assert_allclose(dots, dots[0], rtol=1e-9)


def test_write_keeps_the_last_token_of_a_slot():
    rng = np.random.default_rng(3)
    k = rng.standard_normal((300, 1, 128)).astype(np.float32)
    cache = [np.zeros((1, 1, 128, 128), np.int8), np.zeros((1, 1, 128), np.float32),
             np.zeros((1, 1, 128, 128), np.int8), np.zeros((1, 1, 128), np.float32)]
    sp.kv_write(cache, k, k, [300], [5], n_max=300, wrap=True)
    got = sp.values(cache[0], cache[1])[0, 0]
    for slot in range(128):
        i = max(i for i in range(300) if (5 + i) % 128 == slot)
        assert np.abs(got[slot] - k[i, 0]).max() <= np.abs(k[i]).max() / 127 * 0.5001


def test_tree_of_one_node_sees_reference_window_and_itself():
    B, hk = 1, 1
    z = lambda cap: np.zeros((B, hk, cap, 128))  # noqa: E731
    ref, ring = (z(4), z(4)), (z(128), z(128))
    ref[1][0, 0, :, 0], ring[1][0, 0, :, 0] = 1.0, 2.0
    v = np.zeros((1, 1, 1, 128), np.float32)
    v[..., 0] = 5.0
    q = np.zeros((1, 1, 1, 128), np.float32)     # a zero query averages what it sees
    for n, seen in ((0, 0), (3, 3), (127, 127), (128, 127), (5000, 127)):
        out = sp.rswa_tree(q, q, v, ref, [3], ring, [n])
        assert math.isclose(out[0, 0, 0, 0], (3 * 1 + 2 * seen + 5) / (3 + seen + 1))


def test_tree_nodes_see_their_line_and_a_window_that_moves_with_depth():
    z = np.zeros((1, 1, 128, 128))
    ring = (z, z.copy())
    ring[1][0, 0, :, 1] = np.arange(128)          # token p of 128 committed ones has value p
    k = np.zeros((1, 4, 1, 128), np.float32)
    v = k.copy()
    v[0, :, 0, 0] = [1, 10, 100, 1000]
    out = sp.rswa_tree(k, k, v, (z, z), [0], ring, [128], parent=[[-1, 0, 0, 2]])
    for node, line, depth in ((0, [0], 0), (1, [0, 1], 1), (2, [0, 2], 1), (3, [0, 2, 3], 2)):
        toks = range(1 + depth, 128)              # position 128 + depth, 128 tokens with itself
        count = len(toks) + len(line)
        assert count == 128
        assert math.isclose(out[0, node, 0, 0], sum(10 ** j for j in line) / count)
        assert math.isclose(out[0, node, 0, 1], sum(toks) / count)


def test_verification_keeps_the_targets_distribution():
    # two siblings drawn from q, then the residual: the first emitted token must be distributed as p
    rng = np.random.default_rng(4)
    p, q = np.array([0.5, 0.3, 0.2, 0.0]), np.array([0.1, 0.2, 0.3, 0.4])
    T = 40000
    tokens = rng.choice(4, size=(T, 2), p=q).astype(np.int32)
    target = np.broadcast_to(p.astype(np.float32), (T, 3, 4))
    draft = np.broadcast_to(q.astype(np.float32), (T, 2, 4))
    n, path, nxt = sp.spec_verify(target, draft, tokens, np.tile([[-1, -1]], (T, 1)), None, rng.random((T, 3), np.float32))
    first = np.where(n > 0, tokens[np.arange(T), np.maximum(path[:, 0], 0)], nxt)
    freq = np.bincount(first, minlength=4) / T
    assert np.abs(freq - p).max() < 5 * math.sqrt(0.25 / T)
    # without draft probabilities (chosen drafts)
    n, path, nxt = sp.spec_verify(target, None, np.tile(np.array([[2, 0]], np.int32), (T, 1)), np.tile([[-1, -1]], (T, 1)),
                                  None, rng.random((T, 3), np.float32))
    first = np.where(n > 0, np.array([2, 0])[np.maximum(path[:, 0], 0)], nxt)
    assert np.abs(np.bincount(first, minlength=4) / T - p).max() < 5 * math.sqrt(0.25 / T)


def test_probabilities_sum_to_one_and_follow_the_temperature():
    p = sp.token_probs(np.array([[0.0, math.log(2.0)]]), 0.5)
    np.testing.assert_allclose(p, [[0.2, 0.8]], rtol=1e-12)
