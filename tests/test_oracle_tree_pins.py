"""Pins of oracle/tree.py on CPU: closed forms and brute force."""
import itertools
import math

import numpy as np

import oracle
from oracle import tree as ot


def test_visible_keys_of_a_small_tree_by_hand():
    #     0
    #    / \
    #   1   2
    #   |   |
    #   3   4   and a second root 5
    par = [-1, 0, 0, 1, 2, -1]
    v = ot.visible(par, 6, 3, 0)
    assert v[:, :3].all()
    sees = [{0}, {0, 1}, {0, 2}, {0, 1, 3}, {0, 2, 4}, {5}]
    for i, s in enumerate(sees):
        assert set(np.flatnonzero(v[i, 3:])) == s
    # window 2: a node and the position before it
    v = ot.visible(par, 6, 3, 2)
    rows = [{2, 3}, {3, 4}, {3, 5}, {4, 6}, {5, 7}, {2, 8}]
    for i, s in enumerate(rows):
        assert set(np.flatnonzero(v[i])) == s
    assert (ot.visible(par, 6, 3, 1).sum(axis=1) == 1).all()


def test_a_chain_is_the_causal_block():
    import torch

    g = torch.Generator().manual_seed(3)
    T, Hq, Hkv, D, L = 5, 4, 2, 16, 40
    q = torch.randn((T, Hq, D), generator=g)
    k, v = (torch.randn((5, 8, Hkv, D), generator=g) for _ in range(2))
    oracle.build()
    for window in (0, 7):
        e_o, e_l = oracle.block_attn(q, k, v, torch.arange(5, dtype=torch.int32)[None], torch.tensor([L], dtype=torch.int32),
                                     T, causal=True, window=window, scale=0.25)
        o, l, spread, size = ot.tree_attn(q.double().numpy(), k.reshape(40, Hkv, D).double().numpy(),
                                          v.reshape(40, Hkv, D).double().numpy(), [-1, 0, 1, 2, 3], L - T, window, 0.25)
        np.testing.assert_allclose(o, np.asarray(e_o).reshape(T, Hq, D), rtol=1e-6, atol=1e-6)
        np.testing.assert_allclose(l, np.asarray(e_l).reshape(T, Hq), rtol=1e-6, atol=1e-6)
        assert (spread >= np.abs(o) - 1e-12).all() and (size > 0).all()


def test_equal_scores_average_the_visible_values():
    par = [-1, 0, 0]
    v = np.arange(5.0)[:, None, None] * np.ones((5, 1, 16))
    o, l, _, _ = ot.tree_attn(np.zeros((3, 1, 16)), np.ones((5, 1, 16)), v, par, 2, 0, 1.0)
    np.testing.assert_allclose(o[:, 0, 0], [(0 + 1 + 2) / 3, (0 + 1 + 2 + 3) / 4, (0 + 1 + 2 + 4) / 4])
    np.testing.assert_allclose(l[:, 0], np.log([3, 4, 4]))


def test_log_probabilities_closed_forms():
    x = np.array([[0.0, 0.0, 0.0, 0.0], [math.log(1), math.log(2), -np.inf, math.log(5)], [-np.inf] * 4])
    given, ent, z, top, top_lp = ot.token_logprobs(x, np.array([[3, -1], [2, 9], [0, 1]]), 3, 1.0)
    np.testing.assert_allclose(z, [math.log(4), math.log(8), -np.inf])
    np.testing.assert_allclose(ent[0], math.log(4))
    p = np.array([1, 2, 5]) / 8
    np.testing.assert_allclose(ent[1], -(p * np.log(p)).sum())
    assert ent[2] == 0
    np.testing.assert_allclose(given, [[-math.log(4), -np.inf], [-np.inf] * 2, [-np.inf] * 2])
    assert top.tolist() == [[0, 1, 2], [3, 1, 0], [0, 1, 2]]
    np.testing.assert_allclose(top_lp[1], np.log([5 / 8, 2 / 8, 1 / 8]))
    # temperature 2 halves the logits
    _, _, z2, _, _ = ot.token_logprobs(x[1:2], None, 0, 2.0)
    np.testing.assert_allclose(z2[0], math.log(1 + math.sqrt(2) + math.sqrt(5)))


def test_acceptance_against_every_token_pattern_of_a_tiny_tree():
    par = np.array([[-1, 0, 0, 1, 1, 2]])
    best = [1, 0, 1, 0, 1, 0]
    logits = np.zeros((1, 6, 2))
    for i, t in enumerate(best):
        logits[0, i, t] = 1.0
    for toks in itertools.product((0, 1), repeat=6):
        acc, path, nxt, arg = ot.tree_accept(logits, np.array([toks]), par, [6])
        # every root path that agrees, the greedy choice of the smallest child at each step
        want = [0]
        if toks[1] == 1:
            want.append(1)
            want += [3] if toks[3] == 0 else [4] if toks[4] == 0 else []
        elif toks[2] == 1:
            want.append(2)
            want += [5] if toks[5] == 1 else []
        assert path[0, :len(want)].tolist() == want and (path[0, len(want):] == -1).all()
        assert acc[0] == len(want) - 1 and nxt[0] == best[want[-1]] and arg[0].tolist() == best


def test_moves_against_a_list():
    rng = np.random.default_rng(0)
    cache = rng.normal(size=(2, 6, 4, 1, 2))
    table = np.array([[4, 1, 3]])
    flat = [cache[:, table[0, j // 4], j % 4] for j in range(12)]
    new, lens = ot.tree_commit(cache, table, [11], np.array([[0, 2, 3, 5, -1, -1]]), [3], [6])
    assert lens[0] == 5 + 4
    want = list(flat)
    want[6], want[7], want[8] = flat[7], flat[8], flat[10]
    for j in range(12):
        np.testing.assert_array_equal(new[:, table[0, j // 4], j % 4], want[j])
    # pages of nobody stay
    for pg in (0, 2, 5):
        np.testing.assert_array_equal(new[:, pg], cache[:, pg])
