"""The oracle of trees and beams, pinned: masks and depths by walking up, the
rotation by complex numbers and its group law, tree attention by chains and by
each path alone, the tree's walk by the target's own distribution, beams by full
enumeration, forks by the rows that a sequence reads afterwards."""
import cmath
import itertools
import math

import numpy as np
import pytest

from oracle import candidates as c
from oracle import paged


def random_tree(rng, n, roots=1):
    return [-1 if i < roots else int(rng.integers(0, i)) for i in range(n)]


def test_depths_and_masks_are_the_walk_up():
    rng = np.random.default_rng(0)
    for n in (1, 2, 33, 70):
        parent = random_tree(rng, n, roots=2 if n > 2 else 1)
        seen, depth = c.sees(parent), c.depths(parent)
        words = c.mask_words(seen, 3)
        for i in range(n):
            up, x = [], i
            while x >= 0:
                up.append(x)
                x = parent[x]
            assert sorted(up) == list(np.flatnonzero(seen[i])) and depth[i] == len(up) - 1
            assert sum(int(w) << (32 * k) for k, w in enumerate(words[i])) == sum(1 << j for j in up)
    assert c.mask_words(np.ones((1, 40), bool), 1)[0, 0] == 0xffffffff


@pytest.mark.parametrize("interleaved", [True, False])
def test_turn_is_a_complex_product(interleaved):
    rng = np.random.default_rng(1)
    x = rng.normal(size=64)
    freq = 10000.0 ** (-np.arange(32) / 32)
    for pos in (0, 1, 7, 5000, -3):
        y = c.turn(x, pos, freq, interleaved)
        for i in range(32):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + 32)
            z = complex(x[a], x[b]) * cmath.exp(1j * pos * freq[i])
            assert abs(complex(y[a], y[b]) - z) < 1e-11
    # two turns are one by the sum, far out too, and lengths stay
    far = 2 ** 27 - 1
    y = c.turn(c.turn(x, far, freq, interleaved), -far + 5, freq, interleaved)
    assert np.allclose(y, c.turn(x, 5, freq, interleaved), rtol=0, atol=1e-11)
    assert np.isclose(np.sum(y * y), np.sum(x * x))


def test_tree_attention_of_a_chain_is_causal_and_of_a_path_is_its_own():
    rng = np.random.default_rng(2)
    K, q = rng.normal(size=(20, 576)), rng.normal(size=(6, 2, 576))
    chain = c.sees([-1, 0, 1, 2, 3, 4])
    for got, want in zip(c.tree_attention(q, K, chain, 0.05),
                         paged.chunk_attention(q, K, 20, True, 0.05)):
        assert np.allclose(got, want, rtol=1e-12)
    parent = [-1, 0, 0, 1, 2, 4]
    out, lse, _, _ = c.tree_attention(q, K, c.sees(parent), 0.05)
    for i in range(6):
        up, x = [], i
        while x >= 0:
            up.insert(0, x)
            x = parent[x]
        rows = np.concatenate([K[:14], K[14:][up]])
        o, z, _, _ = paged.chunk_attention(q[i:i + 1], rows, len(rows), True, 0.05)
        assert np.allclose(out[i], o[0], rtol=1e-12) and np.allclose(lse[i], z[0])
    out, lse, _, _ = c.tree_attention(q[:2], K[:2], np.zeros((2, 2), bool), 0.05)
    assert np.all(out == 0) and np.all(np.isneginf(lse))


def test_verified_tokens_follow_the_target():
    # over a grid of uniform numbers the first two tokens have the target's
    # probabilities, whatever the drafts are
    V, grid = 4, 40
    rng = np.random.default_rng(3)
    target = np.round(rng.dirichlet(np.ones(V), 6) * grid) / grid
    target[:, -1] = 1 - target[:, :-1].sum(1)
    target[0] = [0.25, 0.25, 0.25, 0.25]
    parent, tokens = [-1, 0, 0, 1, 1, 2], [9, 2, 0, 1, 3, 2]
    seen = np.zeros((V, V))
    for a, b in itertools.product(range(grid), repeat=2):
        u = [(a + 0.5) / grid, (b + 0.5) / grid, 0.5]
        path, out, n = c.verify_tree(tokens, parent, target, u, 2)
        assert path[:n + 1] == [0] + path[1:n + 1] and out[n] >= 0
        for k in range(n):
            assert parent[path[k + 1]] == path[k] and tokens[path[k + 1]] == out[k]
        if n >= 1:
            seen[out[0], out[1]] += 1 / grid ** 2
    for k, t in ((1, 2), (2, 0)):  # the drafted first tokens
        assert np.allclose(seen[t], target[0, t] * target[k], atol=1e-12)


def test_draw_matches_float_sums_and_the_largest_value():
    rng = np.random.default_rng(4)
    for _ in range(200):
        p = rng.dirichlet(np.ones(7)).astype(np.float32)
        u = np.float32(rng.random())
        run = np.cumsum(p.astype(np.float64))
        assert c.draw(p, u) == int(np.searchsorted(run, float(u) * run[-1], side="right"))
    assert c.draw([0, 0.5, 0, 0.5], 0.0) == 1 and c.draw([0.5, 0.5, 0], 0.99999) == 1
    assert c.draw([0.0, 0.0], 0.3) == -1 and c.draw([1.9] * 9, 0.5) == -1
    assert c.draw([math.nan, -1, 0.5, 2.5, 0.5], 0.6) == 4     # bad ones count as 0
    assert c.draw([1, 3, 3, math.nan], None) == 1 and c.draw([math.nan] * 2, None) == -1
    assert c.draw([-math.inf, -math.inf], None) == 0


def test_walk_ends():
    target = np.eye(3)[[1, 1, 1, 1]]
    assert c.verify_tree([0, 1, 1, 1], [-1, 0, 0, 1], target, None, 5) == ([0, 1, 3, -1, -1, -1],
                                                                         [1, 1, 1, -1, -1, -1], 2)
    assert c.verify_tree([0, 1, 1, 1], [-1, 0, 0, 1], target, None, 1) == ([0, 1], [1, 1], 1)
    assert c.verify_tree([0, 1], [-1, 0], target[:2], [0.5], 0) == ([0], [1], 0)
    assert c.verify_tree([], [], target[:0], [0.5, 0.5], 1) == ([-1, -1], [-1, -1], -1)
    assert c.verify_tree([0, 1], [-1, -1], target[:2], None, 1)[2] == 0   # another root is no child


def test_keep_rows_moves_the_path():
    assert c.keep_rows(list("abcdef"), [0, 2, 5], 2) == ["a", "c", "f", "d", "e", "f"]
    assert c.keep_rows(list("abc"), [0, -1], 0) == list("abc") and c.keep_rows([], [-1], -1) == []


def test_beams_by_enumeration():
    rng = np.random.default_rng(5)
    x, cum = rng.normal(0, 2, (3, 5)), np.array([-1.0, -0.5, -np.inf])
    x[0, 3] = -np.inf
    want = []
    for k, t in itertools.product(range(2), range(5)):
        p = np.exp(x[k, t]) / np.exp(x[k]).sum()
        if p > 0:
            want.append((cum[k] + math.log(p), -k, -t))
    want.sort(reverse=True)
    tokens, parents, scores = c.beam_select(x, cum, 11)
    assert tokens == [-t for _, _, t in want] + [-1] * 2
    assert parents == [-k for _, k, _ in want] + [-1] * 2
    assert np.allclose(scores[:9], [s for s, _, _ in want]) and scores[9:] == [-np.inf] * 2
    # ties: the lower beam, then the lower token
    tokens, parents, _ = c.beam_select(np.zeros((2, 3)), np.zeros(2), 4)
    assert (tokens, parents) == ([0, 1, 2, 0], [0, 0, 0, 1])
    bad = np.array([[math.nan, 1.0, math.inf, 0.0]])
    assert c.beam_select(bad, [0.0], 3)[0] == [1, 3, -1]
    assert math.isclose(c.beam_select(bad, [0.0], 1)[2][0], -math.log(1 + math.exp(-1)))


@pytest.mark.parametrize("length", [0, 1, 15, 16, 17, 32, 48])
def test_fork_reads_the_parents_rows(length):
    page, width = 16, 3
    rows = {(p, r): (p, r) for p in range(8) for r in range(page)}
    table, ctx = [[9, 9, 9], [4, 2, 6]], [1, length]
    row, n, source, copied = c.fork(table, ctx, 1, 7, page, width)
    assert n == length and copied == length % page and len(row) == width
    if source is not None:
        for r in range(copied):
            rows[7, r] = rows[source, r]
    for t in range(length):
        assert rows[row[t // page], t % page] == (table[1][t // page], t % page)
    if length < page * width:
        assert row[length // page] == 7          # where the next row goes
    assert c.fork(table, ctx, -1, 7, page, width) == ([-1] * 3, 0, None, 0)
