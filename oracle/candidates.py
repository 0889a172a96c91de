"""Several continuations of a context over the paged cache: drafted trees and
beams.

A tree's n nodes are a request's newest tokens, the last n of its ctx positions;
node i has a parent of a lower number, or -1 (it follows the cached context):

    position of node i  = ctx - n + (number of its ancestors)
    node i sees         the ctx - n cached positions, its ancestors and itself

The rope pairs (a, b) of a row at position p are turned by p * freq_i:
(a cos - b sin, a sin + b cos); pair i is (2 i, 2 i + 1), or (i, i + 32).

Verification of a tree whose drafts were chosen, not sampled: from the root on,
a token t is drawn from the target's distribution after the node (the first t
whose running sum exceeds u times the sum, in whole multiples of 2^-60; without
u the largest value, the lowest token of it); the first child that holds t is
the next node. The tokens that come out are the target's own samples.

Beams: s(k, t) = cum_k + x_kt - log sum exp x_k; the n largest, ties to the
lower beam, then the lower token. Values of NaN and +infinity count as
-infinity, and what scores -infinity is never chosen.
"""
import math

import numpy as np

D_LATENT = 512


def depths(parent) -> list:
    out = []
    for i, p in enumerate(parent):
        assert -1 <= p < i
        out.append(0 if p < 0 else out[p] + 1)
    return out


def sees(parent) -> np.ndarray:
    """Boolean [n][n]: whether node i sees node j."""
    n = len(parent)
    out = np.eye(n, dtype=bool)
    for i, p in enumerate(parent):
        if p >= 0:
            out[i] |= out[p]
    return out


def mask_words(seen: np.ndarray, words: int) -> np.ndarray:
    """Rows of booleans as uint32 [n][words]: bit j % 32 of word j / 32."""
    n, m = seen.shape
    out = np.zeros((n, words), dtype=np.uint32)
    for j in range(min(m, 32 * words)):
        out[:, j // 32] |= np.where(seen[:, j], np.uint32(1 << (j % 32)), np.uint32(0))
    return out


def turn(x: np.ndarray, pos: int, freq: np.ndarray, interleaved: bool) -> np.ndarray:
    """Float64 rope parts [..][64] of position pos, turned. The angle is reduced by
    whole turns in exact integers."""
    from fractions import Fraction
    two_pi = Fraction(884279719003555, 140737488355328)  # the double; its error below
    low = 2.4492935982947064e-16                         # 2 pi = two_pi + low
    angle = []
    for f in freq:
        a = Fraction(float(f)) * int(pos)
        turns = math.floor(a / two_pi)
        angle.append(float(a - turns * two_pi) - turns * low)
    c, s = np.cos(angle), np.sin(angle)
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :32], x[..., 32:])
    y = np.empty_like(x)
    if interleaved:
        y[..., 0::2], y[..., 1::2] = a * c - b * s, a * s + b * c
    else:
        y[..., :32], y[..., 32:] = a * c - b * s, a * s + b * c
    return y


def tree_attention(q: np.ndarray, K: np.ndarray, seen: np.ndarray, scale: float):
    """q float64 [n][H][576], K float64 [ctx][576], seen boolean [n][n] of the last
    n positions -> out [n][H][512], lse [n][H], and, for error bounds, the weighted
    mean of |V| and the largest scale * sum |q||k|."""
    n, H, _ = q.shape
    out, mean_abs = np.zeros((n, H, D_LATENT)), np.zeros((n, H, D_LATENT))
    lse, size = np.full((n, H), -np.inf), np.zeros((n, H))
    ctx = len(K)
    for i in range(n):
        rows = np.concatenate([np.ones(ctx - n, dtype=bool), seen[i]])
        k = K[rows]
        if len(k) == 0:
            continue
        s = scale * (q[i] @ k.T)
        m = s.max(axis=1, keepdims=True)
        p = np.exp(s - m)
        z = p.sum(axis=1, keepdims=True)
        out[i] = (p @ k[:, :D_LATENT]) / z
        mean_abs[i] = (p @ np.abs(k[:, :D_LATENT])) / z
        lse[i] = (m + np.log(z))[:, 0]
        size[i] = abs(scale) * (np.abs(q[i]) @ np.abs(k).T).max(axis=1)
    return out, lse, mean_abs, size


def draw(p, u) -> int:
    """The token of a row of probabilities for u (None: its largest value), or -1."""
    p = np.asarray(p, dtype=np.float64)
    if u is None:
        if np.all(np.isnan(p)):
            return -1
        return int(np.nanargmax(np.where(np.isnan(p), np.nan, p)))
    w = [int(math.ldexp(v, 60)) if 0 <= v < 2 else 0 for v in p]
    total = sum(w)
    if not 0 < total < 2 ** 64 - 1:
        return -1
    point = int(math.ldexp(float(u), 64)) * total >> 64
    run = 0
    for t, v in enumerate(w):
        run += v
        if run > point:
            return t
    raise AssertionError


def verify_tree(tokens, parent, target, u, depth: int):
    """One request's tree: tokens, parent [n], target [n][V], u [depth + 1] or None
    -> (path [depth + 1], next [depth + 1], accepted)."""
    n = len(parent)
    if n == 0:
        return [-1] * (depth + 1), [-1] * (depth + 1), -1
    path, out = [0], []
    while True:
        t = draw(target[path[-1]], None if u is None else u[len(out)])
        out.append(t)
        child = [i for i in range(path[-1] + 1, n) if parent[i] == path[-1] and tokens[i] == t]
        if t < 0 or not child or len(path) > depth:
            break
        path.append(child[0])
    a = len(path) - 1
    return path + [-1] * (depth - a), out + [-1] * (depth - a), a


def keep_rows(rows, path, accepted: int):
    """A request's new rows (in their order) after the accepted path's have moved to
    the front."""
    out = list(rows)
    for i in range(accepted + 1):
        out[i] = rows[path[i]]
    return out


def beam_scores(logits: np.ndarray, cum: np.ndarray) -> np.ndarray:
    """s [K][V] of one request, float64."""
    x = np.asarray(logits, dtype=np.float64)
    x = np.where(x < np.inf, x, -np.inf)
    c = np.asarray(cum, dtype=np.float64)
    c = np.where(c < np.inf, c, -np.inf)
    out = np.full(x.shape, -np.inf)
    for k in range(x.shape[0]):
        m = x[k].max()
        if m > -np.inf and c[k] > -np.inf:
            out[k] = c[k] + ((x[k] - m) - math.log(np.exp(x[k] - m).sum()))
    return out


def beam_select(logits: np.ndarray, cum: np.ndarray, n: int):
    """One request: (tokens [n], parents [n], scores [n])."""
    s = beam_scores(logits, cum)
    K, V = s.shape
    order = np.argsort(-s.reshape(-1), kind="stable")[:n]
    tokens, parents, scores = [], [], []
    for i in order:
        if s.reshape(-1)[i] > -np.inf:
            tokens.append(int(i % V))
            parents.append(int(i // V))
            scores.append(float(s.reshape(-1)[i]))
    rest = n - len(tokens)
    return tokens + [-1] * rest, parents + [-1] * rest, scores + [-np.inf] * rest


def fork(table, ctx, parent: int, spare: int, page: int, width: int):
    """A new sequence's table row, its length, and the page that its partial last
    page is copied from (None: nothing is copied) -> (row, length, source, rows)."""
    if parent < 0:
        return [-1] * width, 0, None, 0
    old, length = list(table[parent]), int(ctx[parent])
    w, rows = length // page, length % page
    row = old[:w] + ([spare] if w < width else []) + [-1] * (width - w - 1)
    return row[:width], length, old[w] if rows else None, rows
