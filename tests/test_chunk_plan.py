"""CPU restatement of how sfa_mla_chunk splits its work: the closed form of the
units before a row tile against a count, and the pairs' stretches: every unit
of every request in exactly one segment, in order, at most two cut row tiles
for a pair, every cut one beginning in one pair and ending in a later one."""
import random

import pytest

ROWS, KEYS = 128, 256


def key_end(n, ctx, H, causal, j):
    if not causal:
        return ctx
    last = min(n * H - 1, j * ROWS + ROWS - 1)
    return max(0, ctx - n + last // H + 1)


def key_tiles(end):
    return max(1, -(-end // KEYS))


def units_before(n, ctx, H, causal, j):
    if not causal:
        return j * key_tiles(ctx)
    tiles = -(-n * H // ROWS)
    G, c = 2 * H, ((ctx - n) * H + ROWS - 1) >> 7

    def below(N):
        if N <= 0:
            return 0
        k = N // G
        return G * (k * (k - 1) // 2) + k * (N - k * G)

    m = min(j, tiles - 1)
    s = m + below(m + c) - below(c)
    if j == tiles:
        s += key_tiles(key_end(n, ctx, H, causal, tiles - 1))
    return s


def requests(rng, H):
    out = []
    for _ in range(rng.randint(1, 12)):
        n = rng.choice([0, 1, 1, 2, 5, rng.randint(1, 900)])
        ctx = rng.choice([0, n, n + rng.randint(0, 5000), rng.randint(0, 3000)])
        out.append((n, ctx))
    return out


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("H", [1, 5, 16, 64, 128, 130, 1024])
def test_closed_form(H, causal):
    rng = random.Random(H)
    for _ in range(60):
        for n, ctx in requests(rng, H):
            tiles, s = -(-n * H // ROWS), 0
            for j in range(tiles):
                assert units_before(n, ctx, H, causal, j) == s
                s += key_tiles(key_end(n, ctx, H, causal, j))
            if tiles:
                assert units_before(n, ctx, H, causal, tiles) == s


@pytest.mark.parametrize("pairs", [1, 2, 7, 76])
def test_stretches_cover_every_unit_once(pairs):
    rng = random.Random(pairs)
    for _ in range(80):
        H, causal = rng.choice([1, 16, 20, 128]), rng.random() < 0.7
        reqs = [(min(n, 60), ctx) for n, ctx in requests(rng, H)]
        line = [(b, j, t) for b, (n, ctx) in enumerate(reqs) for j in range(-(-n * H // ROWS))
                for t in range(key_tiles(key_end(n, ctx, H, causal, j)))]
        total, got, cut = len(line), [], []
        P = min(pairs, total)
        for p in range(P):
            share, more = divmod(total, P)
            lo = share * p + min(p, more)
            hi = lo + share + (p < more)
            assert hi > lo
            segments = {}
            for b, j, t in line[lo:hi]:
                segments.setdefault((b, j), []).append(t)
            got += line[lo:hi]
            slots = []
            for (b, j), ts in segments.items():
                assert ts == list(range(ts[0], ts[-1] + 1))
                units = key_tiles(key_end(*reqs[b], H, causal, j))
                starts, ends = ts[0] == 0, ts[-1] == units - 1
                if not (starts and ends):
                    slots.append(1 if starts else 0)
                    cut.append((b, j, p, starts, ends))
            assert len(set(slots)) == len(slots)          # one workspace slot for each
        assert got == line
        for b, j in {(c[0], c[1]) for c in cut}:
            chain = [c for c in cut if c[:2] == (b, j)]
            ps = [c[2] for c in chain]
            assert ps == list(range(ps[0], ps[-1] + 1)) and len(ps) > 1
            assert [c[3] for c in chain] == [True] + [False] * (len(ps) - 1)
            assert [c[4] for c in chain] == [False] * (len(ps) - 1) + [True]
