"""Chunk attention over long runs of key tiles: enough work that every CTA pair
walks many tiles within a row tile and several row tiles one after another (the
smaller shapes are split so finely that a pair has one tile of each). Against
the definition in 64 bits, every row."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

from oracle.sfa import bf16_bits_to_f64, round_to_bf16_bits  # noqa: E402
from test_chunk_plan import KEYS, key_end, key_tiles, ROWS  # noqa: E402
from test_gpu_paged import BF16_HALF_STEP, FORMATS, Chunk, random_rows, score_error  # noqa: E402

SCALE = 1 / 24


@pytest.fixture(scope="module")
def d():
    import decode_dsa_kv_gb300 as mod
    return mod


def runs(reqs, H):
    """The key tiles of every segment (row tile, stretch) on a GPU of 76 pairs."""
    line = [(b, j) for b, (n, c) in enumerate(reqs) for j in range(-(-n * H // ROWS))
            for _ in range(key_tiles(key_end(n, c, H, True, j)))]
    out = []
    for p in range(76):
        share, more = divmod(len(line), 76)
        lo = share * p + min(p, more)
        mine = line[lo:lo + share + (p < more)]
        out.append([mine.count(x) for x in dict.fromkeys(mine)])
    return out


def check(c, out, lse):
    """Every row of a Chunk against 64 bits, computed on the GPU."""
    assert c.kv.synchronize() == 0
    at = 0
    for b, (n, ctx) in enumerate(c.reqs):
        K = torch.from_numpy(c.K[b]).cuda()
        V = K[:, :512]
        for i in range(0, n, 16):
            k = min(n, i + 16)
            q = torch.from_numpy(c.q64[at + i:at + k]).cuda().flatten(0, 1)
            limit = ctx - n + torch.arange(i, k, device="cuda").repeat_interleave(c.H) + 1
            hidden = torch.arange(ctx, device="cuda")[None] >= limit[:, None]
            s = (SCALE * (q @ K.T)).masked_fill_(hidden, -torch.inf)
            z = torch.logsumexp(s, 1)
            p = torch.exp(s - z[:, None])
            o, mean_abs = p @ V, p @ V.abs()
            size = SCALE * (q.abs() @ K.abs().T).masked_fill_(hidden, 0).amax(1)
            # A weight: its score's error and its rounding to bf16; the sum of
            # the weights no more. O and the sums grow by one product's keys (16)
            # at a time, each addition off by at most 2^-22 of what is there; a
            # maximum that moves scales them (2^-22 for the power, 2^-24 for the
            # product; at most one a tile); merging is a few additions more.
            grow = (ctx / 16 + 2 * ctx / KEYS + 16) * 2.0 ** -22
            e = (BF16_HALF_STEP + 2 * score_error(size) + grow)[:, None]
            bound = e * (mean_abs + o.abs()) + 1.01 * BF16_HALF_STEP * o.abs() + 2.0 ** -130
            got = out[at + i:at + k].double().flatten(0, 1)
            worst = ((got - o).abs() / bound).max().item()
            assert worst <= 1, (b, i, worst)
            tol = 2 * score_error(size) + grow + 2.0 ** -20 + 2.0 ** -22 * z.abs()
            assert torch.all((lse[at + i:at + k].double().flatten() - z).abs() <= tol), (b, i)
        at += n


# Levels of the scores, in powers of two, through the rope part (bf16 in both
# formats; the queries' is all ones, so a key of x adds 64 x / 24 to every score).
JUMP = 2.375                                 # 2^9.1: the running maximum has to follow


def levelled(order):
    """4000 keys in 16 tiles. Rising: odd tiles up to 13 hold 256 keys of one
    level, even ones a single key 2^9 above it (and 255 at it): the maximum moves
    in every second tile, and what came before is always a third of the sum.
    Falling: the same keys from the last to the first."""
    def rows(rng, c):
        x = bf16_bits_to_f64(random_rows(rng, c, 0.3))
        pos = np.arange(c)
        t = pos // KEYS
        level = JUMP * np.minimum(t // 2, 6.0)
        level[(t % 2 == 0) & (t > 0)] -= JUMP
        level[t == 14] = level[t == 15] = JUMP * 6
        spike = (t % 2 == 0) & (t > 0) & (pos % KEYS == 100)
        level[spike] = JUMP * (t[spike] // 2)
        x[:, 512:] = level[:, None]
        return round_to_bf16_bits(x if order == "rising" else x[::-1])
    return rows


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("order", ["rising", "falling"])
def test_running_maximum_moves_within_a_segment(d, fmt, order):
    reqs = [(256, 4000)]
    longest = max(max(r) for r in runs(reqs, 128))
    assert longest == 16 and min(len(r) for r in runs(reqs, 128)) >= 3
    c = Chunk(d, fmt, 64, 128, reqs, seed=30, rows=levelled(order))
    c.q[..., 512:] = 1
    c.q64[..., 512:] = 1
    if order == "rising":
        # the case is what it is made for: from tile to tile the largest score
        # grows by more than 2^8, and what came before still counts
        s = SCALE * (c.q64[0] @ c.K[0][:3745].T) / np.log(2)
        before, spike = s[:, :14 * KEYS], s[:, 14 * KEYS + 100]
        assert np.mean(spike - before[:, :13 * KEYS].max(1) > 8) > 0.8
        old = np.exp2(before - spike[:, None]).sum(1)
        assert np.median(old / (old + 1)) > 0.25
    check(c, *c.run())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("H, reqs", [
    (128, [(256, 4000)]),
    (128, [(200, 4000), (1, 9000), (40, 3000)]),    # a single token's 36 tiles in one segment
    (130, [(150, 2600), (37, 1999)]),               # row tiles of two tokens
])
def test_many_tiles_a_segment(d, fmt, H, reqs):
    assert max(max(r) for r in runs(reqs, H)) >= 11
    c = Chunk(d, fmt, 32, H, reqs, seed=31)
    first = [x.clone() for x in c.run()]
    check(c, *first)
    out, lse = c.run()
    assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
