"""Draft verification at the edge of its contract: weights that add up to 16 or
more, and bad probabilities in rows of many tiles and blocks. Outputs are
filled before each call: every one of them has to be written."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

import oracle  # noqa: E402

LEFT = 77


def verify(drafts, p, q, u, n_draft=None):
    """(tokens, accepted, error bits) as lists, through the C ABI."""
    import decode_dsa_kv_gb300 as d
    B, n = drafts.shape
    dev = [None if t is None else torch.from_numpy(np.ascontiguousarray(t)).cuda()
           for t in (drafts, n_draft, p, q, u)]
    tokens = torch.full((B, n + 1), LEFT, dtype=torch.int32, device="cuda")
    accepted = torch.full((B,), LEFT, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    V = p.shape[2]
    d.check(d.ts_verify_drafts(dev[0], dev[1], dev[2], V, dev[3], V, dev[4], B, n, V, tokens,
                               accepted, err))
    return tokens.tolist(), accepted.tolist(), d.ts_read_error(err)


def uniform(rng, B, n):
    return rng.random((B, n + 1)).astype(np.float32)


def small(rng, shape, V):
    """Weights that add up to about a half."""
    return (rng.random((*shape, V)) / V).astype(np.float32)


# V: one tile; two tiles; many tiles of several blocks
@pytest.mark.parametrize("V", [40, 5000, 100_001])
@pytest.mark.parametrize("total", [16, 17, 32, 33.5, 48])
def test_a_row_that_adds_up_to_16_or_more_has_no_next_token(V, total):
    import decode_dsa_kv_gb300 as d
    rng = np.random.default_rng(V)
    B = 4
    p = small(rng, (B, 1), V)
    at = np.linspace(0, V - 1, 34).astype(int)
    p[1, 0] = 0
    p[1, 0, at] = total / 34                      # spread over the row
    p[2, 0] = 0
    p[2, 0, :34] = total / 34                     # all in its first tile
    p[3, 0] = 0
    p[3, 0, at] = 15.5 / 34                       # a large row that is allowed
    exact = [sum(int(math.ldexp(float(x), 60)) for x in r[0]) for r in p]
    u = uniform(rng, B, 0)
    drafts = np.zeros((B, 0), dtype=np.int32)
    tokens, accepted, bits = verify(drafts, p, None, u)
    assert bits == d._abi.TS_DEVERR_PROB
    assert accepted == [0] * B
    for b in range(B):
        want, _ = oracle.verify_drafts(drafts[b], 0, p[b], None, u[b])
        assert tokens[b] == want, b
        assert (tokens[b] == [-1]) == (exact[b] >= 2 ** 64 - 1)
    assert tokens[1] == tokens[2] == [-1]


@pytest.mark.parametrize("V", [40, 100_001])
def test_a_residual_or_a_row_after_drafts_that_adds_up_to_16_or_more(V):
    import decode_dsa_kv_gb300 as d
    rng = np.random.default_rng(V)
    B, n = 3, 2
    p, q = small(rng, (B, n + 1), V), small(rng, (B, n), V)
    x = np.full((B, n), 3, dtype=np.int32)
    p[:, :n, 3], q[:, :, 3] = 0.5, 0.25           # accepted, at any u
    p[0, 1], p[0, 1, 3] = 18 / V if V > 9 else 0, 0.0
    q[0, 1] = 0.5 / V                             # request 0: a residual of 17.5 and more
    q[0, 1, 3] = 0.25
    p[1, 2] = 20 / V                              # request 1: the row after its drafts
    u = uniform(rng, B, n)
    tokens, accepted, bits = verify(x, p, q, u)
    assert bits == d._abi.TS_DEVERR_PROB
    assert accepted == [1, 2, 2]
    assert tokens[0] == [3, -1, -1] and tokens[1] == [3, 3, -1]
    for b in range(B):
        want, a = oracle.verify_drafts(x[b], n, p[b], q[b], u[b])
        assert tokens[b] == want and accepted[b] == a, b


@pytest.mark.parametrize("V", [5000, 100_001])
@pytest.mark.parametrize("bad", [math.nan, -0.25, 2.0, math.inf, -math.inf])
def test_bad_probabilities_in_rows_of_many_tiles(V, bad):
    # they count as 0 in the target's row and in the draft's; the rest is exact
    import decode_dsa_kv_gb300 as d
    rng = np.random.default_rng(V)
    B, n = 3, 1
    for where in ("target", "draft", "last"):
        p, q = 2 * small(rng, (B, n + 1), V), 2 * small(rng, (B, n), V)
        x = np.full((B, n), 7, dtype=np.int32)
        p[:, 0, 7], q[:, 0, 7] = 0.0, 0.25        # refused
        if where == "last":
            p[:, 0, 7] = 0.5                      # accepted: the next row counts
            p[1, 1, [9, V // 2, V - 1]] = bad
        else:
            (p if where == "target" else q)[1, 0, [9, V // 2, V - 1]] = bad
        u = uniform(rng, B, n)
        tokens, accepted, bits = verify(x, p, q, u)
        assert bits == d._abi.TS_DEVERR_PROB
        for b in range(B):
            want, a = oracle.verify_drafts(x[b], n, p[b], q[b], u[b])
            assert tokens[b] == want and accepted[b] == a, (where, b)


@pytest.mark.parametrize("bad", [math.nan, -0.25, 2.0])
def test_a_draft_with_a_bad_probability_is_refused(bad):
    import decode_dsa_kv_gb300 as d
    V = 50
    rng = np.random.default_rng(1)
    p, q = small(rng, (2, 2), V), small(rng, (2, 1), V)
    x = np.full((2, 1), 7, dtype=np.int32)
    p[:, 0, 7], q[:, 0, 7] = 0.5, 0.25
    p[0, 0, 7] = bad
    q[1, 0, 7] = bad
    u = uniform(rng, 2, 1)
    tokens, accepted, bits = verify(x, p, q, u)
    assert bits == d._abi.TS_DEVERR_PROB and accepted == [0, 0]
    for b in range(2):
        want, a = oracle.verify_drafts(x[b], 1, p[b], q[b], u[b])
        assert tokens[b] == want and accepted[b] == a, b
