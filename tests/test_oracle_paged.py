"""The paged cache's oracle, pinned: e4m3 against torch's conversion, the scale
rule and round trips, chunk attention against one softmax per token, and draft
verification against float sums and the target's own distribution."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import paged  # noqa: E402
from oracle.sfa import bf16_bits_to_f64, round_to_bf16_bits, sfa_decode  # noqa: E402


def test_e4m3_codes_agree_with_torch():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, paged.e4m3_table(), equal_nan=True)
    rng = np.random.default_rng(0)
    y = np.concatenate([rng.uniform(-448, 448, 4000), rng.normal(0, 2.0 ** -7, 4000),
                        paged.e4m3_table()[:126] + np.diff(paged.e4m3_table()[:127]) / 2,  # ties
                        [0.0, -0.0, 2.0 ** -10, 3 * 2.0 ** -10, 448.0]]).astype(np.float32)
    want = torch.from_numpy(y).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(paged.to_e4m3(y.astype(np.float64)), want)


@pytest.mark.parametrize("top, e", [(448.0, 0), (448.5, 1), (1.75, -8), (1.7500001, -7), (1.0, -8),
                                    (0.0, -120), (2.0 ** -130, -120), (math.inf, 120),
                                    (2.0 ** 127, 119), (1.9921875 * 2.0 ** 127, 120)])
def test_scale_rule(top, e):
    g = np.zeros(128)
    g[5], g[6] = -top, math.nan
    assert paged.scale_of(g) == 2.0 ** e


def test_round_trip_is_within_half_a_step_and_exact_in_bf16():
    rng = np.random.default_rng(1)
    x = round_to_bf16_bits(rng.normal(0, 1, 576) * np.exp(rng.normal(0, 2, 576)))
    raw = paged.pack_row(x, "e4m3")
    assert raw.size == paged.E4M3_ROW
    y, v = paged.unpack_row(raw, "e4m3"), bf16_bits_to_f64(x)
    assert np.array_equal(y[512:], v[512:])
    step = np.repeat(raw[512:528].view(np.float32), 128).astype(np.float64)
    bound = np.maximum(np.abs(v[:512]) * 2.0 ** -4, step * 2.0 ** -10)
    assert np.all(np.abs(y[:512] - v[:512]) <= bound)
    assert np.array_equal(bf16_bits_to_f64(round_to_bf16_bits(y)), y)
    assert np.array_equal(paged.unpack_row(paged.pack_row(x, "bf16"), "bf16"), v)


def test_chunk_attention_is_one_softmax_per_token():
    rng = np.random.default_rng(2)
    K = round_to_bf16_bits(rng.normal(0, 1, (9, 576)))
    q = round_to_bf16_bits(rng.normal(0, 1, (3, 2, 576)))
    out, lse, _, _ = paged.chunk_attention(bf16_bits_to_f64(q), bf16_bits_to_f64(K), 9, True, 0.1)
    for i in range(3):
        o, s = sfa_decode(q[i], K[:7 + i], 0.1)
        assert np.allclose(out[i], o, rtol=1e-12) and np.allclose(lse[i], s, rtol=1e-12)
    out, lse, _, _ = paged.chunk_attention(bf16_bits_to_f64(q), bf16_bits_to_f64(K[:1]), 1, True, 0.1)
    assert np.all(out[:2] == 0) and np.all(np.isneginf(lse[:2]))
    assert np.allclose(out[2], bf16_bits_to_f64(K[0, :512]))


def test_verification_against_float_sums():
    rng = np.random.default_rng(3)
    for _ in range(200):
        n, V = int(rng.integers(0, 4)), int(rng.integers(1, 30))
        p = rng.dirichlet(np.ones(V), n + 1).astype(np.float32)
        q = rng.dirichlet(np.ones(V), n).astype(np.float32).reshape(n, V)
        x = np.array([rng.integers(0, V) for _ in range(n)], dtype=np.int32)
        u = rng.random(n + 1).astype(np.float32)
        tokens, a = paged.verify_drafts(x, n, p, q, u)
        b = 0
        while b < n and np.float64(u[b]) * q[b, x[b]] < p[b, x[b]]:
            b += 1
        assert a == b and list(tokens[:a]) == list(x[:a]) and set(tokens[a + 1:]) <= {-1}
        w = p[a].astype(np.float64) - (q[a] if a < n else 0)
        c = np.cumsum(np.maximum(w, 0))
        if c[-1] > 1e-6:
            assert tokens[a] == int(np.searchsorted(c, np.float64(u[n]) * c[-1], side="right"))


@pytest.mark.parametrize("certain", [False, True])
def test_verified_tokens_follow_the_target(certain):
    # the first token out, over an even grid of both uniforms, has the target's
    # frequencies: sum_x q(x) P(out = t | draft x)
    G, V = 64, 4
    p = np.array([[0.1, 0.4, 0.2, 0.3], [0.25] * 4], dtype=np.float32)
    q = np.array([[0.4, 0.1, 0.3, 0.2]], dtype=np.float32)
    got = np.zeros(V)
    for x in range(V):
        weight = (1.0 if x == 1 else 0.0) if certain else float(q[0, x])
        if not weight:
            continue
        for i in range(G):
            for j in range(G):
                u = np.array([(i + 0.5) / G, (j + 0.5) / G], dtype=np.float32)
                tokens, _ = paged.verify_drafts([x], 1, p, None if certain else q, u)
                got[tokens[0]] += weight / G / G
    # each border of the grid is off by at most one cell in each uniform
    assert np.abs(got - p[0]).max() <= 2 / G
