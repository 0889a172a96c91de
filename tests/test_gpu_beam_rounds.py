"""Beam selection over many long rows, of which a CTA takes pieces of several
rounds: values far above those before them, rows that rise round by round, that
cross the size from which a part takes its largest value for reference, bad
values in late rounds, more equal values than the list holds. Against the oracle
in 64 bits."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

from test_gpu_candidates import check_beams  # noqa: E402

DTYPES = [torch.float32, torch.bfloat16]


@pytest.fixture(scope="module")
def d():
    import decode_dsa_kv_gb300 as mod
    return mod


# A piece is of ceil(units / want) rounds, at most 8: want = min(units, 7 x 152 SMs /
# rows), a unit 2048 fp32 or 4096 bf16 values. (B, K, V, rounds of fp32, of bf16)
SHAPES = [(20, 2, 131072, 3, 2), (32, 5, 50257, 5, 3), (64, 8, 131072, 8, 8)]


def select(d, x, cum, n, want_err=0, shift=3):
    """The call on rows that start between 16-byte boundaries, and the logits as
    the type has them; every `shift`-th value of padding is a NaN outside of them."""
    B, K, V = x.shape
    wide = torch.full((B, K, V + shift), math.nan, dtype=x.dtype, device="cuda")
    wide[:, :, :V] = x
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = d.beam_select(wide[:, :, :V], cum, n, err=err)
    assert d.ts_read_error(err) == want_err
    return got


def check(x, cum, n, got, requests):
    """Those requests, the others by their scores' sizes."""
    host, c = x.double(), cum.cpu().numpy()
    for b in requests:
        check_beams(host[b:b + 1].cpu().numpy(), c[b:b + 1], n, [g[b:b + 1] for g in got])
    # a score is the chosen logit's log-probability and its beam's sum: all of them
    fin = torch.where(host < math.inf, host, -math.inf)
    at, par = got[0].clamp(min=0).long(), got[1].clamp(min=0).long()
    lse = torch.logsumexp(fin, 2)
    want = cum.double().gather(1, par) + (
        fin.gather(1, par[:, :, None].expand(-1, -1, x.shape[2])).gather(2, at[:, :, None])[:, :, 0]
        - lse.gather(1, par))
    live = got[1] >= 0
    tol = 2.0 ** -17 + 2.0 ** -23 * want.abs()      # (check_beams')
    off = (got[2].double() - want).abs()
    assert bool(torch.all((off <= tol) | ~live)), float((off - tol)[live].max())


def normal(shape, seed, scale=2.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return scale * torch.randn(shape, generator=g, device="cuda")


def scores(B, K, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return -3 * torch.rand(B, K, generator=g, device="cuda") - 2


HEIGHTS = [20.0, 24.0, 30.0, 36.0, 40.0, 44.0, 50.0, 100.0]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B, K, V, r32, r16", SHAPES)
@pytest.mark.parametrize("base", [0.0, -30.0])
def test_one_token_far_above_the_rest(d, dtype, B, K, V, r32, r16, base):
    # its place: the row's start, pieces' later rounds, its end
    x = normal((B, K, V), V) + base
    rows = x.view(B * K, V)
    places = [0, 3000, 9000, V // 3, V // 2 + 77, (4 * V) // 5, V - 1]
    for r in range(B * K):
        if r % 9 != 8:                              # (some rows without one)
            rows[r, places[r % 7]] = base + HEIGHTS[(r // 7) % len(HEIGHTS)]
        if r % 4 == 3:                              # a second one, in another part
            rows[r, places[(r + 3) % 7]] = base + HEIGHTS[(r // 7) % len(HEIGHTS)] - 1.5
    x = x.to(dtype)
    cum = scores(B, K, 1)
    got = select(d, x, cum, 8)
    check(x, cum, 8, got, range(0, B, max(1, B // 6)))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("allowed", [1, 2, 40])
def test_rows_of_a_low_value_with_a_few_allowed_tokens(d, dtype, allowed):
    B, K, V, n = 32, 5, 50257, 10
    x = torch.full((B, K, V), -30.0, device="cuda")
    rng = np.random.default_rng(allowed)
    for b in range(B):
        for k in range(K):
            at = torch.from_numpy(rng.choice(V, allowed, replace=False)).cuda()
            x[b, k, at] = torch.from_numpy(rng.uniform(-6, 6, allowed).astype(np.float32)).cuda()
    x = x.to(dtype)
    cum = scores(B, K, 2)
    check(x, cum, n, select(d, x, cum, n), range(0, B, 7))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B, K, V, r32, r16", SHAPES[:2])
@pytest.mark.parametrize("rise", [30.0, 300.0, 3e4, -300.0])
def test_rows_that_rise(d, dtype, B, K, V, r32, r16, rise):
    # from a piece's round to its next (of 2048 or 4096 values)
    t = torch.arange(V, device="cuda")
    x = normal((B, K, V), 5, 1.0) + rise * (t // 2048).float() / (V // 2048)
    x = x.to(dtype)
    cum = scores(B, K, 3)
    check(x, cum, 12, select(d, x, cum, 12), range(0, B, max(1, B // 3)))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("size", [2.0 ** 20, -2.0 ** 20])
@pytest.mark.parametrize("far_first", [False, True])
def test_rows_that_cross_the_references_border_within_a_piece(d, dtype, size, far_first):
    B, K, V = 20, 2, 131072
    near, far = size * (1 - 2.0 ** -7), size * (1 + 2.0 ** -6)
    t = torch.arange(V, device="cuda") // 4096 % 2 == (1 if far_first else 0)
    x = torch.where(t, near, far).expand(B, K, V) + 8192 * torch.round(normal((B, K, V), 6, 1.0))
    x = x.to(dtype)
    cum = scores(B, K, 4)
    got = select(d, x, cum, 20)
    host, c = x.double().cpu().numpy(), cum.cpu().numpy()
    for b in (0, 7, 19):
        check_beams(host[b:b + 1], c[b:b + 1], 20, [g[b:b + 1] for g in got])


@pytest.mark.parametrize("size", [2.0 ** 20, -2.0 ** 20])
def test_rows_a_few_apart_on_both_sides_of_the_border(d, size):
    B, K, V = 20, 2, 131072
    t = torch.arange(V, device="cuda") // 2048 % 3
    x = size + torch.where(t == 0, -4.0, torch.where(t == 1, 2.0, -1.0)).expand(B, K, V)
    x = x + torch.round(4 * normal((B, K, V), 7, 1.0)) / 4
    x = torch.minimum(x, size + torch.tensor(9.0, device="cuda"))
    cum = scores(B, K, 5)
    check(x, cum, 20, select(d, x, cum, 20), (0, 11))


@pytest.mark.parametrize("dtype", DTYPES)
def test_values_behind_rounds_without_any(d, dtype):
    # -infinity, or the type's lowest value, in all rounds but some
    B, K, V = 32, 5, 50257
    x = normal((B, K, V), 8)
    t = torch.arange(V, device="cuda") // 2048
    low = torch.finfo(dtype).min
    x[::2, :, t % 5 != 3] = -math.inf
    x[1::2, :, t % 5 != 2] = low
    x[5, 2] = -math.inf
    x[6] = -math.inf
    x = x.to(dtype)
    cum = scores(B, K, 6)
    got = select(d, x, cum, 16)
    check(x, cum, 16, got, (0, 1, 5, 6, 30, 31))
    assert torch.all(got[1][6] == -1)


@pytest.mark.parametrize("dtype", DTYPES)
def test_bad_values_in_late_rounds(d, dtype):
    B, K, V = 32, 5, 50257
    x = normal((B, K, V), 9)
    x[0, 0, 9000:9500] = math.nan
    x[1, 1, V - 1] = math.inf
    x[2, 2, 8192:] = math.nan
    x[3, 3, ::7] = math.inf
    x[4, 4, :8192] = math.nan
    x[5, 0, 20000] = -math.nan
    x[5, 0, 20001] = 60.0
    x = x.to(dtype)
    cum = scores(B, K, 7)
    got = select(d, x, cum, 9, want_err=d._abi.TS_DEVERR_NAN)
    check(x, cum, 9, got, range(8))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", ["one value", "two values", "nine of ten masked"])
def test_more_equal_values_than_the_list_holds(d, dtype, kind):
    B, K, V, n = 32, 5, 50257, 10
    if kind == "one value":
        x = torch.full((B, K, V), 1.5, device="cuda")
    else:
        z = normal((B, K, V), 10)
        x = torch.where(z > 0, 1.0, -1.0) if kind == "two values" else z
        if kind == "nine of ten masked":
            x[:, :, torch.arange(V, device="cuda") % 10 != 0] = torch.finfo(dtype).min
    x = x.to(dtype)
    cum = scores(B, K, 8)
    got = select(d, x, cum, n)
    check(x, cum, n, got, (0, 13, 31))
    if kind == "one value":                         # ties: the best beam's lowest tokens
        assert torch.equal(got[0], torch.arange(n, device="cuda", dtype=torch.int32).expand(B, n))
        assert torch.equal(got[1].long(), cum.argmax(1, keepdim=True).expand(B, n))
