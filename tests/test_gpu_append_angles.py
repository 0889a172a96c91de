"""Appended rows and queries at the ends of the angles' range: frequencies that
are no numbers, and ones so small that an angle is a tiny part of a turn."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

from test_gpu_paged import BF16_HALF_STEP, bf16, i32, random_rows  # noqa: E402


@pytest.fixture(scope="module")
def d():
    import decode_dsa_kv_gb300 as mod
    return mod


def appended(d, rope, pos, freq, interleaved):
    """rope bf16 [n][64] through a row of the cache and through a query."""
    n = len(pos)
    kv = d.PagedKV(-(-n // 16), 16)
    latent = torch.zeros((n, 512), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((n, 1, 576), dtype=torch.bfloat16, device="cuda")
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    kv.append(latent, rope, i32(pos), slots, torch.from_numpy(np.asarray(freq, dtype=np.float64)).cuda(),
              rope.view(n, 1, 64), q, interleaved=interleaved)
    assert kv.synchronize() == 0
    row = kv.data[:n].view(torch.bfloat16)[:, 512:]
    # (bit for bit, a NaN too)
    assert torch.equal(row.contiguous().view(torch.int16), q[:, 0, 512:].contiguous().view(torch.int16))
    return row.double().cpu().numpy()


@pytest.mark.parametrize("interleaved", [True, False])
def test_a_frequency_that_is_no_number_gives_none(d, interleaved):
    rng = np.random.default_rng(1)
    pos = [0, 1, 77, -3, 2 ** 27 - 1]
    rope = bf16(random_rows(rng, len(pos)))[:, 512:].contiguous()
    freq = 10000.0 ** (-np.arange(32) / 32)
    want = appended(d, rope, pos, freq, interleaved)
    bad = freq.copy()
    bad[3], bad[17], bad[31] = math.nan, math.inf, -math.inf
    got = appended(d, rope, pos, bad, interleaved)
    pair = np.arange(64) // 2 if interleaved else np.arange(64) % 32
    hit = np.isin(pair, [3, 17, 31])
    assert np.all(np.isnan(got[:, hit]))
    assert np.array_equal(got[:, ~hit], want[:, ~hit])


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("sign", [1, -1])
def test_small_angles(d, interleaved, sign):
    # a = 1, b = 0: the turned pair is (cos, sin) itself
    freq = sign * 10.0 ** -np.linspace(3, 10, 32)
    pos = [1, 2, 3, 50, 1000, 4097, 65535]
    one = torch.zeros((len(pos), 64), dtype=torch.bfloat16, device="cuda")
    if interleaved:
        one[:, 0::2] = 1
    else:
        one[:, :32] = 1
    got = appended(d, one, pos, freq, interleaved)
    c, s = (got[:, 0::2], got[:, 1::2]) if interleaved else (got[:, :32], got[:, 32:])
    angle = np.asarray(pos)[:, None] * freq
    # the angle: |pos| 2^-54 of a turn, then 2^-24 of itself; its sine (2 units in
    # the last place of fp32), and one rounding to bf16
    for v, want in ((c, np.cos(angle)), (s, np.sin(angle))):
        bound = (1.01 * BF16_HALF_STEP + 2.0 ** -21) * np.abs(want) + \
            2 * math.pi * 2.0 ** -54 * np.asarray(pos)[:, None]
        assert np.all(np.abs(v - want) <= bound), float((np.abs(v - want) / bound).max())
