"""Appended rows and queries at the ends of the angles' range: frequencies that
are no numbers."""
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
