"""Trees whose lengths are out of order or do not fit their context: what is
planned for the tokens that one request has, or none, and what is reported."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

import oracle  # noqa: E402
from test_gpu_candidates import FORMATS, Trees  # noqa: E402
from test_gpu_paged import i32, output_bound  # noqa: E402


@pytest.fixture(scope="module")
def d():
    import decode_dsa_kv_gb300 as mod
    return mod


@pytest.mark.parametrize("cu, T", [
    ([0, 5, 3], 10), ([5, 0, 3], 8), ([0, 2, 100, 6], 8), ([4, -7, 2, 9], 12), ([0, 2000, 10, 2100], 2200),
    ([0, 1500, 3], 2000), ([1900, 0, 1800], 2000), ([0, 4, 9], 12),
])
def test_tokens_of_one_request_or_none_where_lengths_are_out_of_order(d, cu, T):
    B, page = len(cu) - 1, 16
    ctx = 2208
    pages = ctx // page
    kv = d.PagedKV(B * pages, page)
    table = i32(np.arange(B * pages).reshape(B, pages))
    first = [min(max(x, 0), T) for x in cu[:-1]]
    count = [max(min(x, T) - f, 0) for f, x in zip(first, cu[1:])]
    owners = [[b for b in range(B) if first[b] <= t < first[b] + count[b]] for t in range(T)]
    for _ in range(20):
        pos, slots, mask = kv.plan_tree(None, i32(cu), table, i32([ctx] * B), T, 1024)
        pos, slots, mask = pos.tolist(), slots.tolist(), mask.cpu().numpy()
        for t, who in enumerate(owners):
            if not who:
                assert pos[t] == 0 and slots[t] == -1 and not mask[t].any(), t
            elif len(who) == 1:                       # (tokens that two share: either's)
                b = who[0]
                at = ctx - count[b] + t - first[b]
                assert pos[t] == at and slots[t] == b * ctx + at, t
    e = d._abi
    want = e.TS_DEVERR_ORDER if cu != sorted(cu) or cu[0] < 0 or cu[-1] > T else 0
    want |= e.TS_DEVERR_COUNT if max(count) > 1024 else 0
    assert kv.synchronize() == want


@pytest.mark.parametrize("fmt", FORMATS)
def test_tree_attention_reports_more_nodes_than_positions(d, fmt):
    c = Trees(d, fmt, 16, 16, [(5, 5), (7, 40), (9, 9)], seed=21)
    want, _ = c.run()
    c.check(*c.run())
    # the first request's nodes 0 and 1, the last one's 0 to 8 have no position then
    c.ctx.copy_(i32([3, 40, 0]))
    out, lse = c.run()
    assert c.kv.synchronize() == d._abi.TS_DEVERR_CTX
    assert torch.equal(out[5:12], want[5:12])
    assert torch.all(out[12:] == 0) and torch.all(torch.isneginf(lse[12:]))
    for i in range(5):
        K = c.K[0][:3][c.seen[0][i, 2:]]
        o, z, mean_abs, size = oracle.chunk_attention(c.q64[i:i + 1], K, len(K), False, 1 / 24)
        assert np.all(np.abs(out[i:i + 1].double().cpu().numpy() - o) <= output_bound(o, mean_abs, size))
        assert np.array_equal(np.isneginf(z), torch.isneginf(lse[i:i + 1]).cpu().numpy())
