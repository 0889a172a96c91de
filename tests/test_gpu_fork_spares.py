"""Forked sequences whose next row starts a page: a spare page outside the cache
is reported, though no row is copied there."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

from test_gpu_paged import i32  # noqa: E402


@pytest.fixture(scope="module")
def d():
    import decode_dsa_kv_gb300 as mod
    return mod


@pytest.mark.parametrize("spare, bad", [(-1, True), (8, True), (2 ** 31 - 1, True), (0, False), (7, False)])
@pytest.mark.parametrize("tables", [True, False])
def test_a_spare_page_outside_the_cache_is_reported(d, spare, bad, tables):
    kv = d.PagedKV(8, 16)
    kv.data.copy_(torch.arange(kv.data.numel(), device="cuda").view(kv.data.shape) % 251)
    old = kv.data.clone()
    # lengths that end with a page, and one of 0
    for ctx in (16, 0):
        got = kv.fork(i32([[0]]), i32([spare]), i32([[1, -1]]), i32([ctx]), tables=tables)
        assert kv.synchronize() == (d._abi.TS_DEVERR_SLOT_RANGE if bad else 0)
        assert torch.equal(kv.data, old)
        if tables:
            assert got[0].tolist() == [[1, spare] if ctx else [spare, -1]] and got[1].tolist() == [ctx]


def test_sequences_that_get_no_spare_page_name_any(d):
    # one that fills its table, one that is none
    kv = d.PagedKV(8, 16)
    table, length = kv.fork(i32([[0, -1]]), i32([-1, 99]), i32([[1, 2]]), i32([32]))
    assert kv.synchronize() == 0
    assert table.tolist() == [[1, 2], [-1, -1]] and length.tolist() == [32, 0]
