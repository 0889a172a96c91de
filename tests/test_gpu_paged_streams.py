"""The paged cache's calls on streams other than the one it was made on."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

FORMATS = ["bf16", "e4m3"]


@pytest.mark.parametrize("fmt", FORMATS)
def test_a_new_cache_is_ready_for_any_stream(fmt):
    # the zeros of a new cache are enqueued behind whatever the current stream
    # is busy with; rows written on another stream right away must outlive them
    import decode_dsa_kv_gb300 as d
    n = 40
    x = torch.randn(n, 576, device="cuda").bfloat16()
    slots = torch.randperm(64, device="cuda")[:n].int()
    past = torch.full((1,), 64, dtype=torch.int32, device="cuda")
    want = d.PagedKV(4, 16, fmt)
    want.write(x[:, :512], x[:, 512:], slots)
    assert want.synchronize() == 0
    busy, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(busy):
        torch.cuda._sleep(200_000_000)          # a tenth of a second of work
        kv = d.PagedKV(4, 16, fmt)
    kv.write(x[:, :512], x[:, 512:], slots, stream=other)
    kv.write(x[:1, :512], x[:1, 512:], past, stream=other)     # past the cache: an error bit
    torch.cuda.synchronize()
    assert torch.equal(kv.data, want.data)
    assert kv.synchronize() == d._abi.TS_DEVERR_SLOT_RANGE


@pytest.mark.parametrize("fmt", FORMATS)
def test_a_cache_made_inside_a_capture(fmt):
    # its zeros are part of the graph: every replay starts from an empty cache
    import decode_dsa_kv_gb300 as d
    x = torch.randn(3, 576, device="cuda").bfloat16()
    slots = torch.tensor([5, 0, 63], dtype=torch.int32, device="cuda")
    want = d.PagedKV(4, 16, fmt)
    want.write(x[:, :512], x[:, 512:], slots)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kv = d.PagedKV(4, 16, fmt)
        kv.write(x[:, :512], x[:, 512:], slots)
    for _ in range(2):
        kv.data.fill_(0xA5)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(kv.data, want.data)
    assert kv.synchronize() == 0
