"""PagedKV's checks of its arguments, made before anything touches a device: on
tensors of the CPU, wherever the tests run."""
import pytest

torch = pytest.importorskip("torch")

from _util import ensure_library  # noqa: E402

ensure_library()
import decode_dsa_kv_gb300 as d  # noqa: E402


def attend(**kw):
    kv = d.PagedKV(4, 16, "bf16", device="cpu")
    i32 = dict(dtype=torch.int32)
    return kv.attend(torch.zeros(2, 4, 576, dtype=torch.bfloat16), torch.tensor([0, 2], **i32),
                     torch.zeros(1, 4, **i32), torch.tensor([5], **i32), **kw)


SIZE = d.sfa_chunk_workspace_size(2, 1, 4)


@pytest.mark.parametrize("ws", [
    torch.empty(SIZE, dtype=torch.uint8, device="meta"),      # another device than the cache's
    torch.empty(256, dtype=torch.uint8)[:1].expand(SIZE),     # one byte, named SIZE times
    torch.empty(2 * SIZE, dtype=torch.uint8)[::2],            # bytes apart
    torch.empty(SIZE, dtype=torch.float32),                   # numel() is no count of bytes
], ids=["device", "expanded", "strided", "float"])
def test_a_workspace_that_is_not_the_cache_devices_bytes_is_refused(ws):
    with pytest.raises(ValueError, match="ws: "):
        attend(ws=ws)


@pytest.mark.parametrize("B, k", [(0, 5), (2, 0), (0, 0)])
def test_reading_nothing_returns_nothing(B, k):
    kv = d.PagedKV(4, 16, "e4m3", device="cpu")
    i32 = dict(dtype=torch.int32)
    args = torch.zeros(B, 4, **i32), torch.zeros(B, **i32), torch.zeros(B, k, **i32)
    out = kv.read(*args)
    assert out.dtype == torch.bfloat16 and tuple(out.shape) == (B, k, 576)
    mine = torch.empty(B, k, 576, dtype=torch.bfloat16)
    assert kv.read(*args, out=mine) is mine
    with pytest.raises(ValueError, match="out: "):
        kv.read(*args, out=torch.empty(B, k, 575, dtype=torch.bfloat16))


def test_attending_for_no_request_leaves_every_row_as_it_was():
    kv = d.PagedKV(4, 16, "bf16", device="cpu")
    i32 = dict(dtype=torch.int32)
    for T in (0, 3):
        out = torch.full((T, 4, 512), 3.0, dtype=torch.bfloat16)
        lse = torch.full((T, 4), 5.0)
        o, z = kv.attend(torch.zeros(T, 4, 576, dtype=torch.bfloat16), torch.zeros(1, **i32),
                         torch.zeros(0, 4, **i32), torch.zeros(0, **i32), out=out, lse=lse)
        assert o is out and z is lse and torch.all(out == 3) and torch.all(lse == 5)
