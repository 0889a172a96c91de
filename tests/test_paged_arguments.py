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
