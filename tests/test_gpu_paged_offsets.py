"""Caches, queries and outputs whose offsets pass 32 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

import oracle  # noqa: E402
from oracle.sfa import bf16_bits_to_f64, round_to_bf16_bits  # noqa: E402
from test_gpu_paged import (FORMATS, bf16, bits, i32, output_bound, random_rows,  # noqa: E402
                            score_error)

SIZE = 66 << 30     # above 2^32 pieces of 16 bytes (64 GiB)


@pytest.mark.parametrize("fmt", FORMATS)
def test_rows_past_32_bits_are_written_read_and_attended_to(fmt):
    import decode_dsa_kv_gb300 as d
    if torch.cuda.mem_get_info()[0] < SIZE + (14 << 30):
        torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < SIZE + (14 << 30):
        pytest.skip("needs 80 GiB of free device memory")
    rng = np.random.default_rng(15)
    row = {"bf16": 1152, "e4m3": 656}[fmt]
    pages = SIZE // (64 * row)
    kv = d.PagedKV(pages, 64, fmt)
    assert kv.data.numel() - 64 * row > 1 << 36
    # the last pages, one in the middle and one whose offset's low 32 bits are small
    wrap = (1 << 32) // (64 * row) + 1
    table = np.array([[pages - 1, wrap, 1, pages // 2, pages - 2]], dtype=np.int32)
    ctx = 300
    x = random_rows(rng, ctx)
    t = np.arange(ctx)
    slots = table[0, t // 64].astype(np.int64) * 64 + t % 64
    xt = bf16(x)
    kv.write(xt[:, :512], xt[:, 512:], i32(slots))
    got = bits(kv.read(i32(table), i32([ctx]), i32(t[None])))
    want = np.stack([oracle.unpack_row(oracle.pack_row(r, fmt), fmt) for r in x])
    assert np.array_equal(bf16_bits_to_f64(got[0]), want)
    assert int((kv.data.view(-1, 64 * row).view(torch.int64) != 0).any(1).sum()) == 5
    q = bf16(round_to_bf16_bits(rng.normal(0, 1, (2, 16, 576))))
    near = d.PagedKV(5, 64, fmt)
    near.write(xt[:, :512], xt[:, 512:], i32(t))
    for causal in (True, False):
        out, lse = kv.attend(q, i32([0, 2]), i32(table), i32([ctx]), causal)
        o, z = near.attend(q, i32([0, 2]), i32([[0, 1, 2, 3, 4]]), i32([ctx]), causal)
        assert torch.equal(out, o) and torch.equal(lse, z)
    # queries further apart than their heads: the copying form of Q
    wide = torch.zeros(2, 16 * 576 + 64, dtype=torch.bfloat16, device="cuda")
    wide[:, :16 * 576] = q.flatten(1)
    out, lse = kv.attend(wide[:, :16 * 576].unflatten(1, (16, 576)), i32([0, 2]), i32(table),
                         i32([ctx]), False)
    assert torch.equal(out, o) and torch.equal(lse, z)
    assert kv.synchronize() == 0 and near.synchronize() == 0
    del kv
    torch.cuda.empty_cache()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("pad", [0, 64])        # tokens side by side, and further apart
def test_queries_and_outputs_past_32_bits(fmt, pad):
    import decode_dsa_kv_gb300 as d
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GiB of free device memory")
    rng = np.random.default_rng(16)
    T, H, ctx = 40_000, 128, (300, 77)
    new = (T - 10, 10)
    kv = d.PagedKV(7, 64, fmt)
    table = np.array([[3, 0, 6, 1, 4], [5, 2, 0, 0, 0]], dtype=np.int32)
    x = random_rows(rng, sum(ctx))
    t = np.concatenate([np.arange(c) for c in ctx])
    b = np.repeat([0, 1], ctx)
    xt = bf16(x)
    kv.write(xt[:, :512], xt[:, 512:], i32(table[b, t // 64] * 64 + t % 64))
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    wide = torch.empty(T, H * 576 + pad, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    q = wide[:, :H * 576].unflatten(1, (H, 576))
    assert wide.numel() > 1 << 31 and T * H * 512 > 1 << 31
    out, lse = kv.attend(q, i32([0, new[0], T]), i32(table), i32(ctx), False)
    assert kv.synchronize() == 0
    K = [np.stack([oracle.unpack_row(oracle.pack_row(r, fmt), fmt) for r in x[b == i]])
         for i in (0, 1)]
    # tokens on both sides of the offsets 2^31 and 2^32, and others of every part
    at = sorted({0, 1, 14_563, 14_564, 29_126, 29_128, 32_767, 32_768, T - 11, T - 10, T - 1}
                | set(rng.integers(0, T, 100).tolist()))
    for i in at:
        r = 0 if i < new[0] else 1
        o, z, mean_abs, size = oracle.chunk_attention(
            q[i:i + 1].double().cpu().numpy(), K[r], ctx[r], False, 1 / 24)
        err = np.abs(out[i].double().cpu().numpy() - o[0])
        assert np.all(err <= output_bound(o, mean_abs, size)[0]), i
        assert np.all(np.abs(lse[i].double().cpu().numpy() - z[0])
                      <= 2 * score_error(size)[0] + 2.0 ** -20 + 2.0 ** -22 * np.abs(z[0])), i
    del wide, q, out, lse
    torch.cuda.empty_cache()
