"""Host-side checks of the paged cache's calls: bad arguments come back as
status codes before anything is enqueued. Run without a device (a check that
failed to fire would go on to enqueue work on fake addresses)."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="host checks are exercised on machines without a GPU")

from _util import ensure_library  # noqa: E402

ensure_library()
from decode_dsa_kv_gb300 import _abi  # noqa: E402

L = _abi._lib
OK, INVALID, UNSUPPORTED, WORKSPACE = (_abi.TS_OK, _abi.TS_ERR_INVALID_ARG,
                                       _abi.TS_ERR_UNSUPPORTED, _abi.TS_ERR_WORKSPACE)
A = 0x10000          # a fake, 256-byte aligned address (never dereferenced)
MIS = A + 8          # 8 bytes off a 16-byte boundary


def test_row_bytes():
    assert [L.dsa_cache_row_bytes(f) for f in (0, 1, 2, -1)] == [1152, 656, 0, 0]


def write(latent=A, ls=512, rope=A, rs=64, slots=A, n=4, cache=A, num_slots=64, fmt=0):
    return L.dsa_cache_write(latent, ls, rope, rs, slots, n, cache, num_slots, fmt, None, None)


@pytest.mark.parametrize("kw, want", [
    (dict(n=0), OK), (dict(n=0, latent=None, slots=None), OK), (dict(n=-1), INVALID),
    (dict(latent=None), INVALID), (dict(rope=None), INVALID), (dict(slots=None), INVALID),
    (dict(cache=None), INVALID), (dict(latent=MIS), INVALID), (dict(rope=MIS), INVALID),
    (dict(cache=MIS), INVALID), (dict(ls=504), INVALID), (dict(ls=516), INVALID),
    (dict(rs=56), INVALID), (dict(rs=68), INVALID), (dict(num_slots=0), INVALID),
    (dict(fmt=2), INVALID), (dict(fmt=-1), INVALID),
])
def test_write_refusals(kw, want):
    assert write(**kw) == want


def read(cache=A, num_slots=64, fmt=1, table=A, stride=4, page=16, pos=A, ctx=A, B=1, k=8, sel=A):
    return L.dsa_cache_read(cache, num_slots, fmt, table, stride, page, pos, ctx, B, k, sel, None,
                            None)


PAGING = [
    (dict(cache=None), INVALID), (dict(cache=MIS), INVALID), (dict(num_slots=0), INVALID),
    (dict(num_slots=15), INVALID), (dict(fmt=7), INVALID), (dict(table=None), INVALID),
    (dict(stride=0), INVALID), (dict(page=0), INVALID), (dict(page=8), UNSUPPORTED),
    (dict(page=24), UNSUPPORTED), (dict(page=2048, num_slots=4096), UNSUPPORTED),
    (dict(ctx=None), INVALID), (dict(B=0), INVALID),
]


@pytest.mark.parametrize("kw, want", PAGING + [
    (dict(pos=None), INVALID), (dict(sel=None), INVALID), (dict(sel=MIS), INVALID),
    (dict(k=0), INVALID), (dict(B=1 << 16, k=1 << 15), UNSUPPORTED),
])
def test_read_refusals(kw, want):
    assert read(**kw) == want


def chunk(q=A, qs=16 * 576, cu=A, T=3, B=1, H=16, cache=A, num_slots=64, fmt=1, table=A, stride=4,
          page=16, ctx=A, causal=1, scale=1 / 24, out=A, ws=A, ws_bytes=None):
    if ws_bytes is None:
        ws_bytes = L.sfa_chunk_workspace_size(max(T, 1), max(B, 1), max(H, 1))
    return L.sfa_mla_chunk(q, qs, cu, T, B, H, cache, num_slots, fmt, table, stride, page, ctx,
                           causal, scale, out, None, ws, ws_bytes, None, None)


@pytest.mark.parametrize("kw, want", PAGING + [
    (dict(T=0), OK), (dict(T=0, q=None), OK), (dict(T=-1), INVALID), (dict(H=0), INVALID),
    (dict(q=None), INVALID), (dict(cu=None), INVALID), (dict(out=None), INVALID),
    (dict(ws=None), INVALID), (dict(q=MIS), INVALID), (dict(out=MIS), INVALID),
    (dict(qs=16 * 576 - 8), INVALID), (dict(qs=16 * 576 + 4), INVALID),
    (dict(scale=math.nan), INVALID), (dict(scale=math.inf), INVALID),
    (dict(H=1025, qs=1025 * 576), UNSUPPORTED), (dict(T=1 << 27), UNSUPPORTED),
    (dict(ws=A + 16), WORKSPACE), (dict(ws_bytes=16), WORKSPACE),
])
def test_chunk_refusals(kw, want):
    assert chunk(**kw) == want


def test_chunk_workspace_sizes():
    f = L.sfa_chunk_workspace_size
    assert f(0, 1, 16) == f(1, 0, 16) == f(1, 1, 0) == 0
    assert f(1, 1, 1) > 0 and f(64, 8, 128) >= f(1, 1, 128)


def verify(drafts=A, nd=None, target=A, ts=100, draft=A, ds=100, u=A, B=2, n=3, V=100, tokens=A,
           accepted=A):
    return L.ts_verify_drafts(drafts, nd, target, ts, draft, ds, u, B, n, V, tokens, accepted, None,
                              None)


@pytest.mark.parametrize("kw, want", [
    (dict(B=0), OK), (dict(B=0, target=None), OK), (dict(B=-1), INVALID), (dict(n=-1), INVALID),
    (dict(V=0), INVALID), (dict(drafts=None), INVALID), (dict(target=None), INVALID),
    (dict(u=None), INVALID), (dict(tokens=None), INVALID), (dict(accepted=None), INVALID),
    (dict(ts=99), INVALID), (dict(ds=99), INVALID),
    (dict(V=1 << 26, ts=1 << 26, ds=1 << 26), UNSUPPORTED), (dict(n=70000), UNSUPPORTED),
])
def test_verify_refusals(kw, want):
    assert verify(**kw) == want


def test_python_wrappers_refuse_wrong_tensors():
    import decode_dsa_kv_gb300 as d
    with pytest.raises(ValueError):
        d.PagedKV(4, 16, "fp4", device="cpu")
    kv = d.PagedKV(4, 16, "e4m3", device="cpu")
    assert tuple(kv.data.shape) == (64, 656)
    x = torch.zeros(3, 576, dtype=torch.bfloat16)
    slots = torch.zeros(3, dtype=torch.int32)
    for bad in [(x[:, :512].float(), x[:, 512:], slots), (x[:, :511], x[:, 512:], slots),
                (x[:, :512], x[:, 512:], slots.long()), (x[:, :512], x[:, 512:], slots[:2]),
                (x[:2, :512], x[:, 512:], slots)]:
        with pytest.raises(ValueError):
            kv.write(*bad)
    table, ctx = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    pos = torch.zeros(2, 5, dtype=torch.int32)
    for bad in [(table[:1], ctx, pos), (table, ctx[:1], pos), (table, ctx, pos[0]),
                (table.float(), ctx, pos), (table[:, ::2], ctx, pos)]:
        with pytest.raises(ValueError):
            kv.read(*bad)
    q, cu = torch.zeros(2, 4, 576, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    for bad in [(q, cu[:2], table, ctx), (q.float(), cu, table, ctx), (q[..., :575], cu, table, ctx)]:
        with pytest.raises((ValueError, RuntimeError)):
            kv.attend(*bad)
    p = torch.zeros(2, 4, 50)
    x = torch.zeros(2, 3, dtype=torch.int32)
    u = torch.zeros(2, 4)
    for bad in [(x, p[:, :3], None, u), (x, p.double(), None, u), (x.long(), p, None, u),
                (x, p, p, u), (x, p, None, u[:, :3]), (x, p.transpose(1, 2), None, u)]:
        with pytest.raises(ValueError):
            d.verify_drafts(*bad)


def test_verify_rows_that_lie_closer_than_their_length_are_refused():
    import decode_dsa_kv_gb300 as d
    drafts, u = torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, 2)
    p, q = torch.full((2, 2, 5), 0.2), torch.full((2, 1, 5), 0.2)
    row = torch.full((1, 1, 5), 0.2)
    for target, draft in ((row.expand(2, 2, 5), q), (p, row.expand(2, 1, 5)),
                          (p[:, :1].expand(2, 2, 5), q), (p.transpose(0, 1), q)):
        with pytest.raises(ValueError):
            d.verify_drafts(drafts, target, draft, u)
