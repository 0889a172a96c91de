"""Host-side checks of the calls for trees and beams: bad arguments come back as
status codes, or as ValueErrors of the wrappers, before anything is enqueued. Run
without a device (a check that failed to fire would go on to enqueue work on
fake addresses)."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="host checks are exercised on machines without a GPU")

from _util import ensure_library  # noqa: E402

ensure_library()
import decode_dsa_kv_gb300 as d  # noqa: E402
from decode_dsa_kv_gb300 import _abi  # noqa: E402

L = _abi._lib
OK, INVALID, UNSUPPORTED, WORKSPACE = (_abi.TS_OK, _abi.TS_ERR_INVALID_ARG,
                                       _abi.TS_ERR_UNSUPPORTED, _abi.TS_ERR_WORKSPACE)
A = 0x10000          # a fake, 256-byte aligned address (never dereferenced)
MIS = A + 8          # 8 bytes off a 16-byte boundary
BIG = 1 << 31

PAGING = [(dict(table=None), INVALID), (dict(stride=0), INVALID), (dict(page=0), INVALID),
          (dict(page=8), UNSUPPORTED), (dict(page=24), UNSUPPORTED), (dict(num_slots=15), INVALID),
          (dict(page=2048, num_slots=4096), UNSUPPORTED)]
CACHE = [(dict(cache=None), INVALID), (dict(cache=MIS), INVALID), (dict(num_slots=0), INVALID),
         (dict(fmt=2), INVALID)]


def plan(parent=A, cu=A, T=4, B=2, ctx=A, table=A, stride=4, page=16, num_slots=64, pos=A, slots=A,
         mask=A, words=1):
    return L.dsa_tree_plan(parent, cu, T, B, ctx, table, stride, page, num_slots, pos, slots, mask,
                           words, None, None)


@pytest.mark.parametrize("kw, want", PAGING + [
    (dict(T=0), OK), (dict(T=0, cu=None), OK), (dict(T=-1), INVALID), (dict(B=0), INVALID),
    (dict(cu=None), INVALID), (dict(ctx=None), INVALID), (dict(words=0), INVALID),
    (dict(words=33), UNSUPPORTED), (dict(num_slots=BIG), UNSUPPORTED),
])
def test_plan_refusals(kw, want):
    assert plan(**kw) == want


def append(latent=A, ls=512, rope=A, rs=64, pos=A, slots=A, n=4, freq=A, cache=A, num_slots=64,
           fmt=0, qr=A, qrs=16 * 64, qrh=64, H=16, q=A, qs=16 * 576):
    return L.dsa_cache_append(latent, ls, rope, rs, pos, slots, n, freq, 1, cache, num_slots, fmt, qr,
                              qrs, qrh, H, q, qs, None, None)


@pytest.mark.parametrize("kw, want", CACHE + [
    (dict(n=0), OK), (dict(n=0, latent=None, q=None), OK), (dict(n=-1), INVALID),
    (dict(latent=None), INVALID), (dict(rope=None), INVALID), (dict(pos=None), INVALID),
    (dict(slots=None), INVALID), (dict(freq=None), INVALID), (dict(freq=A + 4), INVALID),
    (dict(latent=MIS), INVALID), (dict(rope=MIS), INVALID), (dict(ls=504), INVALID),
    (dict(ls=516), INVALID), (dict(rs=56), INVALID), (dict(rs=68), INVALID),
    (dict(q=None), INVALID), (dict(q=MIS), INVALID), (dict(qr=MIS), INVALID), (dict(H=0), INVALID),
    (dict(qrs=56), INVALID), (dict(qrs=1028), INVALID), (dict(qrh=56), INVALID),
    (dict(qrh=68), INVALID), (dict(qs=16 * 576 - 8), INVALID), (dict(qs=16 * 576 + 4), INVALID),
    (dict(H=1025, qs=1025 * 576), UNSUPPORTED),
])
def test_append_refusals(kw, want):
    assert append(**kw) == want


def tree(q=A, qs=16 * 576, cu=A, T=3, B=1, H=16, cache=A, num_slots=64, fmt=1, table=A, stride=4,
         page=16, ctx=A, mask=A, words=2, scale=1 / 24, out=A, ws=A, ws_bytes=None):
    if ws_bytes is None:
        ws_bytes = L.sfa_chunk_workspace_size(max(T, 1), max(B, 1), max(H, 1))
    return L.sfa_mla_tree(q, qs, cu, T, B, H, cache, num_slots, fmt, table, stride, page, ctx, mask,
                          words, scale, out, None, ws, ws_bytes, None, None)


@pytest.mark.parametrize("kw, want", CACHE + PAGING + [
    (dict(T=0), OK), (dict(T=0, mask=None), OK), (dict(mask=None), INVALID), (dict(words=0), INVALID),
    (dict(words=33), UNSUPPORTED), (dict(q=MIS), INVALID), (dict(out=None), INVALID),
    (dict(cu=None), INVALID), (dict(ctx=None), INVALID), (dict(B=0), INVALID),
    (dict(qs=16 * 576 - 8), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(ws=A + 16), WORKSPACE), (dict(ws_bytes=16), WORKSPACE),
])
def test_tree_attention_refusals(kw, want):
    assert tree(**kw) == want


def verify(tokens=A, parent=A, cu=A, T=8, B=2, target=A, ts=100, u=A, V=100, depth=3, path=A, next=A,
           accepted=A):
    return L.ts_verify_tree(tokens, parent, cu, T, B, target, ts, u, V, depth, path, next, accepted,
                            None, None)


@pytest.mark.parametrize("kw, want", [
    (dict(B=0), OK), (dict(B=0, target=None), OK), (dict(B=-1), INVALID), (dict(T=-1), INVALID),
    (dict(V=0), INVALID), (dict(depth=-1), INVALID), (dict(tokens=None), INVALID),
    (dict(cu=None), INVALID), (dict(target=None), INVALID), (dict(target=A + 2), INVALID),
    (dict(path=None), INVALID), (dict(next=None), INVALID), (dict(accepted=None), INVALID),
    (dict(ts=99), INVALID), (dict(V=(1 << 20) + 1, ts=1 << 21), UNSUPPORTED),
    (dict(depth=1025), UNSUPPORTED), (dict(B=1 << 29), UNSUPPORTED),
])
def test_verify_refusals(kw, want):
    assert verify(**kw) == want


def keep(cache=A, num_slots=64, fmt=0, table=A, stride=4, page=16, cu=A, T=8, ctx=A, B=2, path=A,
         depth=3, accepted=A, new_len=A):
    return L.dsa_cache_keep(cache, num_slots, fmt, table, stride, page, cu, T, ctx, B, path, depth,
                            accepted, new_len, None, None)


@pytest.mark.parametrize("kw, want", CACHE + PAGING + [
    (dict(B=0), OK), (dict(B=0, path=None), OK), (dict(B=-1), INVALID), (dict(T=-1), INVALID),
    (dict(depth=-1), INVALID), (dict(cu=None), INVALID), (dict(ctx=None), INVALID),
    (dict(path=None), INVALID), (dict(accepted=None), INVALID), (dict(depth=1025), UNSUPPORTED),
    (dict(num_slots=BIG), UNSUPPORTED),
])
def test_keep_refusals(kw, want):
    assert keep(**kw) == want


def beam(logits=A, dtype=0, stride=100, cum=A, B=2, K=3, V=100, n=4, tokens=A, parents=A, scores=A,
         ws=A, ws_bytes=None):
    if ws_bytes is None:
        ws_bytes = L.ts_beam_workspace_size(max(B, 1), max(K, 1), max(V, 1), max(n, 1))
    return L.ts_beam_select(logits, dtype, stride, cum, B, K, V, n, tokens, parents, scores, ws,
                            ws_bytes, None, None)


@pytest.mark.parametrize("kw, want", [
    (dict(B=0), OK), (dict(B=0, logits=None), OK), (dict(B=-1), INVALID), (dict(K=0), INVALID),
    (dict(V=0), INVALID), (dict(n=0), INVALID), (dict(dtype=2), INVALID),
    (dict(logits=None), INVALID), (dict(logits=A + 2), INVALID), (dict(cum=None), INVALID),
    (dict(tokens=None), INVALID), (dict(parents=None), INVALID), (dict(scores=None), INVALID),
    (dict(ws=None), INVALID), (dict(stride=99), INVALID), (dict(n=65), UNSUPPORTED),
    (dict(V=(1 << 30) + 1, stride=BIG), UNSUPPORTED), (dict(K=1 << 10, V=1 << 22, stride=BIG), UNSUPPORTED),
    (dict(B=1 << 20, K=32), UNSUPPORTED), (dict(ws=A + 16), WORKSPACE), (dict(ws_bytes=64), WORKSPACE),
])
def test_beam_refusals(kw, want):
    assert beam(**kw) == want


def test_beam_workspace_sizes():
    f = L.ts_beam_workspace_size
    assert f(0, 1, 10, 1) == f(1, 0, 10, 1) == f(1, 1, 0, 1) == f(1, 1, 10, 0) == f(1, 1, 10, 65) == 0
    assert 0 < f(1, 1, 10, 1) <= f(1, 1, 10, 8) <= f(4, 4, 100000, 8)


def fork(cache=A, num_slots=64, fmt=0, table=A, stride=4, page=16, ctx=A, parents=A, spare=A, B=1,
         K=2, n=2, new_table=A, new_len=A):
    return L.dsa_cache_fork(cache, num_slots, fmt, table, stride, page, ctx, parents, spare, B, K, n,
                            new_table, new_len, None, None)


@pytest.mark.parametrize("kw, want", CACHE + PAGING + [
    (dict(B=0), OK), (dict(B=0, parents=None), OK), (dict(B=-1), INVALID), (dict(K=0), INVALID),
    (dict(n=0), INVALID), (dict(ctx=None), INVALID), (dict(parents=None), INVALID),
    (dict(spare=None), INVALID), (dict(new_len=None), INVALID), (dict(new_table=None), INVALID),
    (dict(B=1 << 20, K=1 << 12), UNSUPPORTED), (dict(B=1 << 20, n=1 << 12), UNSUPPORTED),
])
def test_fork_refusals(kw, want):
    assert fork(**kw) == want


# ---------------------------------------------------------------------------
# The wrappers, on tensors of the CPU
# ---------------------------------------------------------------------------

def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def bf16(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


KV = d.PagedKV(4, 16, "bf16", device="cpu")
FREQ = torch.zeros(32, dtype=torch.float64)


@pytest.mark.parametrize("change", [
    dict(pos=i32(2)), dict(pos=i32(3).long()), dict(slots=i32(4)), dict(freq=FREQ.float()),
    dict(freq=FREQ[:31]), dict(latent=bf16(3, 511)), dict(rope=bf16(3, 64).float()),
    dict(q_rope=bf16(3, 4, 64)), dict(q=bf16(3, 4, 576)),
    dict(q=bf16(3, 4, 576), q_rope=bf16(3, 5, 64)), dict(q=bf16(3, 4, 575), q_rope=bf16(3, 4, 64)),
    dict(q=bf16(3, 576, 4).transpose(1, 2), q_rope=bf16(3, 4, 64)),
    dict(q=bf16(3, 4, 576), q_rope=bf16(3, 64, 4).transpose(1, 2)),
])
def test_append_arguments(change):
    args = dict(latent=bf16(3, 512), rope=bf16(3, 64), pos=i32(3), slots=i32(3), freq=FREQ)
    with pytest.raises(ValueError):
        KV.append(**{**args, **change})


@pytest.mark.parametrize("change", [
    dict(parent=i32(4)), dict(parent=i32(5).long()), dict(cu_q=i32(2)), dict(ctx_len=i32(3)),
    dict(block_table=i32(2)), dict(T=-1), dict(most=0), dict(most=1025),
])
def test_plan_tree_arguments(change):
    args = dict(parent=i32(5), cu_q=i32(3), block_table=i32(2, 4), ctx_len=i32(2), T=5, most=5)
    with pytest.raises(ValueError):
        KV.plan_tree(**{**args, **change})


@pytest.mark.parametrize("tree", [i32(2), i32(3, 1), i32(2, 0), i32(2, 1).long(), i32(2, 2)[:, :1]])
def test_attend_tree_arguments(tree):
    with pytest.raises(ValueError, match="tree"):
        KV.attend(bf16(2, 4, 576), i32(2), i32(1, 4), i32(1), tree=tree)


@pytest.mark.parametrize("change", [
    dict(path=i32(2)), dict(path=i32(3, 4)), dict(path=i32(2, 0)), dict(path=i32(4, 2).t()),
    dict(accepted=i32(3)), dict(cu_q=i32(2)), dict(T=-1), dict(new_len=i32(1)),
    dict(block_table=i32(3, 4)),
])
def test_keep_arguments(change):
    args = dict(path=i32(2, 4), accepted=i32(2), cu_q=i32(3), T=5, block_table=i32(2, 4),
                ctx_len=i32(2))
    with pytest.raises(ValueError):
        KV.keep(**{**args, **change})


@pytest.mark.parametrize("change", [
    dict(parents=i32(4)), dict(parents=i32(4, 2).t()), dict(spare=i32(7)), dict(ctx_len=i32(5)),
    dict(block_table=i32(5, 3), ctx_len=i32(5)), dict(block_table=i32(6)),
])
def test_fork_arguments(change):
    args = dict(parents=i32(2, 4), spare=i32(8), block_table=i32(6, 3), ctx_len=i32(6))
    with pytest.raises(ValueError):
        KV.fork(**{**args, **change})


@pytest.mark.parametrize("change", [
    dict(target=torch.zeros(5, 8).double()), dict(target=torch.zeros(5, 8).t()),
    dict(target=torch.zeros(1, 8).expand(5, 8)), dict(target=torch.zeros(8)), dict(tokens=i32(4)),
    dict(parent=i32(5).long()), dict(cu_q=i32(0)), dict(u=torch.zeros(2, 0)),
    dict(u=torch.zeros(3, 3)), dict(u=None), dict(depth=-1), dict(depth=3), dict(err=i32(2)),
])
def test_verify_tree_arguments(change):
    args = dict(tokens=i32(5), parent=i32(5), cu_q=i32(3), target=torch.zeros(5, 8),
                u=torch.zeros(2, 3))
    with pytest.raises(ValueError):
        d.verify_tree(**{**args, **change})


@pytest.mark.parametrize("change", [
    dict(logits=torch.zeros(2, 8)), dict(logits=torch.zeros(2, 3, 8).half()),
    dict(logits=torch.zeros(2, 8, 3).transpose(1, 2)), dict(logits=torch.zeros(2, 1, 8).expand(2, 3, 8)),
    dict(logits=torch.zeros(3, 2, 8).transpose(0, 1)), dict(cum=torch.zeros(2, 4)),
    dict(cum=torch.zeros(2, 3).double()), dict(ws=torch.zeros(64)), dict(err=i32(2)),
])
def test_beam_select_arguments(change):
    args = dict(logits=torch.zeros(2, 3, 8), cum=torch.zeros(2, 3), n=2)
    with pytest.raises(ValueError):
        d.beam_select(**{**args, **change})


def test_nothing_to_do_returns_at_once():
    pos, slots, mask = KV.plan_tree(i32(0), i32(1), i32(0, 4), i32(0), 0, 40)
    assert tuple(pos.shape) == (0,) and tuple(slots.shape) == (0,) and tuple(mask.shape) == (0, 2)
    KV.append(bf16(0, 512), bf16(0, 64), i32(0), i32(0), FREQ, bf16(0, 4, 64), bf16(0, 4, 576))
    assert tuple(KV.keep(i32(0, 3), i32(0), i32(1), 0, i32(0, 4), i32(0)).shape) == (0,)
    table, length = KV.fork(i32(0, 4), i32(0), i32(0, 3), i32(0))
    assert tuple(table.shape) == (0, 3) and tuple(length.shape) == (0,)
    out, lse = bf16(0, 4, 512), torch.zeros(0, 4)
    assert KV.attend(bf16(0, 4, 576), i32(1), i32(0, 4), i32(0), tree=i32(0, 1), out=out,
                     lse=lse)[0] is out
