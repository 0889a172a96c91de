"""The paged latent cache on the GPU, against its oracle: rows written and read
back bit for bit, chunk attention within derived bounds, draft verification
exactly; refusals of bad data; streams, graphs and a run of all of them."""
import math
import os
import subprocess
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

import oracle  # noqa: E402
from oracle.sfa import bf16_bits_to_f64, round_to_bf16_bits  # noqa: E402

FORMATS = ["bf16", "e4m3"]
BF16_HALF_STEP = 2.0 ** -8       # of a rounding to bf16, relative to the value


@pytest.fixture(scope="module")
def d():
    import decode_dsa_kv_gb300 as mod
    return mod


def bits(x: torch.Tensor) -> np.ndarray:
    return x.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def bf16(x: np.ndarray) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(x).view(np.int16)).cuda().view(torch.bfloat16)


def i32(x) -> torch.Tensor:
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def random_rows(rng, n, size=1.0) -> np.ndarray:
    x = rng.normal(0, size, (n, 576)) * np.exp(rng.normal(0, 0.5, (n, 1)))
    return round_to_bf16_bits(x)


def score_error(size):
    """How far a scaled score may be off, given scale * sum |q||k|. A score is a
    sum of 576 exact products in fp32: at most 36 + 4 roundings or cuts (2^-22
    of the sum of sizes at worst) of partial sums over 16 products each; 2^-22
    more each for the scaling and for the exponential's argument and value."""
    return 40 * 2.0 ** -22 * size + 2.0 ** -21


def output_bound(o, mean_abs, size):
    """How far an output may be off. A weight is off by its score's error and
    its rounding to bf16, the sum of the weights by no more; the output rounds
    once more, and merging parts of a row adds a few fp32 roundings."""
    e = (BF16_HALF_STEP + 2 * score_error(size))[..., None]
    return e * (mean_abs + np.abs(o)) + 1.01 * BF16_HALF_STEP * np.abs(o) + 2.0 ** -130


# ---------------------------------------------------------------------------
# Rows
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n, fused", [(1, False), (7, True), (33, False), (300, True)])
def test_write_puts_rows_into_their_slots_only(d, fmt, n, fused):
    rng = np.random.default_rng(n)
    x = random_rows(rng, n)
    x[0, 128:256] = 0                                     # a group of zeros
    x[0, 5] = 0x0001                                      # bf16's smallest subnormal
    if n > 1:
        x[1, 0:128] = round_to_bf16_bits(rng.normal(0, 1, 128) * 2.0 ** -124)
        x[1, 130] = 0x7f80                                # +inf
        x[1, 300] = 0xffc0                                # NaN
    t = bf16(x)
    wide = torch.zeros(n, 640, dtype=torch.bfloat16, device="cuda")
    wide[:, 8:520], wide[:, 528:592] = t[:, :512], t[:, 512:]
    latent, rope = ((wide[:, 8:520], wide[:, 528:592]) if fused
                    else (t[:, :512].contiguous(), t[:, 512:].contiguous()))
    kv = d.PagedKV(40, 16, fmt)
    kv.data.fill_(0xA5)
    slots = rng.permutation(kv.num_slots)[:n].astype(np.int32)
    skipped = n // 3
    given = slots.copy()
    given[n - skipped:] = -1 - np.arange(skipped)
    kv.write(latent, rope, i32(given))
    assert kv.synchronize() == 0
    want = np.full(kv.data.shape, 0xA5, dtype=np.uint8)
    for i in range(n - skipped):
        want[slots[i]] = oracle.pack_row(x[i], fmt)
    assert np.array_equal(kv.data.cpu().numpy(), want)


@pytest.mark.parametrize("fmt", FORMATS)
def test_write_skips_slots_past_the_cache(d, fmt):
    rng = np.random.default_rng(5)
    kv = d.PagedKV(2, 16, fmt)
    x = random_rows(rng, 3)
    t = bf16(x)
    kv.write(t[:, :512], t[:, 512:], i32([31, 32, 2 ** 31 - 1]))
    assert kv.synchronize() == d._abi.TS_DEVERR_SLOT_RANGE
    want = np.zeros(kv.data.shape, dtype=np.uint8)
    want[31] = oracle.pack_row(x[0], fmt)
    assert np.array_equal(kv.data.cpu().numpy(), want)
    kv.write(t[:0, :512], t[:0, 512:], i32([]))
    assert kv.synchronize() == 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("page, B, k", [(16, 3, 50), (64, 1, 1), (1024, 2, 129)])
def test_read_returns_the_stored_rows(d, fmt, page, B, k):
    rng = np.random.default_rng(page)
    pages = 6 * B
    kv = d.PagedKV(pages, page, fmt)
    n = kv.num_slots
    x = random_rows(rng, n)
    t = bf16(x)
    kv.write(t[:, :512], t[:, 512:], torch.arange(n, dtype=torch.int32, device="cuda"))
    table = rng.permutation(pages).reshape(B, 6).astype(np.int32)
    ctx = rng.integers(4 * page, 6 * page + 1, B).astype(np.int32)
    pos = np.stack([rng.integers(0, c, k) for c in ctx]).astype(np.int32)
    pos[0, -1] = ctx[0] - 1
    got = bits(kv.read(i32(table), i32(ctx), i32(pos)))
    assert kv.synchronize() == 0
    for b in range(B):
        for j in range(k):
            slot = table[b, pos[b, j] // page] * page + pos[b, j] % page
            want = oracle.unpack_row(oracle.pack_row(x[slot], fmt), fmt)
            assert np.array_equal(bf16_bits_to_f64(got[b, j]), want), (b, j)


@pytest.mark.parametrize("fmt", FORMATS)
def test_read_leaves_bad_positions_alone(d, fmt):
    kv = d.PagedKV(4, 16, fmt)
    table, ctx = i32([[0, 4, -1], [3, 2, 1]]), i32([48, 1000])
    pos = i32([[0, 47, 16, 48, -1], [0, 15, 16, 47, 48]])
    out = torch.full((2, 5, 576), 7.0, dtype=torch.bfloat16, device="cuda")
    kv.read(table, ctx, pos, out=out)
    assert kv.synchronize() == d._abi.TS_DEVERR_SLOT_RANGE | d._abi.TS_DEVERR_ID_RANGE
    good = torch.tensor([[1, 0, 0, 0, 0], [1, 1, 1, 1, 0]], dtype=torch.bool)
    o = out.float().cpu()
    assert torch.all(o[good] == 0) and torch.all(o[~good] == 7)


def test_read_rows_feed_the_sparse_decode(d):
    # top-k of the scores, the rows read from the 8-bit pages, sparse decode
    rng = np.random.default_rng(8)
    B, k, H, page, ctx = 2, 64, 16, 32, 500
    kv = d.PagedKV(2 * 16, page, "e4m3")
    x = random_rows(rng, kv.num_slots)
    t = bf16(x)
    kv.write(t[:, :512], t[:, 512:], torch.arange(kv.num_slots, dtype=torch.int32, device="cuda"))
    table = rng.permutation(32).reshape(2, 16).astype(np.int32)
    scores = torch.from_numpy(rng.normal(0, 1, (B, 512)).astype(np.float32)).cuda()
    lens = i32([ctx, ctx - 3])
    ids = torch.empty(B, k, dtype=torch.int32, device="cuda")
    size = d.ts_topk_workspace_size(B, ctx, k)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    d.check(d.ts_topk(scores, 512, lens, B, ctx, k, ids, ws, size, kv.err))
    sel = kv.read(i32(table), lens, ids)
    q = round_to_bf16_bits(rng.normal(0, 1, (B, H, 576)))
    out = torch.empty(B, H, 512, dtype=torch.bfloat16, device="cuda")
    size = d.sfa_workspace_size(B, H, k)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    d.check(d.sfa_mla_decode(bf16(q), sel, B, H, k, 1 / 24, out, None, ws, size, kv.err))
    assert kv.synchronize() == 0
    for b in range(B):
        at = ids[b].cpu().numpy()
        slots = table[b, at // page] * page + at % page
        K = np.stack([oracle.unpack_row(oracle.pack_row(x[i], "e4m3"), "e4m3") for i in slots])
        want, _, mean_abs, size = oracle.chunk_attention(bf16_bits_to_f64(q[b:b + 1]), K, k, False,
                                                         1 / 24)
        err = np.abs(out[b].double().cpu().numpy() - want[0])
        assert np.all(err <= output_bound(want, mean_abs, size)[0])


# ---------------------------------------------------------------------------
# Chunk attention
# ---------------------------------------------------------------------------

class Chunk:
    """Requests of (new tokens, cached positions) over a cache whose unused rows
    all hold NaN bytes; every request's table row ends in invalid pages."""

    def __init__(self, d, fmt, page, H, reqs, seed=0, qsize=1.0, rows=None, pad_q=0, extra=0):
        rng = np.random.default_rng(seed)
        self.d, self.H, self.reqs, self.page = d, H, reqs, page
        B = len(reqs)
        width = max(1, max(-(-c // page) for _, c in reqs)) + 2
        pages = sum(-(-c // page) for _, c in reqs) + 3
        self.kv = d.PagedKV(pages, page, fmt)
        self.kv.data.fill_(0xFF)
        order = rng.permutation(pages)
        table = np.full((B, width), 2 ** 30, dtype=np.int32)
        self.K, slots, new, at = [], [], [], 0
        for b, (_, c) in enumerate(reqs):
            m = -(-c // page)
            table[b, :m] = order[at:at + m]
            at += m
            x = random_rows(rng, c) if rows is None else rows(rng, c)
            t = np.arange(c)
            slots.append(table[b, t // page] * page + t % page)
            new.append(x)
            self.K.append(np.stack([oracle.unpack_row(oracle.pack_row(r, fmt), fmt) for r in x])
                          if c else np.zeros((0, 576)))
        x = bf16(np.concatenate(new).reshape(-1, 576))
        self.kv.write(x[:, :512], x[:, 512:], i32(np.concatenate(slots)))
        self.table, self.ctx = i32(table), i32([c for _, c in reqs])
        self.cu = i32(np.cumsum([0] + [n for n, _ in reqs]))
        self.T = sum(n for n, _ in reqs) + extra
        q = round_to_bf16_bits(rng.normal(0, qsize, (self.T, H, 576)))
        self.q64 = bf16_bits_to_f64(q)
        wide = torch.full((self.T, H * 576 + pad_q), math.nan, dtype=torch.bfloat16, device="cuda")
        wide[:, :H * 576] = bf16(q).view(self.T, H * 576)
        self.q = wide[:, :H * 576].unflatten(1, (H, 576))

    def run(self, causal=True, scale=1 / 24, **kw):
        return self.kv.attend(self.q, self.cu, self.table, self.ctx, causal, scale, **kw)

    def check(self, out, lse, causal=True, scale=1 / 24):
        assert self.kv.synchronize() == 0
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        at = 0
        for b, (n, c) in enumerate(self.reqs):
            o, z, mean_abs, size = oracle.chunk_attention(self.q64[at:at + n], self.K[b], c, causal,
                                                          scale)
            bound = output_bound(o, mean_abs, size)
            err = np.abs(out[at:at + n] - o)
            assert np.all(err <= bound), (b, n, c, float((err / bound).max()))
            got = lse[at:at + n]
            empty = np.isneginf(z)
            assert np.array_equal(np.isneginf(got), empty)
            tol = 2 * score_error(size) + 2.0 ** -20 + 2.0 ** -22 * np.abs(np.where(empty, 0, z))
            with np.errstate(invalid="ignore"):
                assert np.all(np.where(empty, 0, np.abs(got - z)) <= tol), (b, n, c)
            at += n


LENGTHS = {
    "one": [(1, 1)],
    "decode": [(1, 1), (1, 127), (1, 128), (1, 129), (1, 700)],
    "drafts": [(4, 4), (3, 255), (2, 257), (5, 64), (1, 600)],
    "prefill": [(70, 70), (33, 300), (1, 513), (129, 260)],
    "holes": [(0, 0), (2, 40), (0, 300), (3, 0), (5, 3), (1, 129), (0, 1)],
}


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("lengths", list(LENGTHS))
@pytest.mark.parametrize("H, page", [(16, 64), (128, 16), (5, 128), (130, 32)])
def test_chunk_attention(d, fmt, lengths, H, page):
    c = Chunk(d, fmt, page, H, LENGTHS[lengths], seed=H)
    c.check(*c.run())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("H, page, reqs", [
    (1, 1024, [(1, 2500), (3, 1025)]),            # one head: a tile of tokens, large pages
    (128, 64, [(1, 5000)]),                       # one long row: split over the GPU
    (64, 64, [(1, 3000 + 37 * i) for i in range(5)]),
    (20, 16, [(200, 333)]),                       # tokens cut by tile borders
])
def test_chunk_attention_shapes(d, fmt, H, page, reqs):
    c = Chunk(d, fmt, page, H, reqs, seed=1)
    c.check(*c.run())


@pytest.mark.parametrize("fmt", FORMATS)
def test_chunk_without_causal_mask(d, fmt):
    c = Chunk(d, fmt, 32, 16, LENGTHS["drafts"] + LENGTHS["holes"], seed=2)
    c.check(*c.run(causal=False), causal=False)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("scale", [0.5, -0.3, 0.0])
def test_chunk_sharp_scores_and_other_scales(d, fmt, scale):
    # scores in the hundreds: nearly one-hot rows, running maxima far apart
    c = Chunk(d, fmt, 64, 16, [(9, 700), (2, 140)], seed=3, qsize=3.0)
    c.check(*c.run(scale=scale), scale=scale)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("order", [1, -1])
def test_chunk_running_maximum_moves_in_every_tile(d, fmt, order):
    # keys along one direction, growing (or shrinking) with their position
    def rows(rng, c):
        x = 0.05 * rng.normal(0, 1, (c, 576)) + np.linspace(-1, 1, max(c, 1))[::order][:c, None]
        return round_to_bf16_bits(x)
    c = Chunk(d, fmt, 64, 16, [(3, 1500), (40, 640)], seed=4, rows=rows)
    c.q[...] = c.q.abs()
    c.q64 = np.abs(c.q64)
    c.check(*c.run(scale=1.0), scale=1.0)


@pytest.mark.parametrize("fmt", FORMATS)
def test_chunk_strided_queries_and_untouched_rows(d, fmt):
    # tokens further apart than their heads; rows past cu_q[B] stay as they were
    c = Chunk(d, fmt, 64, 20, [(7, 90), (2, 300)], seed=5, pad_q=64, extra=5)
    out = torch.full((c.T, 20, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((c.T, 20), 5.0, device="cuda")
    o, z = c.run(out=out, lse=lse)
    assert o is out and z is lse
    c.check(out, lse)
    assert torch.all(out[9:] == 3) and torch.all(lse[9:] == 5)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("ctx", [200, 9000])   # a row tile by itself; one that is joined
def test_chunk_a_nan_in_a_query_stays_in_its_row(d, fmt, ctx):
    c = Chunk(d, fmt, 64, 20, [(3, ctx)], seed=23)
    want, want_lse = [x.clone() for x in c.run()]
    c.q[1, 7, 100] = math.nan
    out, lse = c.run()
    assert c.kv.synchronize() == 0
    row = torch.zeros(3, 20, dtype=torch.bool, device="cuda")
    row[1, 7] = True
    assert torch.all(torch.isnan(out[row])) and torch.all(torch.isnan(lse[row]))
    assert torch.equal(out[~row], want[~row]) and torch.equal(lse[~row], want_lse[~row])


@pytest.mark.parametrize("fmt", FORMATS)
def test_chunk_large_and_small_latent_groups(d, fmt):
    # groups of 128 whose scales lie far apart: 2^13 and more beside 2^-40 (the
    # scores' weights fall on the last group and the rope part)
    def rows(rng, n):
        x = bf16_bits_to_f64(random_rows(rng, n))
        x[:, :128] *= 2.0 ** 20
        x[:, 128:256] *= 2.0 ** -40
        return round_to_bf16_bits(x)
    c = Chunk(d, fmt, 64, 16, [(3, 700), (1, 70)], seed=24, rows=rows)
    c.q64[:, :, :128] = 0
    c.q[:, :, :128] = 0
    c.check(*c.run())


def test_chunk_without_lse(d):
    c = Chunk(d, "bf16", 64, 16, [(3, 200)], seed=6)
    want, lse = c.run()
    out = torch.zeros_like(want)
    ws = c.kv.workspace(c.T, 1, 16)
    d.check(d.sfa_mla_chunk(c.q, c.q.stride(0), c.cu, c.T, 1, 16, c.kv.data, c.kv.num_slots,
                            d.DSA_CACHE_BF16, c.table, c.table.shape[1], 64, c.ctx, 1, 1 / 24, out,
                            None, ws, ws.numel(), c.kv.err))
    c.check(out, lse)
    assert torch.equal(out, want)


def test_chunk_is_deterministic(d):
    c = Chunk(d, "e4m3", 64, 64, [(1, 3000), (5, 777), (64, 300)], seed=7)
    first = [x.clone() for x in c.run()]
    for _ in range(5):
        again = c.run()
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_attention_over_8_bit_rows_equals_attention_over_their_read_back(d):
    c = Chunk(d, "e4m3", 64, 32, [(3, 900), (1, 130)], seed=8)
    out, lse = c.run()
    other = d.PagedKV(c.kv.num_pages, 64, "bf16")
    for b, (_, n) in enumerate(c.reqs):
        t = torch.arange(n, device="cuda", dtype=torch.int32)
        rows = c.kv.read(c.table[b:b + 1].contiguous(), c.ctx[b:b + 1], t[None].contiguous())[0]
        slots = c.table[b].long()[t.long() // 64] * 64 + t.long() % 64
        other.write(rows[:, :512], rows[:, 512:], slots.int())
    o2, l2 = other.attend(c.q, c.cu, c.table, c.ctx, True, 1 / 24)
    assert other.synchronize() == 0 and c.kv.synchronize() == 0
    assert torch.equal(out, o2) and torch.equal(lse, l2)


@pytest.mark.parametrize("fmt", FORMATS)
def test_chunk_reports_bad_lengths_and_pages(d, fmt):
    abi = d._abi
    c = Chunk(d, fmt, 16, 16, [(2, 40), (3, 64)], seed=9)
    ctx = c.ctx.clone()
    ctx[0] = -4                                          # taken as 0: an empty request
    out, lse = c.kv.attend(c.q, c.cu, c.table, ctx, True, 1 / 24)
    assert c.kv.synchronize() == abi.TS_DEVERR_CTX
    assert torch.all(out[:2] == 0) and torch.all(torch.isneginf(lse[:2]))
    good, _ = c.run()
    assert torch.equal(out[2:], good[2:])
    table = c.table.clone()
    table[0, 1] = c.kv.num_pages                         # just past the cache
    out, _ = c.kv.attend(c.q, c.cu, table, c.ctx, True, 1 / 24)
    assert c.kv.synchronize() == abi.TS_DEVERR_SLOT_RANGE
    assert torch.equal(out[2:], good[2:])
    table[0, 1] = -1
    c.kv.attend(c.q, c.cu, table, c.ctx, True, 1 / 24)
    assert c.kv.synchronize() == abi.TS_DEVERR_SLOT_RANGE
    cu = c.cu.clone()
    cu[2] = 50                                           # past T: taken as T
    out, _ = c.kv.attend(c.q, cu, c.table, c.ctx, True, 1 / 24)
    assert c.kv.synchronize() == abi.TS_DEVERR_ORDER
    assert torch.equal(out, good)


def test_chunk_context_past_the_table_is_refused_on_the_device(d):
    c = Chunk(d, "bf16", 16, 16, [(1, 40)], seed=10)
    table = c.table[:, :3].contiguous()
    ctx = i32([49])
    c.kv.attend(c.q, c.cu, table, ctx, True, 1 / 24)
    assert c.kv.synchronize() & d._abi.TS_DEVERR_CTX


def test_chunk_in_a_captured_graph_follows_its_inputs(d):
    c = Chunk(d, "bf16", 64, 16, [(2, 700), (1, 300)], seed=11)
    out = torch.empty(c.T, 16, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(c.T, 16, device="cuda")
    ws = c.kv.workspace(c.T, 2, 16)
    c.run(out=out, lse=lse, ws=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run(out=out, lse=lse, ws=ws)
    for lens in [(700, 300), (65, 2), (129, 1), (700, 0)]:
        c.ctx.copy_(i32(lens))
        keep, c.K = c.K, [k[:n] for k, n in zip(c.K, lens)]
        c.reqs = list(zip((2, 1), lens))
        g.replay()
        c.check(out, lse)
        c.K = keep


def test_chunks_on_two_streams_at_once(d):
    cs = [Chunk(d, f, 64, 64, [(1, 2000), (9, 500)], seed=12 + i) for i, f in enumerate(FORMATS)]
    want = [[x.clone() for x in c.run()] for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    got = [[] for _ in cs]
    for _ in range(10):
        for i, c in enumerate(cs):
            got[i].append(c.run(stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(len(cs)):
        for o, z in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(z, want[i][1])


def test_chunk_graphs_with_their_own_workspaces_replay_side_by_side(d):
    cs = [Chunk(d, f, 64, 32, [(2, 1500), (5, 300), (1, 40)], seed=20 + i)
          for i, f in enumerate(FORMATS)]
    runs = []
    for c in cs:
        out = torch.empty(c.T, 32, 512, dtype=torch.bfloat16, device="cuda")
        lse = torch.empty(c.T, 32, device="cuda")
        ws = c.kv.workspace(c.T, 3, 32)
        want = [x.clone() for x in c.run(out=out, lse=lse, ws=ws)]
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run(out=out, lse=lse, ws=ws)
        runs.append((g, out, lse, ws, want))
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(5):
        for _, out, lse, _, _ in runs:
            out.fill_(7)
            lse.fill_(7)
        torch.cuda.synchronize()
        for (g, *_), s in zip(runs, streams):
            with torch.cuda.stream(s):
                for _ in range(3):
                    g.replay()
        torch.cuda.synchronize()
        for _, out, lse, _, want in runs:
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("fmt", FORMATS)
def test_chunk_more_requests_than_threads(d, fmt):
    # 1100 requests, every third without a token, every fifth without a context
    reqs = [(0 if i % 3 == 0 else 1 + i % 2, 0 if i % 5 == 0 else 1 + i * 37 % 290)
            for i in range(1100)]
    c = Chunk(d, fmt, 32, 8, reqs, seed=21)
    c.check(*c.run())


@pytest.mark.parametrize("fmt", FORMATS)
def test_chunk_wait_that_runs_out_reports_and_recovers(d, fmt):
    # with a limit of 1 ns the waits give up at once: the call reports it, lets
    # its copies land, frees its tensor memory, and the next call computes
    c = Chunk(d, fmt, 64, 128, [(1, 3000), (9, 500)], seed=22)
    d.ts_set_wait_limit_ns(1)
    try:
        c.run()
        bits = c.kv.synchronize()
    finally:
        d.ts_set_wait_limit_ns(0)
    assert bits == d._abi.TS_DEVERR_TIMEOUT
    for _ in range(2):
        c.check(*c.run())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("H", [1000, 1024])
def test_chunk_most_heads(d, fmt, H):
    c = Chunk(d, fmt, 64, H, [(2, 70), (1, 300)], seed=25)
    c.check(*c.run())


@pytest.mark.parametrize("fmt", FORMATS)
def test_chunk_tokens_before_the_first_request(d, fmt):
    # cu_q starting above 0: the tokens before it are nobody's
    c = Chunk(d, fmt, 32, 20, [(3, 200), (2, 90)], seed=26, extra=4)
    c.check(*c.run())
    want, want_lse = [x.clone() for x in c.run()]
    q = torch.cat([c.q[-4:], c.q[:-4]])
    out = torch.full_like(want, 3.0)
    lse = torch.full_like(want_lse, 5.0)
    c.kv.attend(q, c.cu + 4, c.table, c.ctx, True, 1 / 24, out=out, lse=lse)
    assert c.kv.synchronize() == 0
    assert torch.all(out[:4] == 3) and torch.all(lse[:4] == 5)
    assert torch.equal(out[4:], want[:-4]) and torch.equal(lse[4:], want_lse[:-4])


@pytest.mark.parametrize("fmt", FORMATS)
def test_chunk_requests_that_share_pages(d, fmt):
    c = Chunk(d, fmt, 64, 16, [(2, 500), (2, 500), (2, 500)], seed=27)
    c.table[1] = c.table[0]
    c.table[2, :4] = c.table[0, :4]
    c.K[1] = c.K[0]
    c.K[2] = np.concatenate([c.K[0][:256], c.K[2][256:]])
    c.check(*c.run())


def test_chunk_first_call_of_a_process_inside_a_capture():
    # the launch limits and the tensor maps' encoder are set up by the first call
    code = """
import torch, decode_dsa_kv_gb300 as d
for fmt in ("bf16", "e4m3"):
    kv = d.PagedKV(4, 64, fmt)
    kv.data.zero_()
    table = torch.arange(4, dtype=torch.int32, device="cuda").view(1, 4)
    cu = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    ctx = torch.tensor([200], dtype=torch.int32, device="cuda")
    q = torch.randn(2, 16, 576, device="cuda").bfloat16()
    out = torch.full((2, 16, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(2, 16, device="cuda")
    ws = kv.workspace(2, 1, 16)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kv.attend(q, cu, table, ctx, out=out, lse=lse, ws=ws)
    g.replay()
    assert kv.synchronize() == 0
    assert torch.all(out == 0)
    want = torch.log(torch.tensor([[199.0], [200.0]], device="cuda")).expand(2, 16)
    assert torch.allclose(lse, want, rtol=0, atol=2.0 ** -18)
print("done")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and "done" in r.stdout, r.stderr


def test_cache_past_32_bit_offsets(d):
    # slots whose byte offsets (and 16-byte offsets) pass 2^32
    rng = np.random.default_rng(14)
    pages = (9 << 30) // (64 * 1152)
    kv = d.PagedKV(pages, 64, "bf16")
    last = np.array([[pages - 1, pages - 2, 1, pages // 2]], dtype=np.int32)
    x = random_rows(rng, 250)
    t = np.arange(250)
    slots = last[0, t // 64] * 64 + t % 64
    xt = bf16(x)
    kv.write(xt[:, :512], xt[:, 512:], i32(slots))
    got = bits(kv.read(i32(last), i32([250]), i32(t[None])))
    assert np.array_equal(got[0], x)
    q = round_to_bf16_bits(rng.normal(0, 1, (2, 16, 576)))
    out, _ = kv.attend(bf16(q), i32([0, 2]), i32(last), i32([250]), True, 1 / 24)
    assert kv.synchronize() == 0
    small = d.PagedKV(4, 64, "bf16")
    small.write(xt[:, :512], xt[:, 512:], i32(t))
    want, _ = small.attend(bf16(q), i32([0, 2]), i32([[0, 1, 2, 3]]), i32([250]), True, 1 / 24)
    assert torch.equal(out, want)


# ---------------------------------------------------------------------------
# Draft verification
# ---------------------------------------------------------------------------

def distributions(rng, shape, V, sharp):
    x = rng.normal(0, sharp, (*shape, V))
    x = np.exp(x - x.max(axis=-1, keepdims=True))
    return (x / x.sum(axis=-1, keepdims=True)).astype(np.float32)


def cuda(x):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()


@pytest.mark.parametrize("V", [1, 2, 33, 4095, 4097, 40001])
@pytest.mark.parametrize("n, certain", [(0, True), (1, False), (3, False), (3, True), (9, False)])
def test_verify_equals_the_oracle(d, V, n, certain):
    rng = np.random.default_rng(V + n)
    B = 7
    p = distributions(rng, (B, n + 1), V, 1.0)
    q = None
    x = rng.integers(0, V, (B, n)).astype(np.int32)
    if not certain:
        q = p[:, :n] * np.exp(rng.normal(0, 0.3, (B, n, V)))
        q = (q / np.maximum(q.sum(axis=-1, keepdims=True), 1e-30)).astype(np.float32)
    u = rng.random((B, n + 1)).astype(np.float32)
    u[0] = 0.0                                           # everything with p > 0 is accepted
    u[1, :] = np.float32(1 - 2.0 ** -24)
    u[2, :n] = 0.0
    nd = rng.integers(0, n + 1, B).astype(np.int32)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for counts in (None, nd):
        tokens, accepted = d.verify_drafts(cuda(x), cuda(p), cuda(q), cuda(u), cuda(counts), err)
        assert d.ts_read_error(err) == 0
        for b in range(B):
            want, a = oracle.verify_drafts(x[b], n if counts is None else int(nd[b]), p[b],
                                           None if q is None else q[b], u[b])
            assert int(accepted[b]) == a and tokens[b].tolist() == want, b


def test_verify_rows_with_strides_and_without_weight(d):
    V, n, B = 1001, 2, 3
    rng = np.random.default_rng(1)
    p, q = distributions(rng, (B, n + 1), V, 1.0), distributions(rng, (B, n), V, 1.0)
    q[0, 0] = p[0, 0]                      # no residual: p itself
    x = np.array([[5, 6], [V, 6], [7, -1]], dtype=np.int32)
    u = np.full((B, n + 1), 0.999, dtype=np.float32)
    u[2, 0] = 0.0
    q[0, 0, 5], p[0, 0, 5] = 0.25, 0.0     # certain to be refused
    tp = torch.full((B, n + 1, V + 7), math.nan, device="cuda")
    tp[..., :V] = cuda(p)
    tq = torch.full((B, n, V + 3), math.nan, device="cuda")
    tq[..., :V] = cuda(q)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    tokens, accepted = d.verify_drafts(cuda(x), tp[..., :V], tq[..., :V], cuda(u), None, err)
    assert d.ts_read_error(err) == d._abi.TS_DEVERR_ID_RANGE
    for b in range(B):
        want, a = oracle.verify_drafts(x[b], n, p[b], q[b], u[b])
        assert int(accepted[b]) == a and tokens[b].tolist() == want, b


def test_verify_rows_of_a_larger_tensor(d):
    # one row a request, the requests further apart than the row
    V, B = 700, 3
    rng = np.random.default_rng(2)
    p = distributions(rng, (B, 4), V, 1.0)
    u = rng.random((B, 1)).astype(np.float32)
    none = torch.empty(B, 0, dtype=torch.int32, device="cuda")
    tokens, accepted = d.verify_drafts(none, cuda(p)[:, 1:2], None, cuda(u))
    for b in range(B):
        want, a = oracle.verify_drafts(np.zeros(0, np.int32), 0, p[b, 1:2], None, u[b])
        assert int(accepted[b]) == a == 0 and tokens[b].tolist() == want


def test_verify_large_vocabulary_for_many_requests(d):
    # more requests than SMs, and more tiles than one block has sums for
    B, V = 160, 1_500_001
    target = torch.zeros(B, 1, V, device="cuda")
    at = torch.arange(B, device="cuda") * 9001 % (V - 1)
    rows = torch.arange(B, device="cuda")
    target[rows, 0, at] = 0.25
    target[rows, 0, V - 1] = 0.75
    u = torch.where(rows % 2 == 0, 0.24, 0.26).float().view(B, 1)
    none = torch.empty(B, 0, dtype=torch.int32, device="cuda")
    tokens, accepted = d.verify_drafts(none, target, None, u)
    want = torch.where(rows % 2 == 0, at, V - 1)
    assert torch.equal(tokens[:, 0].long(), want) and torch.all(accepted == 0)


def test_verify_reports_bad_probabilities(d):
    V = 300
    p = np.full((4, 1, V), 1 / V, dtype=np.float32)
    p[0, 0, 3], p[1, 0, 4], p[2, 0, 5] = math.nan, -0.1, 2.0
    p[3] = 0
    u = np.full((4, 1), 0.5, dtype=np.float32)
    for b in range(4):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        tokens, accepted = d.verify_drafts(torch.zeros(1, 0, dtype=torch.int32, device="cuda"),
                                           cuda(p[b:b + 1]), None, cuda(u[b:b + 1]), None, err)
        assert d.ts_read_error(err) == d._abi.TS_DEVERR_PROB
        want, _ = oracle.verify_drafts([], 0, p[b], None, u[b])
        assert tokens[0].tolist() == want and int(accepted[0]) == 0


# ---------------------------------------------------------------------------
# Together
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", FORMATS)
def test_speculative_decoding_steps(d, fmt):
    """Prefill in two chunks, then steps of drafting, writing the drafts' rows,
    attending and verifying; refused drafts' rows are overwritten by the next
    step. The cache's contents are followed on the host."""
    rng = np.random.default_rng(20)
    B, H, n, V, page, width = 3, 16, 3, 50, 16, 12
    kv = d.PagedKV(B * width, page, fmt)
    table = rng.permutation(B * width).reshape(B, width).astype(np.int32)
    rows = [np.zeros((0, 576), dtype=np.uint16) for _ in range(B)]

    def append(counts):
        """New rows for every request behind its valid ones, and the attention over them."""
        new = [random_rows(rng, c) for c in counts]
        where = []
        for b, c in enumerate(counts):
            t = len(rows[b]) + np.arange(c)
            where.append(table[b, t // page] * page + t % page)
            rows[b] = np.concatenate([rows[b], new[b]])
        x = bf16(np.concatenate(new))
        kv.write(x[:, :512], x[:, 512:], i32(np.concatenate(where)))
        q = round_to_bf16_bits(rng.normal(0, 1, (sum(counts), H, 576)))
        out, _ = kv.attend(bf16(q), i32(np.cumsum([0] + list(counts))), i32(table),
                           i32([len(r) for r in rows]), True, 1 / 24)
        assert kv.synchronize() == 0
        got, at = out.double().cpu().numpy(), 0
        for b, c in enumerate(counts):
            K = np.stack([oracle.unpack_row(oracle.pack_row(r, fmt), fmt) for r in rows[b]])
            want, _, mean_abs, size = oracle.chunk_attention(bf16_bits_to_f64(q[at:at + c]), K,
                                                             len(K), True, 1 / 24)
            bound = output_bound(want, mean_abs, size)
            assert np.all(np.abs(got[at:at + c] - want) <= bound), (b, c)
            at += c
        return got

    append([40, 7, 1])
    append([5, 30, 70])
    for _ in range(4):
        append([n + 1] * B)                               # the last token and n drafts
        p, q = distributions(rng, (B, n + 1), V, 0.3), distributions(rng, (B, n), V, 0.3)
        x = rng.integers(0, V, (B, n)).astype(np.int32)
        u = rng.random((B, n + 1)).astype(np.float32)
        tokens, accepted = d.verify_drafts(cuda(x), cuda(p), cuda(q), cuda(u))
        for b in range(B):
            want, a = oracle.verify_drafts(x[b], n, p[b], q[b], u[b])
            assert tokens[b].tolist() == want and int(accepted[b]) == a
            rows[b] = rows[b][:len(rows[b]) - n + a]      # the refused drafts' rows go
