"""Trees and beams over the paged cache on the GPU, against their oracle in 64
bits: plans, turned rows and queries, tree attention, the verified walk, rows
kept, beams, forks; bad data reported and skipped; graphs, streams, and runs of
them together."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

import oracle  # noqa: E402
from oracle import candidates as oc  # noqa: E402
from oracle.sfa import bf16_bits_to_f64, round_to_bf16_bits  # noqa: E402
from test_gpu_paged import (BF16_HALF_STEP, bf16, bits, i32, output_bound, random_rows,  # noqa: E402
                            score_error)

FORMATS = ["bf16", "e4m3"]
FREQ = 10000.0 ** (-np.arange(32) / 32)


@pytest.fixture(scope="module")
def d():
    import decode_dsa_kv_gb300 as mod
    return mod


def forest(rng, n, roots=1):
    return [-1 if i < roots else int(rng.integers(max(-1, i - 9), i)) for i in range(n)]


def table_of(rng, ctx, page, extra=3):
    """A block table [B][..] over pages in random order, rows ending in bad pages."""
    used = [-(-c // page) for c in ctx]
    pages = sum(used) + extra
    table = np.full((len(ctx), max(used) + 2), 2 ** 30, dtype=np.int32)
    order, at = rng.permutation(pages), 0
    for b, m in enumerate(used):
        table[b, :m] = order[at:at + m]
        at += m
    return table, pages, order[at:]


def slot_of(table, page, b, t):
    return int(table[b, t // page]) * page + t % page


# ---------------------------------------------------------------------------
# Plans
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("sizes, most", [([1], 1), ([31, 32, 33], 64), ([64, 0, 1, 5], 64),
                                         ([1024, 2], 1024), ([40, 7], 16), ([100], 128)])
@pytest.mark.parametrize("chains", [False, True])
def test_plan(d, sizes, most, chains):
    rng = np.random.default_rng(sum(sizes))
    B, page, words = len(sizes), 16, -(-most // 32)
    ctx = [n + int(rng.integers(0, 50)) for n in sizes]
    table, pages, _ = table_of(rng, [max(c, 1) for c in ctx], page)
    parents = [list(range(-1, n - 1)) if chains else forest(rng, n, 2) for n in sizes]
    lead, tail = 2, 3                              # tokens that no request has, at both ends
    T = lead + sum(sizes) + tail
    flat = np.concatenate([np.full(lead, 77)] + parents + [np.full(tail, -9)]).astype(np.int32)
    kv = d.PagedKV(pages, page)
    cu = i32(lead + np.cumsum([0] + sizes))
    pos, slots, mask = kv.plan_tree(None if chains else i32(flat), cu, i32(table), i32(ctx), T, most)
    want_bits = d._abi.TS_DEVERR_COUNT if max(sizes) > 32 * words else 0
    assert kv.synchronize() == want_bits
    want_pos, want_slots = np.zeros(T, np.int32), np.full(T, -1, np.int32)
    want_mask = np.zeros((T, words), np.uint32)
    at = lead
    for b, n in enumerate(sizes):
        if n:
            want_pos[at:at + n] = ctx[b] - n + np.array(oc.depths(parents[b]))
            want_slots[at:at + n] = [slot_of(table, page, b, ctx[b] - n + i) for i in range(n)]
            want_mask[at:at + n] = oc.mask_words(oc.sees(parents[b]), words)
        at += n
    assert np.array_equal(pos.cpu().numpy(), want_pos)
    assert np.array_equal(slots.cpu().numpy(), want_slots)
    assert np.array_equal(mask.cpu().numpy().view(np.uint32), want_mask)


def test_plan_reports_what_is_wrong(d):
    e = d._abi
    kv = d.PagedKV(8, 16)
    table, ctx = i32([[0, 1, 2, 99], [3, 4, -1, 5]]), i32([60, 40])
    pos, slots, mask = kv.plan_tree(i32([-1, 5, 1, -2, 0, 1]), i32([0, 4, 6]), table, ctx, 6, 4)
    assert kv.synchronize() == e.TS_DEVERR_PARENT | e.TS_DEVERR_SLOT_RANGE
    assert pos.tolist() == [56, 56, 57, 56, 38, 38]
    assert mask.view(-1).tolist() == [1, 2, 6, 8, 1, 2]
    assert slots.tolist() == [-1] * 6              # (pages 99 and -1)
    _, slots, _ = kv.plan_tree(None, i32([0, 3, 2]), table, i32([16, 16]), 4, 4)
    assert kv.synchronize() == e.TS_DEVERR_ORDER
    assert slots.tolist()[:3] == [13, 14, 15]
    _, slots, _ = kv.plan_tree(None, i32([0, 3, 4]), table, i32([2, 70]), 4, 4)
    assert kv.synchronize() == e.TS_DEVERR_CTX     # fewer than the nodes; past the table (64)
    assert slots.tolist() == [-1, 0, 1, 5 * 16 + 15]
    many = 1026
    parent = torch.full((many,), -1, dtype=torch.int32, device="cuda")
    kv = d.PagedKV(80, 16)
    pos, slots, mask = kv.plan_tree(parent, i32([0, many]), i32([list(range(70))]), i32([1100]), many,
                                    1024)
    assert kv.synchronize() == e.TS_DEVERR_COUNT
    assert slots[1023] == 1100 - many + 1023 and slots[1024:].tolist() == [-1, -1]
    assert not mask[1024:].any()


# ---------------------------------------------------------------------------
# Appending
# ---------------------------------------------------------------------------

def check_turned(got, x, pos, interleaved):
    """bf16 values [..][64] of one position against x turned."""
    y = oc.turn(x, pos, FREQ, interleaved)
    size = np.abs(oc.turn(np.abs(x), 0, FREQ, interleaved))
    a, b = (size[..., 0::2], size[..., 1::2]) if interleaved else (size[..., :32], size[..., 32:])
    both = np.repeat(a + b, 2, axis=-1) if interleaved else np.concatenate([a + b, a + b], -1)
    # the angle's rounding to fp32 (2^-25 of a turn and what precedes it, below
    # 2^-26), sine and cosine (2^-23) and three roundings of the sum: 2^-21 of
    # |a| + |b| in all; then the rounding to bf16
    bound = 2.0 ** -21 * both + 1.01 * BF16_HALF_STEP * np.abs(y) + 2.0 ** -130
    assert np.all(np.abs(got - y) <= bound)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("n, H, fused", [(1, 16, False), (5, 1, True), (33, 17, True), (9, 128, False),
                                         (3, 200, True), (40, 0, False)])
def test_append(d, fmt, interleaved, n, H, fused):
    rng = np.random.default_rng(n + H)
    x = random_rows(rng, n)
    t = bf16(x)
    wide = torch.full((n, 640), math.nan, dtype=torch.bfloat16, device="cuda")
    wide[:, 8:520], wide[:, 528:592] = t[:, :512], t[:, 512:]
    latent, rope = ((wide[:, 8:520], wide[:, 528:592]) if fused
                    else (t[:, :512].contiguous(), t[:, 512:].contiguous()))
    pos = rng.integers(0, 200000, n).astype(np.int32)
    pos[0] = 2 ** 27 - 1
    if n > 2:
        pos[1], pos[2] = 0, -5
    kv = d.PagedKV(40, 16, fmt)
    kv.data.fill_(0xA5)
    slots = rng.permutation(kv.num_slots)[:n].astype(np.int32)
    given = slots.copy()
    skipped = n // 4
    given[n - skipped:] = -1 - np.arange(skipped)
    args, q = {}, None
    if H:
        qr = round_to_bf16_bits(rng.normal(0, 2, (n, H, 64)))
        q = torch.full((n, H * 576 + 8), 3.0, dtype=torch.bfloat16, device="cuda")
        part = torch.full((n, H, 192 if fused else 64), math.nan, dtype=torch.bfloat16, device="cuda")
        part[:, :, -64:] = bf16(qr)
        args = dict(q=q[:, :H * 576].unflatten(1, (H, 576)), q_rope=part[:, :, -64:])
    kv.append(latent, rope, i32(pos), i32(given), torch.from_numpy(FREQ).cuda(),
              interleaved=interleaved, **args)
    assert kv.synchronize() == 0
    got = kv.data.cpu().numpy()
    untouched = np.ones(kv.num_slots, bool)
    untouched[slots[:n - skipped]] = False
    assert np.all(got[untouched] == 0xA5)
    split = 1024 if fmt == "bf16" else 528
    for i in range(n - skipped):
        row = got[slots[i]]
        assert np.array_equal(row[:split], oracle.pack_row(x[i], fmt)[:split])
        check_turned(bf16_bits_to_f64(row[split:].copy().view(np.uint16)),
                     bf16_bits_to_f64(x[i, 512:]), int(pos[i]), interleaved)
    if H:
        qs = q.cpu()
        assert torch.all(qs[:, H * 576:] == 3)
        qs = qs[:, :H * 576].unflatten(1, (H, 576))
        assert torch.all(qs[:, :, :512] == 3)
        for i in range(n):                         # (a skipped row's queries too)
            check_turned(qs[i, :, 512:].double().numpy(), bf16_bits_to_f64(qr[i]), int(pos[i]),
                         interleaved)


def test_append_in_place_and_past_the_cache(d):
    rng = np.random.default_rng(3)
    n, H = 4, 20
    t = bf16(random_rows(rng, n))
    q = bf16(round_to_bf16_bits(rng.normal(0, 1, (n, H, 576))))
    other = q.clone()
    freq, pos = torch.from_numpy(FREQ).cuda(), i32([5, 6, 7, 100000])
    kv = d.PagedKV(2, 16)
    kv.append(t[:, :512], t[:, 512:], pos, i32([0, 31, 32, 2 ** 31 - 1]), freq, q[:, :, 512:], q)
    assert kv.synchronize() == d._abi.TS_DEVERR_SLOT_RANGE
    kv2 = d.PagedKV(2, 16)
    out = torch.zeros_like(other)
    kv2.append(t[:, :512], t[:, 512:], pos, i32([0, 31, -1, -1]), freq,
               other[:, :, 512:].contiguous(), out)
    assert kv2.synchronize() == 0
    assert torch.equal(q[:, :, 512:], out[:, :, 512:]) and torch.equal(q[:, :, :512], other[:, :, :512])
    assert torch.equal(kv.data, kv2.data)


def test_append_at_position_zero_is_write(d):
    rng = np.random.default_rng(4)
    n = 50
    t = bf16(random_rows(rng, n))
    t[3, 515], t[4, 20] = math.inf, math.nan
    for fmt in FORMATS:
        a, b = d.PagedKV(4, 16, fmt), d.PagedKV(4, 16, fmt)
        where = torch.randperm(64, device="cuda")[:n].to(torch.int32)
        a.write(t[:, :512], t[:, 512:], where)
        # (angle 0: cos 1, sin 0; infinity times 0 is no number, so row 3 differs)
        b.append(t[:, :512], t[:, 512:], torch.zeros(n, dtype=torch.int32, device="cuda"), where,
                 torch.from_numpy(FREQ).cuda())
        same = (a.data == b.data).all(1)
        same[where[3].long()] = True
        assert torch.all(same)


# ---------------------------------------------------------------------------
# Tree attention
# ---------------------------------------------------------------------------

class Trees:
    """Requests of (nodes, cached positions, the nodes among them) over a cache
    whose other rows all hold NaN bytes. `seen`: which nodes each node sees."""

    def __init__(self, d, fmt, page, H, reqs, seed=0, seen=None, extra=0, words=None, pad_q=0):
        rng = np.random.default_rng(seed)
        self.d, self.H, self.reqs = d, H, reqs
        ctx = [c for _, c in reqs]
        table, pages, _ = table_of(rng, [max(c, 1) for c in ctx], page)
        self.kv = d.PagedKV(pages, page, fmt)
        self.kv.data.fill_(0xFF)
        self.K, rows, slots = [], [], []
        for b, c in enumerate(ctx):
            x = random_rows(rng, c)
            rows.append(x)
            slots += [slot_of(table, page, b, t) for t in range(c)]
            self.K.append(np.stack([oracle.unpack_row(oracle.pack_row(r, fmt), fmt) for r in x])
                          if c else np.zeros((0, 576)))
        t = bf16(np.concatenate(rows).reshape(-1, 576))
        self.kv.write(t[:, :512], t[:, 512:], i32(slots))
        most = max(n for n, _ in reqs)
        self.seen = [oc.sees(forest(rng, n, 2 if n > 1 else 1)) if seen is None else seen(rng, n)
                     for n, _ in reqs]
        words = words or -(-max(most, 1) // 32)
        self.T = sum(n for n, _ in reqs) + extra
        mask = np.concatenate([oc.mask_words(s, words) for s in self.seen if len(s)]
                              + [np.full((extra, words), 0xffffffff, np.uint32)])
        self.mask = i32(mask.view(np.int32))
        q = round_to_bf16_bits(rng.normal(0, 1.5, (self.T, H, 576)))
        self.q64 = bf16_bits_to_f64(q)
        wide = torch.full((self.T, H * 576 + pad_q), math.nan, dtype=torch.bfloat16, device="cuda")
        wide[:, :H * 576] = bf16(q).view(self.T, H * 576)
        self.q = wide[:, :H * 576].unflatten(1, (H, 576))
        self.cu, self.ctx = i32(np.cumsum([0] + [n for n, _ in reqs])), i32(ctx)
        self.table = i32(table)

    def run(self, scale=1 / 24, **kw):
        return self.kv.attend(self.q, self.cu, self.table, self.ctx, scale=scale, tree=self.mask, **kw)

    def check(self, out, lse, scale=1 / 24, every=1):
        assert self.kv.synchronize() == 0
        out, lse, at = out.double().cpu().numpy(), lse.double().cpu().numpy(), 0
        for b, (n, c) in enumerate(self.reqs):
            for i in range(0, n, every):
                rows = np.concatenate([np.ones(c - n, bool), self.seen[b][i]])
                K = self.K[b][rows]
                o, z, mean_abs, size = oracle.chunk_attention(self.q64[at + i:at + i + 1], K, len(K),
                                                              False, scale)
                bound = output_bound(o, mean_abs, size)
                err = np.abs(out[at + i:at + i + 1] - o)
                assert np.all(err <= bound), (b, i, float((err / bound).max()))
                empty = np.isneginf(z)
                got = lse[at + i:at + i + 1]
                assert np.array_equal(np.isneginf(got), empty)
                tol = 2 * score_error(size) + 2.0 ** -20 + 2.0 ** -22 * np.abs(np.where(empty, 0, z))
                with np.errstate(invalid="ignore"):
                    assert np.all(np.where(empty, 0, np.abs(got - z)) <= tol), (b, i)
            at += n


SHAPES = {
    "one": [(1, 1)],
    "small": [(3, 3), (5, 40), (1, 256), (2, 257), (16, 300)],
    "bits": [(33, 33), (64, 400), (31, 257), (32, 288), (65, 512)],
    "holes": [(0, 30), (4, 260), (0, 0), (7, 7), (12, 255)],
}


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("shape", list(SHAPES))
@pytest.mark.parametrize("H, page", [(16, 64), (128, 16), (5, 128), (77, 32)])
def test_tree_attention(d, fmt, shape, H, page):
    c = Trees(d, fmt, page, H, SHAPES[shape], seed=H)
    c.check(*c.run())


@pytest.mark.parametrize("fmt", FORMATS)
def test_tree_attention_with_any_mask(d, fmt):
    # random bits (nodes that do not see themselves, or see later ones), rows that
    # see nothing at all, more words than the nodes need, tokens of no request
    def random_bits(rng, n):
        s = rng.random((n, n)) < 0.4
        s[::3] = False
        return s
    c = Trees(d, fmt, 32, 24, [(40, 40), (9, 9), (70, 330), (3, 200)], seed=2, seen=random_bits,
              extra=3, words=4)
    out = torch.full((c.T, 24, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((c.T, 24), 7.0, device="cuda")
    c.check(*c.run(out=out, lse=lse))
    assert torch.all(out[-3:] == 7) and torch.all(lse[-3:] == 7)
    assert torch.all(out[:40:3] == 0) and torch.all(torch.isneginf(lse[:40:3]))


@pytest.mark.parametrize("fmt", FORMATS)
def test_tree_attention_of_chains_is_the_causal_one(d, fmt):
    c = Trees(d, fmt, 64, 32, [(5, 300), (1, 77), (33, 600)], seed=3,
              seen=lambda rng, n: np.tri(n, dtype=bool), pad_q=64)
    out, lse = c.run()
    c.check(out, lse)
    o2, l2 = c.kv.attend(c.q, c.cu, c.table, c.ctx)
    assert torch.allclose(out.float(), o2.float(), rtol=2.0 ** -6, atol=2.0 ** -6)
    assert torch.allclose(lse, l2, rtol=0, atol=1e-4)


@pytest.mark.parametrize("H, reqs", [(16, [(9, 300), (40, 41), (1, 700)]), (128, [(100, 3300)] * 4)])
def test_tree_attention_over_8_bit_rows_is_that_over_their_read_back(d, H, reqs):
    c = Trees(d, "e4m3", 64, H, reqs, seed=6)
    out, lse = c.run()
    assert c.kv.synchronize() == 0
    wide = d.PagedKV(c.kv.num_pages, 64, "bf16")
    for b, (_, n) in enumerate(reqs):
        pos = torch.arange(n, dtype=torch.int32, device="cuda").view(1, n)
        rows = c.kv.read(c.table[b:b + 1], c.ctx[b:b + 1], pos)[0]
        at = torch.arange(n, device="cuda")
        slots = c.table[b].long()[at // 64] * 64 + at % 64
        wide.write(rows[:, :512], rows[:, 512:], slots.to(torch.int32))
    assert c.kv.synchronize() == 0
    o2, l2 = wide.attend(c.q, c.cu, c.table, c.ctx, scale=1 / 24, tree=c.mask)
    assert wide.synchronize() == 0
    assert torch.equal(out, o2) and torch.equal(lse, l2)


def test_tree_attention_reports_more_nodes_than_bits(d):
    c = Trees(d, "bf16", 16, 16, [(40, 40), (3, 20)], seed=4, words=1)
    out, lse = c.run()
    assert c.kv.synchronize() == d._abi.TS_DEVERR_COUNT
    # what the words name is attended to all the same
    c.seen[0][:, 32:] = False
    c.check(out, lse, every=7)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("reqs, H", [([(100, 3300)] * 4, 128), ([(90, 9000), (1, 10), (120, 6000), (7, 7)], 128)])
def test_tree_attention_in_rounds_of_whole_row_tiles(d, fmt, reqs, H):
    # 64 key tiles a pair and more: the pairs take row tiles in turn
    c = Trees(d, fmt, 64, H, reqs, seed=5)
    out, lse = c.run()
    c.check(out, lse, every=37)
    o2, l2 = c.run()
    assert torch.equal(out, o2) and torch.equal(lse, l2)


# ---------------------------------------------------------------------------
# Verification
# ---------------------------------------------------------------------------

def drafted(rng, V, sizes, sharp=2.0, roots=1):
    """Trees whose children often hold likely tokens of their parents' rows."""
    T = sum(sizes)
    z = rng.normal(0, sharp, (T, V))
    p = np.exp(z - z.max(1, keepdims=True))
    p = (p / p.sum(1, keepdims=True)).astype(np.float32)
    parents, tokens, at = [], [], 0
    for n in sizes:
        par = [-1 if i < roots else int(rng.integers(i // 3, i)) for i in range(n)]
        order = np.argsort(-p[at:at + n], axis=1)
        seen = {}
        for i, x in enumerate(par):
            r = seen.get(x, 0)
            seen[x] = r + 1
            tokens.append(int(order[max(x, 0), min(r, V - 1)]))
        parents += par
        at += n
    return p, parents, tokens


def check_walk(d, p, parents, tokens, sizes, u, depth, got, lead=0):
    path, out, accepted = (x.cpu().numpy() for x in got)
    at = lead
    for b, n in enumerate(sizes):
        want = oc.verify_tree(tokens[at:at + n], parents[at:at + n], p[at:at + n],
                              None if u is None else u[b], depth)
        assert list(path[b]) == want[0] and list(out[b]) == want[1] and accepted[b] == want[2], b
        at += n


@pytest.mark.parametrize("sampled", [True, False])
@pytest.mark.parametrize("V, sizes, depth", [
    (1, [3], 2), (5, [1, 7, 40], 6), (130, [9, 0, 64], 3), (1001, [30] * 3, 8), (4096, [5], 0),
    (5003, [12, 100], 4), (20000, [20] * 2, 5),
])
def test_verify_tree(d, sampled, V, sizes, depth):
    rng = np.random.default_rng(V)
    p, parents, tokens = drafted(rng, V, sizes, sharp=4.0)
    B = len(sizes)
    u = rng.random((B, depth + 1)).astype(np.float32) if sampled else None
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pad = 3 if V % 2 else 0                       # rows that start between 16-byte boundaries
    target = torch.full((len(p), V + pad), math.nan, device="cuda")
    target[:, :V] = torch.from_numpy(p).cuda()
    got = d.verify_tree(i32(tokens), i32(parents), i32(np.cumsum([0] + sizes)), target[:, :V],
                        torch.from_numpy(u).cuda() if sampled else None, depth, err=err)
    assert d.ts_read_error(err) == 0
    check_walk(d, p, parents, tokens, sizes, u, depth, got)


@pytest.mark.parametrize("B, V", [(1, 131072), (40, 70001), (160, 33000), (1, 1 << 20)])
def test_verify_tree_of_large_vocabularies(d, B, V):
    # against sums in double on the GPU: 2^-60 a token apart from the oracle's
    depth, n = 3, 4
    g = torch.Generator(device="cuda").manual_seed(V)
    target = torch.softmax(6 * torch.randn(B * n, V, generator=g, device="cuda"), 1)
    u = torch.rand(B, depth + 1, generator=g, device="cuda")
    u[0] = torch.tensor([0.0, 0.999999, 0.5, 0.25], device="cuda")
    parents, cu = [-1, 0, 1, 2] * B, torch.arange(0, B * n + 1, n, dtype=torch.int32, device="cuda")
    run = target.double().cumsum(1)
    tokens = torch.zeros(B, n, dtype=torch.int32, device="cuda")
    drawn = [(run[i::n] <= u[:, i:i + 1].double() * run[i::n, -1:]).sum(1) for i in range(n)]
    for i in range(1, n):                          # drafts that come true, but every other request's last
        tokens[:, i] = drawn[i - 1].int()
    tokens[1::2, 3] += 1
    path, out, accepted = d.verify_tree(tokens.view(-1), i32(parents), cu, target, u)
    good = accepted == torch.where(torch.arange(B, device="cuda") % 2 == 1, 2, 3)
    assert torch.all(good)
    for i in range(n):
        at = accepted >= i
        assert torch.equal(out[at, i], drawn[i][at].int())
        assert torch.equal(path[:, i], torch.where(at, i, -1).int())


def test_verify_tree_corners(d):
    e = d._abi
    err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(p, parent, tokens, sizes, u, depth):
        p = np.asarray(p, dtype=np.float32)
        got = d.verify_tree(i32(tokens), None if parent is None else i32(parent),
                            i32(np.cumsum([0] + sizes)), torch.from_numpy(p).cuda(),
                            None if u is None else torch.tensor(u, dtype=torch.float32).cuda(), depth,
                            err=err)
        par = parent
        if parent is None:
            par = sum((list(range(-1, n - 1)) for n in sizes), [])
        check_walk(d, p, par, tokens, sizes, u, depth, got)
        return d.ts_read_error(err)

    rng = np.random.default_rng(1)
    one = np.eye(6, dtype=np.float32)
    # the lowest child of two with the token; a child of another parent; a second root
    assert run(one[[2, 3, 4, 1, 5]], [-1, 0, 0, 1, -1], [0, 2, 2, 3, 2], [5], [[.5] * 4], 3) == 0
    assert run(one[[2, 3, 4]], None, [0, 2, 3], [3], None, 5) == 0          # chains, greedy
    # equal values: the lower token; -0 equals 0; all -infinity: token 0
    assert run([[0, 7, 7, 1], [-0.0, 0, -1, 0], [-math.inf] * 4], [-1, 0, 1], [0, 1, 0], [3], None, 4) == 0
    assert run([[math.nan, 1, 3, 3]], [-1], [0], [1], None, 1) == e.TS_DEVERR_NAN
    assert run([[math.nan] * 4], [-1], [0], [1], None, 1) == e.TS_DEVERR_NAN
    # bad probabilities count as 0; rows of nothing, or of 16 and more, have no token
    assert run([[math.nan, .5, -1, 2.5, .5, -0.0]], [-1], [0], [1], [[.75]], 0) == e.TS_DEVERR_PROB
    assert run([[0.0] * 5, [.2] * 5], [-1, -1], [0, 0], [1, 1], [[.5], [.5]], 0) == e.TS_DEVERR_PROB
    assert run(np.full((1, 40), 1.9), [-1], [0], [1], [[.5]], 0) == e.TS_DEVERR_PROB
    assert run(np.full((1, 7), 1.9), [-1], [0], [1], [[.999]], 0) == 0       # 13.3
    # u at its ends, zeros at the row's ends
    p = np.array([[0, 0, .25, .75, 0]] * 2, np.float32)
    assert run(p, [-1, -1], [0, 0], [1, 1], [[0.0], [1 - 2.0 ** -24]], 0) == 0
    # many nodes, the child far behind
    n = 1024
    par = [-1] + [0] * (n - 1)
    toks = [0] + [int(x) for x in rng.permutation(n - 1) + 1]
    p = np.zeros((n, n), np.float32)
    p[0, toks[1000]] = 1
    p[1000, 3] = 1
    assert run(p, par, toks, [n], [[.5, .5]], 1) == 0


# ---------------------------------------------------------------------------
# Rows kept
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("page", [16, 64])
def test_keep(d, fmt, page):
    rng = np.random.default_rng(page)
    sizes, ctx = [6, 1, 60, 0, 33, 9], [20, 40, 200, 5, 33, 70]
    paths = [[0, 2, 5], [0], [0] + sorted(rng.choice(np.arange(1, 60), 35, replace=False).tolist()), [],
             list(range(33)), [0, 1, 3, 4]]
    depth = 40
    path = np.full((6, depth + 1), -1, np.int32)
    for b, x in enumerate(paths):
        path[b, :len(x)] = x
    accepted = [len(x) - 1 for x in paths]
    table, pages, _ = table_of(rng, ctx, page)
    kv = d.PagedKV(pages, page, fmt)
    kv.data.copy_(torch.from_numpy(rng.integers(0, 256, tuple(kv.data.shape)).astype(np.uint8)))
    want = kv.data.cpu().numpy().copy()
    old = want.copy()
    for b, (n, c) in enumerate(zip(sizes, ctx)):
        rows = oc.keep_rows([old[slot_of(table, page, b, c - n + i)] for i in range(n)], paths[b],
                            accepted[b])
        for i, r in enumerate(rows):
            want[slot_of(table, page, b, c - n + i)] = r
    lens = i32(ctx)
    new = kv.keep(i32(path), i32(accepted), i32(np.cumsum([0] + sizes)), sum(sizes), i32(table), lens,
                  new_len=lens)
    assert kv.synchronize() == 0 and new is lens
    assert np.array_equal(kv.data.cpu().numpy(), want)
    assert new.tolist() == [c - n + a + 1 for c, n, a in zip(ctx, sizes, accepted)]


def test_keep_reports_bad_paths_and_leaves_their_rows(d):
    e = d._abi
    kv = d.PagedKV(8, 16)
    kv.data.copy_(torch.arange(kv.data.numel(), device="cuda").view(kv.data.shape) % 251)
    old = kv.data.clone()
    table, cu = i32([[0, 1], [2, 3], [4, 5]]), i32([0, 5, 10, 15])
    bad = [[0, 3, 2, -1], [0, 1, 5, -1], [1, 2, 3, -1]]     # falls; past the nodes; not from 0
    new = kv.keep(i32(bad), i32([2, 2, 2]), cu, 15, table, i32([20, 20, 20]))
    assert kv.synchronize() == e.TS_DEVERR_PARENT and torch.equal(kv.data, old)
    assert new.tolist() == [15, 15, 15]
    kv.keep(i32([[0, 2, 4, -1]] * 3), i32([4, -2, 3]), cu, 15, table, i32([20, 20, 20]))
    assert kv.synchronize() == e.TS_DEVERR_PARENT and torch.equal(kv.data, old)
    new = kv.keep(i32([[0, 2, 4, -1]] * 3), i32([2, 2, 2]), cu, 15, i32([[0, 8], [2, -1], [4, 5]]),
                  i32([20, 20, 12]))
    assert kv.synchronize() == e.TS_DEVERR_SLOT_RANGE and new.tolist() == [18, 18, 10]
    want = old.clone()
    want[4 * 16 + 8], want[4 * 16 + 9] = old[4 * 16 + 9], old[4 * 16 + 11]
    assert torch.equal(kv.data, want)


# ---------------------------------------------------------------------------
# Beams
# ---------------------------------------------------------------------------

def check_beams(logits, cum, n, got):
    """Scores within their error, in order; the chosen ones are the oracle's but
    where scores lie closer together than that."""
    tokens, parents, scores = (x.cpu().numpy() for x in got)
    B, K = cum.shape
    for b in range(B):
        s = oc.beam_scores(logits[b], cum[b])
        wt, wp, ws = oc.beam_select(logits[b], cum[b], n)
        live = int(np.sum(np.isfinite(ws)))
        assert np.all(tokens[b, live:] == -1) and np.all(parents[b, live:] == -1)
        assert np.all(np.isneginf(scores[b, live:]))
        chosen = list(zip(parents[b, :live].tolist(), tokens[b, :live].tolist()))
        assert len(set(chosen)) == live
        for i, (k, t) in enumerate(chosen):
            # the score's rounding to fp32, and the log of a sum of which each part
            # is off by 2^-22 and its argument's rounding (2^-24 of up to log2 V + 1
            # on average), added up in fp32 over some 100 terms
            tol = 2.0 ** -17 + 2.0 ** -23 * abs(ws[i])
            assert abs(scores[b, i] - s[k, t]) <= tol and abs(s[k, t] - ws[i]) <= tol, (b, i)
        for i in range(1, live):                  # equal ones in their order
            if chosen[i][0] == chosen[i - 1][0]:
                k, (t0, t1) = chosen[i][0], (chosen[i - 1][1], chosen[i][1])
                x0, x1 = float(logits[b][k][t0]), float(logits[b][k][t1])
                assert x0 > x1 or (x0 == x1 and t0 < t1)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B, K, V, n", [(1, 1, 1, 1), (1, 1, 7, 3), (2, 3, 1000, 5), (1, 4, 33333, 8),
                                        (1, 1, 131072, 64), (3, 5, 50257, 33), (20, 8, 4099, 16),
                                        (1, 70, 513, 64), (600, 2, 300, 4)])
def test_beam_select(d, dtype, B, K, V, n):
    rng = np.random.default_rng(V + n)
    x = torch.from_numpy(rng.normal(0, 3, (B * K, V + 3)).astype(np.float32)).cuda().to(dtype)
    logits = x[:, :V].unflatten(0, (B, K))        # (rows that start between 16-byte boundaries)
    cum = rng.uniform(-4, 0, (B, K)).astype(np.float32)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = d.beam_select(logits, torch.from_numpy(cum).cuda(), n, err=err)
    assert d.ts_read_error(err) == 0
    host = logits.double().cpu().numpy()
    check_beams(host, cum, n, got)
    if K == 1:                                    # one beam: the order is the logits'
        for b in range(B):
            want = oc.beam_select(host[b], cum[b], n)
            assert got[0][b].tolist() == want[0]


KINDS = ["equal", "rising", "falling", "lowest", "masked", "dead", "large", "mixed", "two values"]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("V, n", [(90, 7), (40000, 10), (40000, 64)])
def test_beam_select_of_odd_rows(d, dtype, kind, V, n):
    rng = np.random.default_rng(n)
    B, K, low = 2, 3, torch.finfo(dtype).min
    x = torch.from_numpy(rng.normal(0, 2, (B, K, V)).astype(np.float32)).cuda()
    cum = torch.tensor([[0.0, -1.0, -2.0], [-0.5, -0.5, -0.5]], device="cuda")
    if kind == "equal":
        x.fill_(1.5)
    elif kind in ("rising", "falling"):
        x = torch.arange(V, device="cuda").float().expand(B, K, V) * 1e-3
        x = x.contiguous() if kind == "rising" else x.flip(2).contiguous()
    elif kind == "lowest":
        x.fill_(low)
    elif kind == "masked":
        x[:, :, torch.from_numpy(rng.random(V) < 0.9).cuda()] = -math.inf
        x[0, 0] = -math.inf                       # a beam with no token
        x[1, :, :] = -math.inf                    # fewer continuations than asked for
        x[1, 1, V // 2] = 3.0
    elif kind == "dead":
        cum[0, 1] = cum[1, 0] = cum[1, 1] = cum[1, 2] = -math.inf
    elif kind == "large":
        x = x * 1e4 + 3e5
    elif kind == "mixed":
        x[:, :, V // 2:] = low
        x[0, 0, : V // 3] = 3e7
    else:
        x = torch.where(x > 0, 1.0, -1.0)
    x = x.to(dtype)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = d.beam_select(x, cum, n, err=err)
    assert d.ts_read_error(err) == 0
    host, c = x.double().cpu().numpy(), cum.cpu().numpy()
    check_beams(host, c, n, got)
    if kind in ("equal", "lowest"):               # ties: the lower beam, then the lower token
        for b in range(B):
            want = oc.beam_select(host[b], c[b], n)
            assert got[0][b].tolist() == want[0] and got[1][b].tolist() == want[1]


@pytest.mark.parametrize("size", [2.0 ** 20, -2.0 ** 20])
@pytest.mark.parametrize("first", [0, 1])
def test_beam_select_where_the_sums_change_their_reference(d, size, first):
    # values on both sides of the size from which a part of a row takes its largest
    # value for reference, in parts of one row, a few apart
    rng = np.random.default_rng(12)
    V = 40000
    x = np.empty((1, 2, V), dtype=np.float32)
    near, far = size * (1 - 2.0 ** -18), size * (1 + 2.0 ** -19)     # 4 within, 2 past
    x[0, :, :V // 2] = near if first else far
    x[0, :, V // 2:] = far if first else near
    x += rng.integers(-4, 5, x.shape).astype(np.float32) / 8
    cum = np.array([[0.0, -0.5]], dtype=np.float32)
    got = d.beam_select(torch.from_numpy(x).cuda(), torch.from_numpy(cum).cuda(), 20)
    check_beams(x.astype(np.float64), cum, 20, got)
    # the scores' differences from the logits are the sums' logarithms
    for k in range(2):
        mine = got[1][0] == k
        t = got[0][0][mine].long().cpu().numpy()
        want = oc.beam_scores(x[0], cum[0])[k, t]
        assert np.all(np.abs(got[2][0][mine].double().cpu().numpy() - want) < 1e-5)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_beam_select_reports_nan_and_infinity(d, dtype):
    rng = np.random.default_rng(7)
    x = torch.from_numpy(rng.normal(0, 2, (2, 3, 5000)).astype(np.float32)).cuda()
    x[0, 0, ::5] = math.nan
    x[0, 1, 7] = math.inf
    x[0, 2] = math.nan
    x = x.to(dtype)
    cum = torch.tensor([[0.0, -0.1, -0.2], [math.nan, math.inf, -0.2]], device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = d.beam_select(x, cum, 9, err=err)
    assert d.ts_read_error(err) == d._abi.TS_DEVERR_NAN
    check_beams(x.double().cpu().numpy(), cum.cpu().numpy(), 9, got)
    assert torch.all(got[1][0] < 2) and torch.all(got[1][1] == 2)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("page", [16, 256])
def test_fork(d, fmt, page):
    rng = np.random.default_rng(page)
    B, K, n, width = 3, 4, 5, 4
    ctx = rng.integers(0, width * page + 1, B * K).astype(np.int32)
    ctx[:5] = [0, page, page + 1, width * page, 2 * page - 1]
    used = [-(-int(c) // page) for c in ctx]
    pages = sum(used) + B * n
    order = rng.permutation(pages)
    table, at = np.full((B * K, width), -1, np.int32), 0
    for i, m in enumerate(used):
        table[i, :m] = order[at:at + m]
        at += m
    spare = order[at:].astype(np.int32)
    parents = rng.integers(0, K, (B, n)).astype(np.int32)
    parents[0] = [0, 1, 2, 3, 3]
    parents[1, :2] = [0, -1]
    kv = d.PagedKV(pages, page, fmt)
    kv.data.copy_(torch.from_numpy(rng.integers(0, 256, tuple(kv.data.shape)).astype(np.uint8)))
    old = kv.data.cpu().numpy().copy()
    other = d.PagedKV(pages, page, fmt)
    other.data.copy_(kv.data)
    new_table, new_len = kv.fork(i32(parents), i32(spare), i32(table), i32(ctx))
    assert kv.synchronize() == 0
    assert other.fork(i32(parents), i32(spare), i32(table), i32(ctx), tables=False) is None
    assert other.synchronize() == 0 and torch.equal(other.data, kv.data)
    want = old.copy()
    for i in range(B * n):
        p = int(parents.reshape(-1)[i])
        p = p if p < 0 else i // n * K + p
        row, length, source, rows = oc.fork(table, ctx, p, int(spare[i]), page, width)
        assert new_table[i].tolist() == row and int(new_len[i]) == length, i
        if source is not None:
            a, z = int(spare[i]) * page, source * page
            want[a:a + rows] = old[z:z + rows]
    assert np.array_equal(kv.data.cpu().numpy(), want)


def test_fork_reports_what_is_wrong_and_keeps_an_only_child_in_place(d):
    e = d._abi
    kv = d.PagedKV(8, 16)
    kv.data.copy_(torch.arange(kv.data.numel(), device="cuda").view(kv.data.shape) % 251)
    old = kv.data.clone()
    table, ctx = i32([[0, 1], [2, 99]]), i32([20, 20])
    t, n = kv.fork(i32([[0, 2, -2]]), i32([1, 5, 6]), table, ctx)   # its own page; no such beams
    assert kv.synchronize() == e.TS_DEVERR_PARENT and torch.equal(kv.data, old)
    assert t.tolist() == [[0, 1], [-1, -1], [-1, -1]] and n.tolist() == [20, 0, 0]
    kv.fork(i32([[1, 0, 0]]), i32([5, 8, -1]), table, ctx)          # bad source, bad spare pages
    assert kv.synchronize() == e.TS_DEVERR_SLOT_RANGE and torch.equal(kv.data, old)
    t, n = kv.fork(i32([[1, 0]]), i32([5, 6]), table, i32([-1, 40]))
    assert kv.synchronize() == e.TS_DEVERR_CTX and n.tolist() == [32, 0]
    assert t.tolist() == [[2, 99], [6, -1]] and torch.equal(kv.data, old)


# ---------------------------------------------------------------------------
# Together
# ---------------------------------------------------------------------------

class Step:
    """One drafting step of two requests: a tree grown level by level by
    beam_select, its plan, its rows and queries appended, attended to, verified,
    its accepted rows kept and read back. The draft's and the target's logits are
    tables indexed by token, so every part can be followed on the host."""
    V, H, page, W, depth = 50, 16, 16, 3, 3

    def __init__(self, d, fmt):
        self.d, g = d, torch.Generator(device="cuda").manual_seed(11)
        self.draft = 2 * torch.randn(self.V, self.V, generator=g, device="cuda")
        self.target = torch.softmax(self.draft + 0.5 * torch.randn(self.V, self.V, generator=g,
                                                                   device="cuda"), 1)
        self.emb = torch.randn(self.V, 576, generator=g, device="cuda", dtype=torch.bfloat16)
        self.wq = torch.randn(self.V, self.H, 576, generator=g, device="cuda", dtype=torch.bfloat16)
        self.kv = d.PagedKV(24, self.page, fmt)
        self.table = torch.arange(24, dtype=torch.int32, device="cuda").view(2, 12)
        self.ctx = i32([37, 80])
        self.freq = torch.from_numpy(FREQ).cuda()
        n = int(self.ctx.max())
        rows = torch.randn(2, n, 576, generator=g, device="cuda", dtype=torch.bfloat16)
        for b in range(2):
            pos = torch.arange(n, dtype=torch.int32, device="cuda")
            self.kv.append(rows[b, :, :512], rows[b, :, 512:], pos, self.table[b, 0] * 16 + pos, self.freq)
        self.last = i32([3, 7])
        self.u = torch.rand(2, self.depth + 1, generator=g, device="cuda")
        self.nodes = 1 + self.W * self.depth
        self.cu = torch.arange(0, 2 * self.nodes + 1, self.nodes, dtype=torch.int32, device="cuda")

    def run(self):
        d, W, V = self.d, self.W, self.V
        tokens, parents = [self.last.view(2, 1)], [torch.full_like(self.last, -1).view(2, 1)]
        cum = torch.zeros(2, 1, device="cuda")
        level = torch.zeros(2, 1, dtype=torch.int32, device="cuda")   # the level's node numbers
        for k in range(self.depth):
            logits = self.draft[tokens[-1].long()]
            t, p, cum = d.beam_select(logits, cum, W, err=self.kv.err)
            parents.append(level.gather(1, p.long()))
            tokens.append(t)
            level = torch.arange(1 + k * W, 1 + (k + 1) * W, dtype=torch.int32,
                                 device="cuda").expand(2, W).contiguous()
        tokens, parents = torch.cat(tokens, 1).view(-1), torch.cat(parents, 1).view(-1)
        T = 2 * self.nodes
        ctx = self.ctx + self.nodes
        kv = self.kv
        pos, slots, mask = kv.plan_tree(parents, self.cu, self.table, ctx, T, self.nodes)
        x, q = self.emb[tokens.long()], self.wq[tokens.long()].clone()
        kv.append(x[:, :512], x[:, 512:], pos, slots, self.freq, q[:, :, 512:], q)
        out, lse = kv.attend(q, self.cu, self.table, ctx, tree=mask)
        path, nxt, accepted = d.verify_tree(tokens, parents, self.cu, self.target[tokens.long()],
                                            self.u, err=kv.err)
        new = kv.keep(path, accepted, self.cu, T, self.table, ctx)
        sel = kv.read(self.table, new, (new.view(2, 1) - 1).contiguous())
        return dict(tokens=tokens, parents=parents, pos=pos, mask=mask, q=q, out=out, lse=lse, path=path,
                    next=nxt, accepted=accepted, new=new, sel=sel)


@pytest.mark.parametrize("fmt", FORMATS)
def test_a_drafting_step(d, fmt):
    s = Step(d, fmt)
    before = s.kv.data.cpu().numpy().copy()
    r = {k: v.cpu() for k, v in s.run().items()}
    assert s.kv.synchronize() == 0
    table, H = s.table.cpu().numpy(), s.H
    for b in range(2):
        at, n, ctx = b * s.nodes, s.nodes, int(s.ctx[b])
        parent, tokens = r["parents"][at:at + n].tolist(), r["tokens"][at:at + n].tolist()
        assert r["pos"][at:at + n].tolist() == [ctx + e for e in oc.depths(parent)]
        # the tree's first level is the draft's best tokens after the last one
        best = np.argsort(-s.draft[s.last[b]].cpu().double().numpy(), kind="stable")[:s.W]
        assert tokens[1:1 + s.W] == best.tolist()
        # rows: the cached ones, then the nodes', turned by their own positions
        K = [oracle.unpack_row(before[slot_of(table, s.page, b, t)], fmt) for t in range(ctx)]
        for i in range(n):
            row = bits(s.emb[tokens[i]].view(1, 576))[0]
            turned = oc.turn(bf16_bits_to_f64(row[512:]), ctx + oc.depths(parent)[i], FREQ, True)
            row = np.concatenate([row[:512], round_to_bf16_bits(turned)])
            K.append(oracle.unpack_row(oracle.pack_row(row, fmt), fmt))
        K = np.stack(K)
        q = r["q"][at:at + n].double().numpy()
        o, z, mean_abs, size = oc.tree_attention(q, K, oc.sees(parent), 1 / 24)
        # (a rope value at the middle between two bf16 values may round the other way
        # on the two sides: 64 values of 576, half a step each, move a score by less
        # than 2^-8 of |q||k|)
        slack = 2 * 2.0 ** -8 * size[..., None] * (mean_abs + np.abs(o))
        assert np.all(np.abs(r["out"][at:at + n].double().numpy() - o)
                      <= output_bound(o, mean_abs, size) + slack)
        want = oc.verify_tree(tokens, parent, s.target.cpu().numpy()[tokens], s.u[b].cpu().numpy(), s.depth)
        assert (r["path"][b].tolist(), r["next"][b].tolist(), int(r["accepted"][b])) == want
        a = want[2]
        assert int(r["new"][b]) == ctx + a + 1
        # the last kept row is the last accepted node's
        x = bits(s.emb[tokens[want[0][a]]].view(1, 576))[0]
        got = r["sel"][b, 0].double().numpy()
        assert np.array_equal(got[:512], oracle.unpack_row(oracle.pack_row(x, fmt), fmt)[:512])
        check_turned(got[512:], bf16_bits_to_f64(x[512:]), ctx + a, True)


@pytest.mark.parametrize("fmt", FORMATS)
def test_a_captured_step_replays_with_new_inputs(d, fmt):
    s = Step(d, fmt)
    start = s.kv.data.clone()
    s.run()
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            got = s.run()
    for seed in (1, 2):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        s.u.copy_(torch.rand(s.u.shape, generator=gen, device="cuda"))
        s.last.copy_(torch.randint(0, s.V, (2,), generator=gen, device="cuda"))
        s.ctx.copy_(i32([20 + seed, 70 - seed]))
        s.kv.data.copy_(start)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        replayed = {k: v.clone() for k, v in got.items()}
        s.kv.data.copy_(start)
        eager = s.run()
        assert s.kv.synchronize() == 0
        for k in eager:
            assert torch.equal(replayed[k], eager[k]), (k, seed)


def test_steps_on_two_streams_do_not_meet(d):
    a, b = Step(d, "bf16"), Step(d, "e4m3")
    starts = a.kv.data.clone(), b.kv.data.clone()
    wants = [{k: v.clone() for k, v in x.run().items()} for x in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for x, s in zip((a, b), starts):
            x.kv.data.copy_(s)
        torch.cuda.synchronize()
        got = []
        for x, st in zip((a, b), streams):
            with torch.cuda.stream(st):
                got.append(x.run())
        torch.cuda.synchronize()
        for g, w in zip(got, wants):
            assert all(torch.equal(g[k], w[k]) for k in w)


@pytest.mark.parametrize("fmt", FORMATS)
def test_a_beam_search_reads_what_its_sequences_wrote(d, fmt):
    # three steps of 2 requests x 3 beams: rows stand for tokens, so that a
    # sequence's history can be read back from its pages
    V, K, page, g = 40, 3, 16, torch.Generator(device="cuda").manual_seed(5)
    score = 2 * torch.randn(V, V, generator=g, device="cuda")
    emb = torch.zeros(V, 576, dtype=torch.bfloat16, device="cuda")
    emb[torch.arange(V), torch.arange(V)] = 1.0
    start, steps, S = 14, 5, 2 * K
    kv = d.PagedKV(S * 2 + steps * S, page, fmt)
    free = list(range(S * 2, S * 2 + steps * S))
    table = torch.full((S, 3), -1, dtype=torch.int32, device="cuda")
    table[:, 0] = torch.arange(S, device="cuda")
    table[:, 1] = torch.arange(S, 2 * S, device="cuda")
    ctx = torch.full((S,), start, dtype=torch.int32, device="cuda")
    first = torch.randint(0, V, (S, start), generator=g, device="cuda")
    history = [h.tolist() for h in first]
    for t in range(start):
        x = emb[first[:, t]]
        kv.write(x[:, :512], x[:, 512:], table[:, t // page] * page + t % page)
    cum = torch.zeros(2, K, device="cuda")
    for step in range(steps):
        logits = score[[h[-1] for h in history]].view(2, K, V)
        tokens, parents, new_cum = d.beam_select(logits, cum, K, err=kv.err)
        for b in range(2):
            want = oc.beam_select(logits[b].double().cpu().numpy(), cum[b].cpu().numpy(), K)
            assert tokens[b].tolist() == want[0] and parents[b].tolist() == want[1]
        cum = new_cum
        spare = i32(free[step * S:(step + 1) * S])
        table, ctx = kv.fork(parents, spare, table, ctx)
        x = emb[tokens.view(-1).long()]
        at = table.long().gather(1, (ctx.long() // page).view(-1, 1)).view(-1) * page + ctx % page
        kv.write(x[:, :512], x[:, 512:], at.to(torch.int32))
        ctx = ctx + 1
        history = [history[b * K + int(parents[b, j])] + [int(tokens[b, j])]
                   for b in range(2) for j in range(K)]
        n = start + step + 1
        pos = torch.arange(n, dtype=torch.int32, device="cuda").repeat(S, 1)
        rows = kv.read(table, ctx, pos)
        assert kv.synchronize() == 0
        assert rows[:, :, :512].argmax(2).tolist() == history


@pytest.mark.parametrize("fmt", FORMATS)
def test_rows_past_32_bit_offsets(d, fmt):
    # a cache of more than 2^32 bytes: rows appended, kept and forked at its end
    page = 64
    pages = (1 << 32) // (page * d.dsa_cache_row_bytes(0 if fmt == "bf16" else 1)) + 40
    kv = d.PagedKV(pages, page, fmt)
    rng = np.random.default_rng(1)
    x = random_rows(rng, 6)
    t = bf16(x)
    end = pages - 1
    slots = [end * page + i for i in range(6)]
    kv.append(t[:, :512], t[:, 512:], i32([0] * 6), i32(slots), torch.from_numpy(FREQ).cuda())
    kv.keep(i32([[0, 2, 5]]), i32([2]), i32([0, 6]), 6, i32([[end]]), i32([6]))
    table, length = kv.fork(i32([[0]]), i32([end - 3]), i32([[end]]), i32([5]))
    assert kv.synchronize() == 0 and table.tolist() == [[end - 3]] and length.tolist() == [5]
    want = [oracle.pack_row(x[i], fmt) for i in (0, 2, 5, 3, 4)]
    split = 1024 if fmt == "bf16" else 528
    got = kv.data[(end - 3) * page:(end - 3) * page + 6].cpu().numpy()
    for i in range(5):
        assert np.array_equal(got[i, :split], want[i][:split])
    assert not got[5].any()


@pytest.mark.parametrize("fmt", FORMATS)
def test_a_request_behind_ones_that_share_tokens_is_attended_to_in_full(d, fmt):
    # two requests over the same tokens (reported) have more rows to merge than the
    # call has; the rows of the request behind them are merged all the same
    c = Trees(d, fmt, 64, 16, [(30, 3000), (8, 2500)], seed=9, seen=lambda rng, n: np.tri(n, dtype=bool))
    want, lse = c.run()
    c.check(want, lse, every=11)
    table, ctx = c.table, c.ctx
    four = torch.cat([table[:1], table[:1], table[:1], table[1:]]).contiguous()
    lens = torch.cat([ctx[:1], ctx[:1], ctx[:1], ctx[1:]]).contiguous()
    cu = i32([0, 30, 0, 30, 38])
    for tree in (None, c.mask):
        out, z = c.kv.attend(c.q, cu, four, lens, tree=tree)
        assert c.kv.synchronize() == d._abi.TS_DEVERR_ORDER
        assert torch.allclose(out[30:].float(), want[30:].float(), rtol=2.0 ** -6, atol=2.0 ** -6)
        assert torch.allclose(z[30:], lse[30:], rtol=0, atol=1e-4)
