"""Timed cases of the operators that follow several continuations of a context
over the paged latent cache: drafted trees and beams.

A cache row holds a token's 512 latent and 64 rope values, as 576 bf16 (fmt
"bf16", 1152 bytes), or as 512 e4m3 codes, 4 float scales (one for each 128
codes, a power of two) and 64 bf16 (fmt "e4m3", 656 bytes). A request's position
t lies in row t % page of page table[b][t // page]. A request's n new tokens are
its last n positions. As a tree, node i has the parent parent[i] < i among them
(-1: none, it follows the cached context); its position in the text is the first
new one's plus its depth.

  append  new tokens' rows into their slots, the rope pairs of rows and queries
          turned by their positions on the way; for a tree, its positions,
          slots and ancestor masks made from the parents first
  tree    absorbed-MLA attention of a tree's nodes over the cached context and
          their ancestors
  verify  a tree of drafts against the target's probabilities from given uniform
          numbers (or against its largest value): the accepted path, the token
          after it, and the path's rows moved together
  beam    the n best continuations of K beams over the vocabulary; with fork, the
          sequences' block tables reordered and their last pages copied

`run` is the plain form, or with `own` the library's calls.
"""
import math
import random

import torch

own = False

D, DV, ROPE, GROUP = 576, 512, 64, 128
ROW = {"bf16": 1152, "e4m3": 656}
SCALE = 1.0 / math.sqrt(D)
DEV = "cuda"


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one request's next token, 16 heads
        {"name": "append_one_bf16", "op": "append", "fmt": "bf16", "B": 1, "n": 1, "H": 16,
         "ctx": 4096, "page": 64, "mix": 0, "tree": False, "pairs": 1, "fused": False},
        # a step of 32 requests that each verify a drafted tree, the projections' outputs fused
        {"name": "append_trees_e4m3", "op": "append", "fmt": "e4m3", "B": 32, "n": 61, "H": 128,
         "ctx": 2048, "page": 64, "mix": 1, "tree": True, "pairs": 1, "fused": True},
        # a prefill chunk of 4095 tokens, rotated by halves
        {"name": "append_chunk_bf16", "op": "append", "fmt": "bf16", "B": 1, "n": 4095, "H": 128,
         "ctx": 16384, "page": 64, "mix": 0, "tree": False, "pairs": 0, "fused": True},
        # the smallest tree: one request, 16 nodes, 16 heads
        {"name": "tree_one_bf16", "op": "tree", "fmt": "bf16", "B": 1, "n": 16, "H": 16,
         "ctx": 4096, "page": 64, "mix": 0},
        # many requests, small ragged trees over short contexts, small pages
        {"name": "tree_small_e4m3", "op": "tree", "fmt": "e4m3", "B": 32, "n": 8, "H": 64,
         "ctx": 2048, "page": 16, "mix": 2},
        # ragged trees over long 8-bit contexts
        {"name": "tree_long_e4m3", "op": "tree", "fmt": "e4m3", "B": 4, "n": 61, "H": 128,
         "ctx": 32768, "page": 128, "mix": 3},
        # the largest: 16 requests, 64 nodes each
        {"name": "tree_batch_bf16", "op": "tree", "fmt": "bf16", "B": 16, "n": 64, "H": 128,
         "ctx": 8192, "page": 64, "mix": 0},
        # one request, greedy
        {"name": "verify_one_greedy", "op": "verify", "fmt": "bf16", "B": 1, "n": 16, "V": 32000,
         "depth": 5, "page": 64, "mix": 0, "sampled": False},
        # a batch's trees over a large vocabulary, sampled
        {"name": "verify_batch", "op": "verify", "fmt": "e4m3", "B": 32, "n": 61, "V": 131072,
         "depth": 8, "page": 64, "mix": 4, "sampled": True},
        # four beams of one request
        {"name": "beam_one_fp32", "op": "beam", "fmt": "bf16", "B": 1, "K": 4, "n": 4, "V": 32000,
         "half": False, "fork": True, "ctx": 1000, "page": 64},
        # a level of 16 requests' draft trees: ten nodes each, ten of their children kept
        {"name": "beam_level_fp32", "op": "beam", "fmt": "bf16", "B": 16, "K": 10, "n": 10,
         "V": 50257, "half": False, "fork": False, "ctx": 64, "page": 16},
        # eight beams of 64 requests over a large vocabulary in bf16, and their states
        {"name": "beam_batch_bf16", "op": "beam", "fmt": "e4m3", "B": 64, "K": 8, "n": 8,
         "V": 131072, "half": True, "fork": True, "ctx": 300, "page": 64},
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over the logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["append", "tree", "tree", "verify", "beam"])
    c = {"op": op, "fmt": rng.choice(["bf16", "e4m3"]), "page": rng.choice([16, 32, 64, 128])}
    H = rng.choice([16, 32, 64, 128, rng.randint(1, 128)])
    if op == "append":
        tree = rng.random() < 0.5
        B = _log(rng, 1, 32)
        n = _log(rng, 1, 64) if tree else _log(rng, 1, 4095 // B)
        return dict(c, B=B, n=n, H=H, ctx=_log(rng, n, 16384), mix=rng.randint(0, 1000), tree=tree,
                    pairs=rng.randint(0, 1), fused=rng.random() < 0.5)
    if op == "tree":
        # B * n * H * ctx within the largest listed case's
        B, ctx = _log(rng, 1, 32), _log(rng, 1, 32768)
        n = max(1, min(_log(rng, 1, 256), ctx, 1_000_000_000 // (B * H * ctx)))
        return dict(c, B=B, n=n, H=H, ctx=ctx, mix=rng.randint(0, 1000))
    if op == "verify":
        return dict(c, B=_log(rng, 1, 32), n=rng.randint(1, 61), V=_log(rng, 1000, 131072),
                    depth=rng.randint(1, 8), mix=rng.randint(0, 1000), sampled=rng.random() < 0.7)
    return dict(c, B=_log(rng, 1, 64), K=rng.randint(1, 8), n=rng.choice([1, 4, 8, rng.randint(1, 32)]),
                V=_log(rng, 1000, 131072), half=rng.random() < 0.5, fork=rng.random() < 0.5,
                ctx=_log(rng, 1, 300))


def _lengths(case):
    """New tokens and cached tokens (the new ones among them) of each request:
    all alike for mix 0, else ragged."""
    B, n, ctx, mix = case["B"], case["n"], case.get("ctx", 300), case["mix"]
    ctx = max(ctx, n)
    if mix == 0:
        return [n] * B, [ctx] * B
    r = random.Random(mix)
    new = [r.randint(1, n) for _ in range(B)]
    new[r.randrange(B)] = n
    cached = [r.randint(x, ctx) for x in new]
    cached[r.randrange(B)] = ctx
    return new, cached


def _parents(case, new):
    """Each request's tree: node 0 is its root, node i's parent one of the nodes
    i // 4 .. i - 1."""
    r = random.Random(case["mix"] + 7)
    return [[-1] + [r.randrange(i // 4, i) for i in range(1, n)] for n in new]


def _pairs_of_tree(parents, cached):
    """(node, position) pairs that attend."""
    total = 0
    for par, c in zip(parents, cached):
        depth = []
        for p in par:
            depth.append(0 if p < 0 else depth[p] + 1)
        total += sum(c - len(par) + d + 1 for d in depth)
    return total


def work(case):
    op = case["op"]
    if op == "append":
        new, _ = _lengths(case)
        n = sum(new)
        nbytes = n * (1152 + 4 + 4 + ROW[case["fmt"]] + case["H"] * ROPE * 4)
        if case["tree"]:
            nbytes += n * (4 + 4 * _words(new))
        return {"bytes": nbytes, "flops": n * (1 + case["H"]) * ROPE * 3}
    if op == "tree":
        new, cached = _lengths(case)
        H = case["H"]
        return {"bytes": sum(cached) * ROW[case["fmt"]]
                + sum(new) * (H * (2 * D + 2 * DV + 4) + 4 * _words(new)),
                "flops": 2 * _pairs_of_tree(_parents(case, new), cached) * H * (D + DV)}
    if op == "verify":
        # one row of the target for each node on the path (some 0.55 of the draws meet a child),
        # and the path's rows moved
        rows = case["B"] * (1 - 0.55 ** (min(case["depth"], case["n"]) + 1)) / 0.45
        return {"bytes": rows * (case["V"] * 4 + 2 * ROW[case["fmt"]]), "flops": rows * case["V"]}
    size = 2 if case["half"] else 4
    nbytes = case["B"] * (case["K"] * case["V"] * size + case["n"] * 12)
    if case["fork"]:
        nbytes += case["B"] * case["n"] * 2 * (case["ctx"] % case["page"]) * ROW[case["fmt"]]
    return {"bytes": nbytes, "flops": case["B"] * case["K"] * case["V"] * 3}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _pack(x, fmt):
    """bf16 rows [n][576] as cache rows (bytes [n][ROW])."""
    if fmt == "bf16":
        return x.contiguous().view(torch.uint8)
    g = x[:, :DV].float().view(-1, DV // GROUP, GROUP)
    amax = g.abs().amax(2)
    # the smallest power of two with amax / scale <= 448 = 0.875 * 2^9, at least 2^-120
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-120)
    e = torch.where(amax > 0, e, torch.full_like(e, -120))
    scale = torch.ldexp(torch.ones_like(amax), e)
    codes = (g * torch.ldexp(torch.ones_like(amax), -e).unsqueeze(2)).clamp(-448, 448)
    codes = codes.to(torch.float8_e4m3fn).view(torch.uint8).view(-1, DV)
    return torch.cat([codes, scale.view(torch.uint8),
                      x[:, DV:].contiguous().view(torch.uint8)], 1)


def _views(cache, fmt):
    """The values that a cache's bytes stand for."""
    if fmt == "bf16":
        return {"rows": cache.view(torch.bfloat16)}
    return {"codes": cache[:, :DV].view(torch.float8_e4m3fn),
            "scales": cache[:, DV:DV + 16].view(torch.float32),
            "rope": cache[:, DV + 16:].view(torch.bfloat16)}


def _rows(n, g):
    """Latent rows: unit normal, each row with a size of its own."""
    x = torch.randn(n, D, generator=g, device=DEV, dtype=torch.bfloat16)
    return x * torch.exp(0.5 * torch.randn(n, 1, generator=g, device=DEV)).to(torch.bfloat16)


def _cache(slots, fmt, g):
    out = torch.empty(slots, ROW[fmt], dtype=torch.uint8, device=DEV)
    for a in range(0, slots, 1 << 18):
        out[a:a + (1 << 18)] = _pack(_rows(min(1 << 18, slots - a), g), fmt)
    return out


def _table(lens, width, page, g, spare=0):
    """A block table [B][width] with pages in random order, -1 past a request's
    last, the pages' rows, and `spare` pages that no request has."""
    used = [-(-n // page) for n in lens]
    pages = max(1, sum(used) + spare)
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(lens), max(1, width)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = order[at:at + n]
        at += n
    return table, pages * page, order[at:at + spare].contiguous()


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _words(new):
    return -(-max(new) // 32)


def _masks(parents, words):
    """Bit j of node i's mask: j is i or an ancestor of it; int32 [T][words]."""
    out = []
    for par in parents:
        m = []
        for i, p in enumerate(par):
            m.append((m[p] if p >= 0 else 0) | 1 << i)
        out += [[(x >> 32 * w & 0xffffffff) - (1 << 32) * (x >> (32 * w + 31) & 1)
                 for w in range(words)] for x in m]
    return _ints(out)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op = case["op"]
    s = dict(case)
    page = case["page"]
    if op == "beam":
        B, K, n, V, ctx = case["B"], case["K"], case["n"], case["V"], case["ctx"]
        logits = 2.5 * torch.randn(B * K, V, generator=g, device=DEV)
        s["logits"] = logits.to(torch.bfloat16) if case["half"] else logits
        s["cum"] = -3 * torch.rand(B, K, generator=g, device=DEV) - 2
        if case["fork"]:
            width = -(-(ctx + 1) // page)
            s["table"], slots, s["spare"] = _table([ctx] * (B * K), width, page, g, B * n)
            s["cache"] = _cache(slots, case["fmt"], g)
            s["ctx_len"] = _ints([ctx] * (B * K))
        return s
    new, cached = _lengths(case)
    s["T"], s["most_new"], s["most_ctx"] = sum(new), max(new), max(cached)
    s["words"] = _words(new)
    s["table"], slots, _ = _table(cached, -(-max(cached) // page), page, g)
    s["cache"] = _cache(slots, case["fmt"], g)
    s["cu_q"] = torch.tensor([0] + new, device=DEV).cumsum(0).to(torch.int32)
    s["ctx_len"] = _ints(cached)
    parents = _parents(case, new)
    if op == "append":
        T, H = s["T"], case["H"]
        s["freq"] = 10000.0 ** (-torch.arange(ROPE // 2, device=DEV, dtype=torch.float64) / 32)
        x, wide = _rows(T, g), case["fused"]
        s["latent"], s["rope"] = ((x[:, :DV], x[:, DV:]) if wide
                                  else (x[:, :DV].contiguous(), x[:, DV:].contiguous()))
        # the up-projection's 128 values and the rope part of a head lie side by side where fused
        part = torch.randn(T, H, 192 if wide else 64, generator=g, device=DEV, dtype=torch.bfloat16)
        s["q_rope"] = part[:, :, 128:] if wide else part
        s["q"] = torch.randn(T, H, D, generator=g, device=DEV, dtype=torch.bfloat16)
        if case["tree"]:
            s["parent"] = _ints(sum(parents, []))
        else:
            at = torch.cat([torch.arange(c - n, c) for n, c in zip(new, cached)]).to(DEV)
            b = torch.arange(len(new), device=DEV).repeat_interleave(s["cu_q"].diff().long())
            s["pos"] = at.to(torch.int32)
            s["slots"] = (s["table"].long()[b, at // page] * page + at % page).to(torch.int32)
    elif op == "tree":
        s["mask"] = _masks(parents, s["words"])
        s["q"] = 1.5 * torch.randn(s["T"], case["H"], D, generator=g, device=DEV,
                                   dtype=torch.bfloat16)
    else:
        B, V, T = case["B"], case["V"], s["T"]
        flat = sum(parents, [])
        s["parent"] = _ints(flat)
        logits = 7 * torch.randn(T, V, generator=g, device=DEV)
        # a node's children: the likeliest tokens by a draft that is a little off
        top = (logits + torch.randn(T, V, generator=g, device=DEV)).topk(32, 1).indices
        s["target"] = torch.softmax(logits, 1)
        first = sum(([sum(new[:b])] * n for b, n in enumerate(new)), [])
        seen, rank = {}, []
        for a, p in zip(first, flat):
            rank.append(seen.get((a, p), 0) % 32)
            seen[a, p] = seen.get((a, p), 0) + 1
        at = torch.tensor([a + max(p, 0) for a, p in zip(first, flat)], device=DEV)
        s["tokens"] = top[at, torch.tensor(rank, device=DEV)].to(torch.int32)
        u = torch.rand(B, case["depth"] + 1, generator=g, device=DEV)
        s["u"] = u if case["sampled"] else None
    return s


# ---------------------------------------------------------------------------
# The plain forms and the library's calls
# ---------------------------------------------------------------------------

def _unpack(rows, fmt):
    """Cache rows (bytes [..][ROW]) as float rows [..][576]."""
    if fmt == "bf16":
        return rows.view(torch.bfloat16).float()
    codes = rows[..., :DV].view(torch.float8_e4m3fn).float().unflatten(-1, (DV // GROUP, GROUP))
    scale = rows[..., DV:DV + 16].contiguous().view(torch.float32)
    rope = rows[..., DV + 16:].contiguous().view(torch.bfloat16).float()
    return torch.cat([(codes * scale.unsqueeze(-1)).flatten(-2), rope], -1)


def _requests(s):
    """For every token its request and its number there; a request's tokens."""
    first, count = s["cu_q"][:-1].long(), s["cu_q"].long().diff()
    t = torch.arange(s["T"], device=DEV)
    b = torch.bucketize(t, s["cu_q"][1:].long(), right=True)
    return b, t - first[b], first, count


def _plain_plan(s):
    """Positions, slots and masks of the trees' nodes, the ancestors found by
    doubling the steps upwards."""
    b, i, first, count = _requests(s)
    T, n, page = s["T"], 32 * s["words"], s["page"]
    has = torch.zeros(T, n, dtype=torch.bool, device=DEV)      # ancestors, the node among them
    has.scatter_(1, i[:, None], True)
    parent = s["parent"].long()
    up = torch.where(parent < 0, T, first[b] + parent)         # T: past the root
    up = torch.cat([up, torch.tensor([T], device=DEV)])
    has = torch.cat([has, torch.zeros(1, n, dtype=torch.bool, device=DEV)])
    for _ in range(max(1, math.ceil(math.log2(s["most_new"])))):
        has, up = has | has[up], up[up]
    has = has[:T]
    base = (s["ctx_len"].long() - count)[b]
    at = base + i
    slots = s["table"].long()[b, at // page] * page + at % page
    bit = torch.ones((), dtype=torch.int64, device=DEV) << torch.arange(32, device=DEV)
    mask = (has.view(T, s["words"], 32) * bit).sum(2)
    return base + has.sum(1) - 1, slots, torch.where(mask >= 1 << 31, mask - (1 << 32), mask)


def _turn(x, cos, sin, pairs):
    """Rope parts [..][64] turned: pairs (2 i, 2 i + 1), or (i, i + 32) by halves."""
    x = x.float()
    a, b = (x[..., 0::2], x[..., 1::2]) if pairs else (x[..., :32], x[..., 32:])
    y = a * cos - b * sin, a * sin + b * cos
    return (torch.stack(y, -1).flatten(-2) if pairs else torch.cat(y, -1)).to(torch.bfloat16)


def _plain_append(s):
    out = {}
    if s["tree"]:
        pos, slots, mask = _plain_plan(s)
        out = {"pos": pos.to(torch.int32), "slots": slots.to(torch.int32),
               "mask": mask.to(torch.int32)}
    else:
        pos, slots = s["pos"], s["slots"].long()
    angle = pos.double()[:, None] * s["freq"]
    cos, sin = angle.cos().float(), angle.sin().float()
    x = torch.cat([s["latent"], _turn(s["rope"], cos, sin, s["pairs"])], 1)
    s["cache"][slots] = _pack(x, s["fmt"])
    s["q"][:, :, DV:] = _turn(s["q_rope"], cos[:, None], sin[:, None], s["pairs"])
    return dict(out, q=s["q"], **_views(s["cache"], s["fmt"]))


def _plain_tree(s):
    B, H, n, L, page = s["B"], s["H"], s["most_new"], s["most_ctx"], s["page"]
    b, i, first, count = _requests(s)
    ctx = s["ctx_len"].long()
    at = torch.arange(L, device=DEV)
    slot = s["table"].long()[:, at // page].clamp(min=0) * page + at % page
    K = _unpack(s["cache"][slot], s["fmt"])                               # [B][L][576]
    node = (first[:, None] + torch.arange(n, device=DEV)).clamp(max=s["T"] - 1)
    q = s["q"][node].float()                                              # [B][n][H][576]
    S = torch.matmul(q.view(B, n * H, D), K.transpose(1, 2)).view(B, n, H, L)
    S *= SCALE
    j = at - (ctx - count)[:, None]                                       # [B][L]: new token's number
    word = (j >> 5).clamp(0, s["words"] - 1)
    bits = s["mask"][node].gather(2, word[:, None].expand(B, n, L)) >> (j & 31)[:, None] & 1
    sees = torch.where(j[:, None] < 0, True, (bits != 0) & (at < ctx[:, None])[:, None])
    S.masked_fill_(~sees[:, :, None], -math.inf)
    m = S.amax(3, keepdim=True).clamp(min=-3e38)
    p = S.sub_(m).exp_()
    z = p.sum(3)
    o = torch.matmul(p.view(B, n * H, L), K[..., :DV]).view(B, n, H, DV)
    o /= z.clamp(min=1e-38).unsqueeze(3)
    lse = m.squeeze(3) + z.log()
    return {"out": o[b, i].to(torch.bfloat16), "lse": lse[b, i]}


def _plain_verify(s):
    B, V, depth, page = s["B"], s["V"], s["depth"], s["page"]
    b, i, first, count = _requests(s)
    r = torch.arange(B, device=DEV)
    node = torch.zeros(B, dtype=torch.int64, device=DEV)
    going = torch.ones(B, dtype=torch.bool, device=DEV)
    far = 1 << 30
    path, tokens, accepted = [node], [], node
    for step in range(depth + 1):
        p = s["target"][first + node]
        if s["u"] is None:
            t = p.argmax(1)
        else:
            below = p.double().cumsum(1)
            t = (below <= s["u"][:, step:step + 1].double() * below[:, -1:]).sum(1).clamp(max=V - 1)
        tokens.append(torch.where(going, t, -1))
        # the first child with that token
        child = torch.where((s["parent"] == node[b]) & (s["tokens"] == t[b]), i, far)
        child = torch.full((B,), far, device=DEV).scatter_reduce_(0, b, child, "amin")
        going = going & (child < far)
        if step < depth:
            node = torch.where(going, child, node)
            path.append(torch.where(going, child, -1))
            accepted = accepted + going
    path = torch.stack(path, 1)
    # the path's rows, from their places among the new tokens to the first ones
    base = (s["ctx_len"].long() - count)[:, None]
    table = s["table"].long()
    src, dst = base + path.clamp(min=0), base + torch.arange(depth + 1, device=DEV)
    keep = path >= 0
    src = (table.gather(1, src // page) * page + src % page)[keep]
    dst = torch.where(keep, dst, base)
    dst = (table.gather(1, dst // page) * page + dst % page)[keep]
    s["cache"][dst] = s["cache"][src]
    return dict(path=path.to(torch.int32), tokens=torch.stack(tokens, 1).to(torch.int32),
                accepted=accepted.to(torch.int32),
                length=(base[:, 0] + accepted + 1).to(torch.int32),
                **_views(s["cache"], s["fmt"]))


def _plain_beam(s):
    B, K, n, V = s["B"], s["K"], s["n"], s["V"]
    x = s["logits"].float()
    m = x.amax(1, keepdim=True)
    lse = m.double() + (x - m).exp().sum(1, keepdim=True, dtype=torch.float64).log()
    # a beam's best by value, then the lower token: whole numbers in the values' order
    k = x.view(torch.int32).long()
    k = torch.where(k < 0, -(k & 0x7fffffff), k)
    k = k * (1 << 20) + (V - 1 - torch.arange(V, device=DEV))
    token = V - 1 - (k.topk(n, 1).values & ((1 << 20) - 1))                # [B K][n]
    score = s["cum"].double().view(-1, 1) + (x.gather(1, token).double() - lse)
    # all beams' best in one line, ties to the lower beam and token
    best = score.view(B, K * n).sort(dim=1, descending=True, stable=True)
    at = best.indices[:, :n]
    parent = at // n
    out = {"scores": best.values[:, :n].float(), "parents": parent.to(torch.int32),
           "tokens": token.view(B, K * n).gather(1, at).to(torch.int32)}
    if s["fork"]:
        page, ctx = s["page"], s["ctx"]
        old = (torch.arange(B, device=DEV)[:, None] * K + parent).view(-1)
        table = s["table"][old]
        last, rows = ctx // page, ctx % page
        r = torch.arange(rows, device=DEV)
        table[:, last] = s["spare"]
        src = (s["table"][old, last].long()[:, None] * page + r).view(-1)
        dst = (s["spare"].long()[:, None] * page + r).view(-1)
        s["cache"][dst] = s["cache"][src]
        out |= {"table": table, "length": s["ctx_len"][old], **_views(s["cache"], s["fmt"])}
    return out


def _empty(*shape, dtype=torch.int32):
    return torch.empty(shape, dtype=dtype, device=DEV)


def _own(s):
    import decode_dsa_kv_gb300 as d
    op, B, page = s["op"], s["B"], s["page"]
    fmt = {"bf16": d.DSA_CACHE_BF16, "e4m3": d.DSA_CACHE_E4M3}[s["fmt"]]
    cache, table = s.get("cache"), s.get("table")
    if op == "append":
        T, out = s["T"], {}
        pos, slots = s.get("pos"), s.get("slots")
        if s["tree"]:
            pos, slots, mask = _empty(T), _empty(T), _empty(T, s["words"])
            d.check(d.dsa_tree_plan(s["parent"], s["cu_q"], T, B, s["ctx_len"], table,
                                    table.shape[1], page, cache.shape[0], pos, slots, mask,
                                    s["words"]), "dsa_tree_plan")
            out = {"pos": pos, "slots": slots, "mask": mask}
        q_rope = s["q_rope"]
        d.check(d.dsa_cache_append(s["latent"], s["latent"].stride(0), s["rope"],
                                   s["rope"].stride(0), pos, slots, T, s["freq"], s["pairs"],
                                   cache, cache.shape[0], fmt, q_rope, q_rope.stride(0),
                                   q_rope.stride(1), s["H"], s["q"], s["H"] * D),
                "dsa_cache_append")
        return dict(out, q=s["q"], **_views(cache, s["fmt"]))
    if op == "tree":
        T, H = s["T"], s["H"]
        out = _empty(T, H, DV, dtype=torch.bfloat16)
        lse = _empty(T, H, dtype=torch.float32)
        size = d.sfa_chunk_workspace_size(T, B, H)
        ws = _empty(size, dtype=torch.uint8)
        d.check(d.sfa_mla_tree(s["q"], H * D, s["cu_q"], T, B, H, cache, cache.shape[0], fmt,
                               table, table.shape[1], page, s["ctx_len"], s["mask"], s["words"],
                               SCALE, out, lse, ws, size), "sfa_mla_tree")
        return {"out": out, "lse": lse}
    if op == "verify":
        depth = s["depth"]
        path, tokens, accepted, length = (_empty(B, depth + 1), _empty(B, depth + 1), _empty(B),
                                          _empty(B))
        d.check(d.ts_verify_tree(s["tokens"], s["parent"], s["cu_q"], s["T"], B, s["target"],
                                 s["V"], s["u"], s["V"], depth, path, tokens, accepted),
                "ts_verify_tree")
        d.check(d.dsa_cache_keep(cache, cache.shape[0], fmt, table, table.shape[1], page,
                                 s["cu_q"], s["T"], s["ctx_len"], B, path, depth, accepted,
                                 length), "dsa_cache_keep")
        return dict(path=path, tokens=tokens, accepted=accepted, length=length,
                    **_views(cache, s["fmt"]))
    K, n, V = s["K"], s["n"], s["V"]
    tokens, parents, scores = _empty(B, n), _empty(B, n), _empty(B, n, dtype=torch.float32)
    size = d.ts_beam_workspace_size(B, K, V, n)
    ws = _empty(size, dtype=torch.uint8)
    d.check(d.ts_beam_select(s["logits"], d.TS_BF16 if s["half"] else d.TS_FP32, V, s["cum"], B, K,
                             V, n, tokens, parents, scores, ws, size), "ts_beam_select")
    out = {"scores": scores, "parents": parents, "tokens": tokens}
    if s["fork"]:
        width = table.shape[1]
        new_table, length = _empty(B * n, width), _empty(B * n)
        d.check(d.dsa_cache_fork(cache, cache.shape[0], fmt, table, width, page, s["ctx_len"],
                                 parents, s["spare"], B, K, n, new_table, length),
                "dsa_cache_fork")
        out |= {"table": new_table, "length": length, **_views(cache, s["fmt"])}
    return out


def run(state):
    if own:
        return _own(state)
    return {"append": _plain_append, "tree": _plain_tree, "verify": _plain_verify,
            "beam": _plain_beam}[state["op"]](state)


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def _values64(byte_rows, fmt):
    if fmt == "bf16":
        return byte_rows.contiguous().view(torch.bfloat16).double()
    parts = [byte_rows[:, 128 * i:128 * i + 128].contiguous().view(torch.float8_e4m3fn).double()
             * byte_rows[:, 512 + 4 * i:516 + 4 * i].contiguous().view(torch.float32).double()
             for i in range(4)]
    return torch.cat(parts + [byte_rows[:, 528:].contiguous().view(torch.bfloat16).double()], 1)


def _fields64(cache, fmt):
    return {k: v.double() for k, v in _views(cache, fmt).items()}


def _turn64(x, pos, freq, pairs):
    """Pair i as a complex number, times e^(i pos freq_i)."""
    x = x.double()
    z = torch.complex(*((x[..., 0::2], x[..., 1::2]) if pairs else (x[..., :32], x[..., 32:])))
    e = pos.double()[:, None] * freq
    z = z * torch.polar(torch.ones_like(e), e).view(-1, *[1] * (x.dim() - 2), 32)
    y = torch.empty_like(x)
    if pairs:
        y[..., 0::2], y[..., 1::2] = z.real, z.imag
    else:
        y[..., :32], y[..., 32:] = z.real, z.imag
    return y


def _exact_append(case, s):
    new, cached = _lengths(case)
    page, table, out = case["page"], s["table"].tolist(), {}
    pos, slots, masks = [], [], []
    for b, (par, c) in enumerate(zip(_parents(case, new), cached)):
        depth, bits = [], []
        for i, p in enumerate(par):
            depth.append((0 if p < 0 else depth[p] + 1) if case["tree"] else i)
            bits.append({i} | (bits[p] if case["tree"] and p >= 0 else set()))
            at = c - len(par) + i
            pos.append(c - len(par) + depth[i])
            slots.append(table[b][at // page] * page + at % page)
            words = [sum(1 << k for k in range(32) if 32 * w + k in bits[i])
                     for w in range(s["words"])]
            masks.append([w - (1 << 32) if w >> 31 else w for w in words])
    if case["tree"]:
        out = {"pos": _ints(pos), "slots": _ints(slots), "mask": _ints(masks)}
    out |= _fields64(s["cache"], case["fmt"])
    at, pos = torch.tensor(slots, device=DEV), torch.tensor(pos, device=DEV)
    rope = _turn64(s["rope"], pos, s["freq"], case["pairs"])
    q = s["q"].double()
    q[:, :, DV:] = _turn64(s["q_rope"], pos, s["freq"], case["pairs"])
    out["q"] = q
    x = s["latent"].double()
    if case["fmt"] == "bf16":
        out["rows"][at] = torch.cat([x, rope], 1)
        return out
    for i in range(4):
        part = x[:, 128 * i:128 * i + 128]
        top = part.abs().amax(1)
        e = torch.ceil(torch.log2(top / 448))
        e = torch.where(torch.exp2(e - 1) * 448 >= top, e - 1, e)     # log2 rounded up
        e = torch.where(torch.exp2(e) * 448 < top, e + 1, e).clamp(min=-120)
        out["codes"][at, 128 * i:128 * i + 128] = part / torch.exp2(e)[:, None]
        out["scales"][at, i] = torch.exp2(e)
    out["rope"][at] = rope
    return out


def _exact_tree(case, s):
    new, cached = _lengths(case)
    H, page = case["H"], case["page"]
    outs, lses, at = [], [], 0
    for b, (par, c) in enumerate(zip(_parents(case, new), cached)):
        n = len(par)
        t = torch.arange(c, device=DEV)
        K = _values64(s["cache"][s["table"][b].long()[t // page] * page + t % page], case["fmt"])
        sees = torch.ones(n, c, dtype=torch.bool)
        sees[:, c - n:] = torch.eye(n, dtype=torch.bool)
        for i, p in enumerate(par):
            if p >= 0:
                sees[i, c - n:] |= sees[p, c - n:]
        sees = sees.to(DEV)
        step = max(1, 100_000_000 // (H * c))
        for i in range(0, n, step):
            k = min(n, i + step)
            z = (s["q"][at + i:at + k].double().reshape(-1, D) @ K.T) / math.sqrt(D)
            z = torch.where(sees[i:k].repeat_interleave(H, 0), z, -math.inf)
            lse = torch.logsumexp(z, 1)
            outs.append((torch.exp(z - lse[:, None]) @ K[:, :DV]).view(k - i, H, DV))
            lses.append(lse.view(k - i, H))
        at += n
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}


def _exact_verify(case, s):
    new, cached = _lengths(case)
    parents, V, depth, page = _parents(case, new), case["V"], case["depth"], case["page"]
    tokens, table = s["tokens"].tolist(), s["table"].tolist()
    rows = s["cache"].clone()
    paths, outs, accepted, length, at = [], [], [], [], 0
    for b, (par, c) in enumerate(zip(parents, cached)):
        n, path, out = len(par), [0], []
        while True:
            p = s["target"][at + path[-1]].double()
            if s["u"] is None:
                t = int(p.argmax())
            else:
                w = torch.cumsum(p, 0)
                point = w[-1:] * s["u"][b, len(out)].double()
                t = min(V - 1, int(torch.searchsorted(w, point, right=True)))
            out.append(t)
            child = [i for i in range(n) if par[i] == path[-1] and tokens[at + i] == t]
            if not child or len(path) > depth:
                break
            path.append(child[0])

        def slot(t):
            return table[b][t // page] * page + t % page
        for k, i in enumerate(path):
            rows[slot(c - n + k)] = s["cache"][slot(c - n + i)]
        a = len(path) - 1
        paths.append(path + [-1] * (depth - a))
        outs.append(out + [-1] * (depth - a))
        accepted.append(a)
        length.append(c - n + a + 1)
        at += n
    return dict(path=_ints(paths), tokens=_ints(outs), accepted=_ints(accepted),
                length=_ints(length), **_fields64(rows, case["fmt"]))


def _exact_beam(case, s):
    B, K, n, V = case["B"], case["K"], case["n"], case["V"]
    scores, parents, tokens = [], [], []
    for b in range(B):
        x = s["logits"][b * K:(b + 1) * K].double()
        total = s["cum"][b].double()[:, None] + torch.log_softmax(x, 1)
        v, at = total.view(-1).sort(dim=0, descending=True, stable=True)
        scores.append(v[:n])
        parents.append(at[:n] // V)
        tokens.append(at[:n] % V)
    scores, parents, tokens = (torch.stack(x) for x in (scores, parents, tokens))
    out = {"scores": scores, "parents": parents.to(torch.int32), "tokens": tokens.to(torch.int32)}
    if case["fork"]:
        page, ctx = case["page"], case["ctx"]
        table, spare, rows = s["table"].tolist(), s["spare"].tolist(), s["cache"].clone()
        made = []
        for i, p in enumerate(parents.view(-1).tolist()):
            old = table[i // n * K + p]
            made.append(old[:ctx // page] + [spare[i]] + [-1] * (len(old) - ctx // page - 1))
            a, z = spare[i] * page, old[ctx // page] * page
            if ctx % page:
                rows[a:a + ctx % page] = s["cache"][z:z + ctx % page]
        out |= {"table": _ints(made), "length": _ints([ctx] * (B * n)),
                **_fields64(rows, case["fmt"])}
    return out


def exact(case, seed):
    if case["op"] == "tree" and work(case)["flops"] > 8e12:
        return None
    return {"append": _exact_append, "tree": _exact_tree, "verify": _exact_verify,
            "beam": _exact_beam}[case["op"]](case, prepare(case, seed))
