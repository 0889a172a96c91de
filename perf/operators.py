"""Timed cases of the paged latent cache's operators.

A paged cache holds one latent row per token: 512 latent and 64 rope values, as
576 bf16 (1152 bytes, fmt "bf16"), or as 512 e4m3 codes, 4 float scales (one
for each 128 codes, a power of two) and 64 bf16 (656 bytes, fmt "e4m3"). A page is
page_size consecutive rows; a request's position t lies in row t % page_size
of page block_table[b][t // page_size].

  write   new tokens' rows into their slots (quantised for e4m3)
  read    selected positions back as bf16 rows, the selection buffer that the
          sparse decode attention takes
  chunk   absorbed-MLA attention of each request's newest tokens (one for a
          decode step, a few drafted ones, a prefill chunk) over its cache,
          causal among the new tokens
  verify  drafted tokens against the target's probabilities from given
          uniform numbers: how many are accepted, and the token after them

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
        # one decode step of 32 requests appends one row each
        {"name": "write_step_e4m3", "op": "write", "fmt": "e4m3", "n": 32, "slots": 8192,
         "fused": False},
        # a prefill chunk, latent and rope parts lying in one projection's output
        {"name": "write_chunk_bf16", "op": "write", "fmt": "bf16", "n": 4095, "slots": 16384,
         "fused": True},
        # a whole 32,768-token context quantised as it is written
        {"name": "write_context_e4m3", "op": "write", "fmt": "e4m3", "n": 32768, "slots": 65536,
         "fused": False},
        # one request's selection at the smallest top-k
        {"name": "read_one_e4m3", "op": "read", "fmt": "e4m3", "B": 1, "k": 256, "ctx": 4096,
         "page": 64},
        # a decode step's selections of 32 requests out of long contexts
        {"name": "read_batch_e4m3", "op": "read", "fmt": "e4m3", "B": 32, "k": 2048, "ctx": 65536,
         "page": 64},
        # the smallest decode: one token, 16 heads
        {"name": "chunk_one_bf16", "op": "chunk", "fmt": "bf16", "B": 1, "n": 1, "H": 16,
         "ctx": 4096, "page": 64, "mix": 0},
        # a decode step of 32 requests over contexts of many lengths
        {"name": "chunk_decode_e4m3", "op": "chunk", "fmt": "e4m3", "B": 32, "n": 1, "H": 128,
         "ctx": 65536, "page": 64, "mix": 1},
        # drafted tokens verified: up to four new tokens a request, small pages
        {"name": "chunk_draft_bf16", "op": "chunk", "fmt": "bf16", "B": 32, "n": 4, "H": 128,
         "ctx": 8192, "page": 16, "mix": 2},
        # chunked prefill: 2048 new tokens behind 6144 cached ones
        {"name": "chunk_prefill_bf16", "op": "chunk", "fmt": "bf16", "B": 1, "n": 2048, "H": 128,
         "ctx": 8192, "page": 64, "mix": 0},
        # several requests' ragged chunks over an 8-bit cache
        {"name": "chunk_ragged_e4m3", "op": "chunk", "fmt": "e4m3", "B": 4, "n": 500, "H": 64,
         "ctx": 16384, "page": 128, "mix": 3},
        # one request, one draft
        {"name": "verify_one", "op": "verify", "B": 1, "n": 1, "V": 32000},
        # a batch's drafts over a large vocabulary
        {"name": "verify_batch", "op": "verify", "B": 128, "n": 4, "V": 131072},
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over the logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["write", "read", "chunk", "chunk", "chunk", "verify"])
    fmt = rng.choice(["bf16", "e4m3"])
    if op == "write":
        n = _log(rng, 1, 32768)
        return {"op": op, "fmt": fmt, "n": n, "slots": rng.randint(n, 65536),
                "fused": rng.random() < 0.5}
    page = rng.choice([16, 32, 64, 128])
    if op == "read":
        ctx = _log(rng, 256, 65536)
        return {"op": op, "fmt": fmt, "B": _log(rng, 1, 32), "k": _log(rng, 1, min(2048, ctx)),
                "ctx": ctx, "page": page}
    if op == "verify":
        return {"op": op, "B": _log(rng, 1, 128), "n": rng.randint(1, 4),
                "V": _log(rng, 1000, 131072)}
    # chunk: B * n * H * ctx within the largest listed case's work and scores
    B, ctx = _log(rng, 1, 32), _log(rng, 1, 65536)
    H = rng.choice([16, 32, 64, 128, rng.randint(1, 128)])
    n = _log(rng, 1, 2048)
    n = max(1, min(n, ctx, 1_600_000_000 // (B * H * ctx)))
    return {"op": op, "fmt": fmt, "B": B, "n": n, "H": H, "ctx": ctx, "page": page,
            "mix": rng.randint(0, 1000)}


def _lengths(case):
    """New tokens and cached tokens (the new ones among them) of each request:
    all alike for mix 0, else ragged; a request may have no new token."""
    B, n, ctx, mix = case["B"], case["n"], case["ctx"], case["mix"]
    if mix == 0:
        return [n] * B, [ctx] * B
    r = random.Random(mix)
    new = [r.randint(0, n) if n > 1 else 1 for _ in range(B)]
    new[r.randrange(B)] = n
    cached = [_log(r, max(1, x), ctx) for x in new]
    cached[r.randrange(B)] = ctx
    return new, cached


def work(case):
    op = case["op"]
    if op == "write":
        return {"bytes": case["n"] * (1152 + 4 + ROW[case["fmt"]]), "flops": 0}
    if op == "read":
        return {"bytes": case["B"] * case["k"] * (ROW[case["fmt"]] + 4 + 1152), "flops": 0}
    if op == "verify":
        # one target row for each request, and the draft's at the first refusal
        rows = case["B"] * (2 - 0.7 ** case["n"])
        return {"bytes": rows * case["V"] * 4, "flops": rows * case["V"]}
    new, cached = _lengths(case)
    H = case["H"]
    pairs = sum(n * c - n * (n - 1) // 2 for n, c in zip(new, cached))
    rows = sum(c for n, c in zip(new, cached) if n)
    return {"bytes": rows * ROW[case["fmt"]] + sum(new) * H * (D + DV + 2) * 2,
            "flops": 2 * pairs * H * (D + DV)}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _pack(x, fmt):
    """bf16 rows [n][576] as cache rows (bytes [n][ROW])."""
    if fmt == "bf16":
        return x.contiguous().view(torch.uint8)
    g = x[:, :DV].float().view(-1, DV // GROUP, GROUP)
    amax = g.abs().nan_to_num(nan=0.0).amax(2)
    # the smallest power of two with amax / scale <= 448 = 0.875 * 2^9, at least 2^-120
    m, e = torch.frexp(amax.clamp(max=3.3895313892515355e38))
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


def _table(lens, width, page, g):
    """A block table [B][width] with pages in random order, -1 past a request's last."""
    used = [-(-n // page) for n in lens]
    order = torch.randperm(max(1, sum(used)), generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(lens), max(1, width)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = order[at:at + n]
        at += n
    return table, max(1, sum(used)) * page


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op = case["op"]
    s = dict(case)
    if op == "write":
        x = _rows(case["n"], g)
        if case["fused"]:
            s["latent"], s["rope"] = x[:, :DV], x[:, DV:]
        else:
            s["latent"], s["rope"] = x[:, :DV].contiguous(), x[:, DV:].contiguous()
        s["where"] = torch.randperm(case["slots"], generator=g, device=DEV)[:case["n"]].to(torch.int32)
        s["cache"] = _cache(case["slots"], case["fmt"], g)
    elif op == "read":
        B, k, ctx, page = case["B"], case["k"], case["ctx"], case["page"]
        s["table"], slots = _table([ctx] * B, -(-ctx // page), page, g)
        s["cache"] = _cache(slots, case["fmt"], g)
        s["ctx_len"] = torch.full((B,), ctx, dtype=torch.int32, device=DEV)
        pos = torch.rand(B, ctx, generator=g, device=DEV).argsort(1)[:, :k]
        s["pos"] = pos.sort(1).values.to(torch.int32).contiguous()
    elif op == "chunk":
        new, cached = _lengths(case)
        H, page = case["H"], case["page"]
        s["T"], s["most_new"], s["most_ctx"] = sum(new), max(new), max(cached)
        s["table"], slots = _table(cached, -(-max(cached) // page), page, g)
        s["cache"] = _cache(slots, case["fmt"], g)
        s["cu_q"] = torch.tensor([0] + new, device=DEV).cumsum(0).to(torch.int32)
        s["ctx_len"] = torch.tensor(cached, dtype=torch.int32, device=DEV)
        s["q"] = 1.5 * torch.randn(s["T"], H, D, generator=g, device=DEV, dtype=torch.bfloat16)
    else:
        B, n, V = case["B"], case["n"], case["V"]
        logits = 2.5 * torch.randn(B, n + 1, V, generator=g, device=DEV)
        s["target"] = torch.softmax(logits, 2)
        logits = logits[:, :n] + 0.8 * torch.randn(B, n, V, generator=g, device=DEV)
        s["draft"] = torch.softmax(logits, 2)
        noise = torch.rand(B, n, V, generator=g, device=DEV).clamp_(min=1e-20).log_().neg_().log_()
        s["drafts"] = (logits - noise).argmax(2).to(torch.int32)
        s["u"] = torch.rand(B, n + 1, generator=g, device=DEV)
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


def _plain_write(s):
    x = torch.cat([s["latent"], s["rope"]], 1)
    s["cache"][s["where"].long()] = _pack(x, s["fmt"])
    return _views(s["cache"], s["fmt"])


def _plain_read(s):
    pos = s["pos"].long()
    slot = s["table"].long().gather(1, pos // s["page"]) * s["page"] + pos % s["page"]
    return _unpack(s["cache"][slot], s["fmt"]).to(torch.bfloat16)


def _plain_chunk(s):
    B, H, n, L, page = s["B"], s["H"], s["most_new"], s["most_ctx"], s["page"]
    first, count = s["cu_q"][:-1].long(), s["cu_q"].long().diff()
    ctx = s["ctx_len"].long()
    at = torch.arange(L, device=DEV)
    slot = s["table"].long()[:, at // page].clamp(min=0) * page + at % page
    K = _unpack(s["cache"][slot], s["fmt"])                               # [B][L][576]
    i = torch.arange(n, device=DEV)
    q = s["q"][(first[:, None] + i).clamp(max=s["T"] - 1)].float()        # [B][n][H][576]
    S = torch.matmul(q.view(B, n * H, D), K.transpose(1, 2)).view(B, n, H, L)
    S *= SCALE
    limit = (ctx - count)[:, None] + i + 1                                # [B][n]
    S.masked_fill_((at >= limit[:, :, None])[:, :, None], -math.inf)
    m = S.amax(3, keepdim=True).clamp(min=-3e38)
    p = S.sub_(m).exp_()
    z = p.sum(3)
    o = torch.matmul(p.view(B, n * H, L), K[..., :DV]).view(B, n, H, DV)
    o /= z.clamp(min=1e-38).unsqueeze(3)
    lse = m.squeeze(3) + z.log()
    t = torch.arange(s["T"], device=DEV)
    b = torch.bucketize(t, s["cu_q"][1:].long(), right=True)
    return {"out": o[b, t - first[b]].to(torch.bfloat16), "lse": lse[b, t - first[b]]}


def _plain_verify(s):
    B, n, V = s["B"], s["n"], s["V"]
    x = s["drafts"].long().unsqueeze(2)
    p, q = s["target"][:, :n].gather(2, x).squeeze(2), s["draft"].gather(2, x).squeeze(2)
    take = s["u"][:, :n].double() * q.double() < p.double()
    a = take.long().cumprod(1).sum(1)
    b = torch.arange(B, device=DEV)
    p = s["target"][b, a].double()
    q = s["draft"][b, a.clamp(max=n - 1)].double() * (a < n).unsqueeze(1)
    w = (p - q).clamp_(min=0)
    w = torch.where(w.sum(1, keepdim=True) > 0, w, p)
    below = w.cumsum(1)
    token = (below <= s["u"][:, n:].double() * below[:, -1:]).sum(1).clamp(max=V - 1)
    i = torch.arange(n + 1, device=DEV)
    drafts = torch.cat([s["drafts"].long(), token[:, None]], 1)
    out = torch.where(i < a[:, None], drafts,
                      torch.where(i == a[:, None], token[:, None], torch.full_like(drafts, -1)))
    return {"tokens": out.to(torch.int32), "accepted": a.to(torch.int32)}


def _own(s):
    import decode_dsa_kv_gb300 as d
    op = s["op"]
    if op == "verify":
        B, n = s["B"], s["n"]
        tokens = torch.empty(B, n + 1, dtype=torch.int32, device=DEV)
        accepted = torch.empty(B, dtype=torch.int32, device=DEV)
        d.check(d.ts_verify_drafts(s["drafts"], None, s["target"], s["V"], s["draft"], s["V"],
                                   s["u"], B, n, s["V"], tokens, accepted), "ts_verify_drafts")
        return {"tokens": tokens, "accepted": accepted}
    cache, fmt = s["cache"], {"bf16": d.DSA_CACHE_BF16, "e4m3": d.DSA_CACHE_E4M3}[s["fmt"]]
    if op == "write":
        d.check(d.dsa_cache_write(s["latent"], s["latent"].stride(0), s["rope"],
                                  s["rope"].stride(0), s["where"], s["n"], cache,
                                  cache.shape[0], fmt), "dsa_cache_write")
        return _views(cache, s["fmt"])
    if op == "read":
        sel = torch.empty(s["B"], s["k"], D, dtype=torch.bfloat16, device=DEV)
        d.check(d.dsa_cache_read(cache, cache.shape[0], fmt, s["table"], s["table"].shape[1],
                                 s["page"], s["pos"], s["ctx_len"], s["B"], s["k"], sel),
                "dsa_cache_read")
        return sel
    T, H = s["T"], s["H"]
    out = torch.empty(T, H, DV, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(T, H, dtype=torch.float32, device=DEV)
    size = d.sfa_chunk_workspace_size(T, s["B"], H)
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)
    d.check(d.sfa_mla_chunk(s["q"], H * D, s["cu_q"], T, s["B"], H, cache, cache.shape[0], fmt,
                            s["table"], s["table"].shape[1], s["page"], s["ctx_len"], 1, SCALE,
                            out, lse, ws, size), "sfa_mla_chunk")
    return {"out": out, "lse": lse}


def run(state):
    if own:
        return _own(state)
    return {"write": _plain_write, "read": _plain_read, "chunk": _plain_chunk,
            "verify": _plain_verify}[state["op"]](state)


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


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "write":
        out = {k: v.double() for k, v in _views(s["cache"], case["fmt"]).items()}
        where = s["where"].long()
        x, r = s["latent"].double(), s["rope"].double()
        if case["fmt"] == "bf16":
            out["rows"][where] = torch.cat([x, r], 1)
            return out
        scales = out["scales"]
        for i in range(4):
            part = x[:, 128 * i:128 * i + 128]
            top = part.abs().amax(1)
            e = torch.ceil(torch.log2(top / 448))
            e = torch.where(torch.exp2(e - 1) * 448 >= top, e - 1, e)     # log2 rounded up
            e = torch.where(torch.exp2(e) * 448 < top, e + 1, e).clamp(min=-120)
            out["codes"][where, 128 * i:128 * i + 128] = part / torch.exp2(e)[:, None]
            scales[where, i] = torch.exp2(e)
        out["rope"][where] = r
        return out
    if op == "read":
        B, k, page = case["B"], case["k"], case["page"]
        out = []
        for b in range(B):
            t = s["pos"][b].long()
            out.append(_values64(s["cache"][s["table"][b].long()[t // page] * page + t % page],
                                 case["fmt"]))
        return torch.stack(out)
    if op == "verify":
        n, V = case["n"], case["V"]
        tokens, accepted = [], []
        for b in range(case["B"]):
            p, q = s["target"][b].double(), s["draft"][b].double()
            a = 0
            while a < n and s["u"][b, a].item() * q[a, s["drafts"][b, a]].item() \
                    < p[a, s["drafts"][b, a]].item():
                a += 1
            w = p[a] if a == n else torch.clamp(p[a] - q[a], min=0)
            if w.sum().item() == 0:
                w = p[a]
            c = torch.cumsum(w, 0)
            t = int(torch.searchsorted(c, c[-1:] * s["u"][b, n].double(), right=True).item())
            tokens.append(s["drafts"][b, :a].tolist() + [min(t, V - 1)] + [-1] * (n - a))
            accepted.append(a)
        return {"tokens": torch.tensor(tokens, dtype=torch.int32),
                "accepted": torch.tensor(accepted, dtype=torch.int32)}
    if work(case)["flops"] > 8e12:
        return None
    new, cached = _lengths(case)
    H, page = case["H"], case["page"]
    outs, lses = [], []
    at = 0
    for b, (n, c) in enumerate(zip(new, cached)):
        t = torch.arange(c, device=DEV)
        K = _values64(s["cache"][s["table"][b].long()[t // page] * page + t % page], case["fmt"])
        step = max(1, 100_000_000 // (H * c))
        for i in range(0, n, step):
            k = min(n, i + step)
            q = s["q"][at + i:at + k].double().reshape(-1, D)
            z = (q @ K.T) / math.sqrt(D)
            last = (c - n + torch.arange(i, k, device=DEV)).repeat_interleave(H)
            z = torch.where(t[None] <= last[:, None], z, -math.inf)
            lse = torch.logsumexp(z, 1)
            outs.append((torch.exp(z - lse[:, None]) @ K[:, :DV]).view(k - i, H, DV))
            lses.append(lse.view(k - i, H))
        at += n
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
