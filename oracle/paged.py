"""The paged latent cache: row formats, chunk attention and draft verification.

Rows are 576 bf16 values (512 latent, 64 rope). The 8-bit format stores the
latent part as e4m3 codes with one power-of-two scale for each 128 values:

    s    = the smallest 2^e, e >= -120, with max |x| / s <= 448 (NaN left out;
           2^120 where a value is infinite)
    code = the e4m3 value nearest to x / s, ties to even, at most 448 in size

Attention of a chunk ([TS] MLA section: one latent row is K and V; chunked
prefill and drafted tokens attend causally to the cache they were appended
to): token i of a request's n newest, over the positions j < limit of its
ctx_len cached ones, limit = ctx_len - n + i + 1 (causal) or ctx_len:

    s_j = scale * q . K_j,  out = softmax(s) K[:, 0:512],  lse = log sum exp s

and out = 0, lse = -inf where no position is left.

Verification of drafts: x_i is accepted while u_i q_i(x_i) < p_i(x_i); after a
accepted drafts the next token is the first t whose running sum of
w = max(p_a - q_a, 0) (p_a after the last draft, or where w vanishes) exceeds
u_n sum w; in whole multiples of 2^-60. A sum of 0, or of 16 or more (2^64 - 1
multiples), has no such t: -1.
"""
import math

import numpy as np

from .sfa import bf16_bits_to_f64

D_LATENT = 512
GROUP = 128
E4M3_ROW = 656


def e4m3_table() -> np.ndarray:
    """The 256 values of e4m3: sign, 4 exponent bits (bias 7), 3 mantissa bits;
    no infinities, 0x7f and 0xff are NaN."""
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10)
        if (c & 0x7f) == 0x7f:
            v = math.nan
        out[c] = -v if c & 0x80 else v
    return out


_TABLE = e4m3_table()


def scale_of(group: np.ndarray) -> float:
    a = np.abs(group[~np.isnan(group)])
    top = a.max() if a.size else 0.0
    if math.isinf(top):
        return 2.0 ** 120
    e = -120
    while top > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def to_e4m3(y: np.ndarray) -> np.ndarray:
    """Codes of the nearest e4m3 values of float64 y (ties to even, saturating)."""
    y = np.asarray(y, dtype=np.float64)
    a = np.minimum(np.abs(np.where(np.isnan(y), 0.0, y)), 448.0)
    _, e = np.frexp(a)                       # a in [2^(e-1), 2^e)
    step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    r = np.rint(a / step) * step             # ties to even
    pos = np.searchsorted(_TABLE[:127], r)
    assert np.array_equal(_TABLE[pos], r)
    code = pos.astype(np.uint8) | np.where(np.signbit(y), 0x80, 0).astype(np.uint8)
    return np.where(np.isnan(y), 0x7f, code).astype(np.uint8)


def pack_row(row_bits: np.ndarray, fmt: str) -> np.ndarray:
    """One latent row (uint16 [576] bf16 bits) as the cache's bytes."""
    row_bits = np.asarray(row_bits, dtype=np.uint16)
    if fmt == "bf16":
        return row_bits.view(np.uint8).copy()
    x = bf16_bits_to_f64(row_bits)
    codes, scales = [], []
    for g in range(D_LATENT // GROUP):
        part = x[g * GROUP:(g + 1) * GROUP]
        s = scale_of(part)
        scales.append(s)
        codes.append(to_e4m3(part / s))
    return np.concatenate([np.concatenate(codes), np.array(scales, np.float32).view(np.uint8),
                           row_bits[D_LATENT:].view(np.uint8)])


def unpack_row(raw: np.ndarray, fmt: str) -> np.ndarray:
    """Float64 values [576] that a cache row stands for."""
    raw = np.ascontiguousarray(raw, dtype=np.uint8)
    if fmt == "bf16":
        return bf16_bits_to_f64(raw.view(np.uint16))
    scales = raw[512:528].copy().view(np.float32).astype(np.float64)
    with np.errstate(over="ignore"):
        lat = _TABLE[raw[:512]] * np.repeat(scales, GROUP)
    lat = np.where(np.abs(lat) >= 2.0 ** 128, np.copysign(np.inf, lat), lat)
    return np.concatenate([lat, bf16_bits_to_f64(raw[528:].copy().view(np.uint16))])


def chunk_attention(q: np.ndarray, K: np.ndarray, ctx: int, causal: bool, scale: float):
    """q float64 [n][H][576], K float64 [ctx][576] -> out [n][H][512], lse [n][H], and,
    for error bounds, the weighted mean of |V| and the largest scale * sum |q||k|."""
    n, H, _ = q.shape
    out = np.zeros((n, H, D_LATENT))
    mean_abs = np.zeros((n, H, D_LATENT))
    lse = np.full((n, H), -np.inf)
    size = np.zeros((n, H))
    for i in range(n):
        limit = max(0, ctx - n + i + 1) if causal else ctx
        if limit == 0:
            continue
        k = K[:limit]
        s = scale * (q[i] @ k.T)
        m = s.max(axis=1, keepdims=True)
        p = np.exp(s - m)
        z = p.sum(axis=1, keepdims=True)
        out[i] = (p @ k[:, :D_LATENT]) / z
        mean_abs[i] = (p @ np.abs(k[:, :D_LATENT])) / z
        lse[i] = (m + np.log(z))[:, 0]
        size[i] = abs(scale) * (np.abs(q[i]) @ np.abs(k).T).max(axis=1)
    return out, lse, mean_abs, size


def verify_drafts(drafts, n_draft: int, target, draft, u):
    """One request: drafts [n], target float32 [n+1][V], draft float32 [n][V] or
    None, u float32 [n+1] -> (tokens [n+1], accepted), whole-number arithmetic."""
    n, V = len(drafts), target.shape[1]

    def fixed(p):
        p = np.asarray(p, dtype=np.float64)
        good = (p >= 0) & (p < 2)
        return [int(math.ldexp(v, 60)) if g else 0 for v, g in zip(p, good)]

    a = 0
    while a < n_draft:
        x = int(drafts[a])
        if not 0 <= x < V:
            break
        p = float(target[a, x])
        q = 1.0 if draft is None else float(draft[a, x])
        if not (0 <= p < 2 and 0 <= q < 2) or not float(u[a]) * q < p:
            break
        a += 1
    p = fixed(target[a])
    w = list(p)
    if a < n_draft:
        if draft is None:
            if 0 <= int(drafts[a]) < V:
                w[int(drafts[a])] = 0
        else:
            w = [max(x - y, 0) for x, y in zip(p, fixed(draft[a]))]
    if sum(w) == 0:
        w = p
    total = sum(w)
    token = -1
    if 0 < total < 2 ** 64 - 1:
        r = int(math.ldexp(float(u[n]), 64)) * total >> 64
        run = 0
        for t in range(V):
            run += w[t]
            if run > r:
                token = t
                break
    return [int(x) for x in drafts[:a]] + [token] + [-1] * (n - a), a
