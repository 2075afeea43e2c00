"""The operators around the step in numpy, 64 bits: what the GPU tests compare
with.  Written from the definitions in include/dllm.h, on [request][token]
arrays; the page layout appears only in ``pages_of`` and ``values_of``."""
import numpy as np

GROUP = 32
BIT = [(c // 2 + 4 * (c % 2)) * 4 for c in range(8)]   # first bit of channel c in its word of 8


def to_bf16(x):
    """The nearest bf16 values (ties to even) of finite x, as uint16 patterns."""
    u = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def from_bf16(u):
    return (np.asarray(u).astype(np.uint32) << 16).view(np.float32)


def quantise(x):
    """Codes [..., D], steps and zero points [..., D/32] of x [..., D]."""
    g = np.asarray(x, dtype=np.float64).reshape(*x.shape[:-1], -1, GROUP)
    with np.errstate(invalid="ignore", over="ignore"):
        low, high = np.minimum(g.min(-1), 0.0), np.maximum(g.max(-1), 0.0)
        bad = ~np.isfinite(g).all(-1)
        need = np.where(bad, 1.0, np.maximum(high - low, 1e-30)) / 15
        unit = np.exp2(np.floor(np.log2(need)) - 3)
        step = np.maximum(np.ceil(need / unit) * unit, 2.0 ** -18)
        z = np.minimum(np.rint(-np.where(bad, 0.0, low) / step), 15)
        step = np.minimum(step, 768.0)
        u = np.clip(np.rint(np.where(bad[..., None], 0.0, g) / step[..., None]) + z[..., None], 0, 15)
        u, z = np.where(bad[..., None], 0, u), np.where(bad, 0, z)
    step = np.where(bad, np.nan, step)
    return u.reshape(x.shape).astype(np.int64), step, z


def dequantise(u, step, z):
    g = u.reshape(*u.shape[:-1], u.shape[-1] // GROUP, GROUP)
    return (step[..., None] * (g - z[..., None])).reshape(u.shape)


def pages_of(k, v, page):
    """Page bytes [n, heads, page * (D + D/8)] of k and v [n, heads, page, D]."""
    n, heads, _, D = k.shape
    parts = []
    for x in (k, v):
        u, step, z = quantise(x)
        word = np.zeros((n, heads, page, D // 8), dtype=np.uint64)
        for c in range(8):
            word |= u[..., c::8].astype(np.uint64) << BIT[c]
        par = np.where(np.isnan(step), 0x7E00,
                       (np.nan_to_num(step) * 16).astype(np.float16).view(np.uint16) | z.astype(np.uint16))
        parts += [word.astype(np.uint32).view(np.uint8).reshape(n, heads, -1),
                  par.astype(np.uint16).view(np.uint8).reshape(n, heads, -1)]
    return np.concatenate(parts, -1)


def values_of(raw, page, D):
    """(k, v) [..., page, D] in 64 bits of page bytes [..., page * (D + D/8)]."""
    out = []
    lead = raw.shape[:-1]
    half = page * (D // 2 + D // 16)
    for part in (raw[..., :half], raw[..., half:]):
        word = np.ascontiguousarray(part[..., :page * D // 2]).view(np.uint32).reshape(*lead, page, D // 8)
        u = np.stack([(word >> BIT[c]) & 15 for c in range(8)], -1).reshape(*lead, page, D).astype(np.int64)
        par = np.ascontiguousarray(part[..., page * D // 2:]).view(np.uint16).reshape(*lead, page, D // GROUP)
        step = (par & 0x7F80).astype(np.uint16).view(np.float16).astype(np.float64) / 16
        step = np.where((par & 0x7C00) == 0x7C00, np.nan, step)
        out.append(dequantise(u, step, (par & 15).astype(np.float64)))
    return out


def tokens_of(pages, table, n, page, D):
    """(k, v) [heads, n, D] of one request's first n tokens."""
    need = -(-n // page)
    k, v = values_of(pages[table[:need]], page, D)   # [need, heads, page, D]
    join = lambda t: t.transpose(1, 0, 2, 3).reshape(t.shape[1], need * page, D)[:, :n]  # noqa: E731
    return join(k), join(v)


def attend(q, k, v, scale):
    """(out [L, H, D], lse [L, H], weight of each token [heads, n]) of one
    request, q [L, H, D], k and v [heads, n, D]; and the magnitudes the
    tolerances are made of: sum |q k| scale at its largest per row [L, H], and
    the attention of |v| [L, H, D]."""
    L, H, D = q.shape
    heads, n = k.shape[:2]
    G = H // heads
    out = np.zeros((L, H, D))
    spread = np.zeros((L, H, D))
    size = np.zeros((L, H))
    lse = np.full((L, H), -np.inf)
    w = np.zeros((heads, n))
    for h in range(H if n else 0):
        a = scale * (q[:, h].astype(np.float64) @ k[h // G].T)
        m = a.max(-1, keepdims=True)
        p = np.exp(a - m)
        z = p.sum(-1, keepdims=True)
        p /= z
        lse[:, h] = (m + np.log(z))[:, 0]
        out[:, h] = p @ v[h // G]
        spread[:, h] = p @ np.abs(v[h // G])
        size[:, h] = abs(scale) * (np.abs(q[:, h].astype(np.float64)) @ np.abs(k[h // G]).T).max(-1)
        w[h // G] += p.sum(0)
    return out, lse, w, size, spread


def evict(weights, keep, recent):
    """Positions that stay of one head's weights [n], ascending."""
    n = len(weights)
    k = min(max(keep, 0), n)
    r = min(recent, k)
    w = np.where(np.isnan(weights), -np.inf, weights.astype(np.float64))[: n - r]
    # a NaN sorts below every number, -inf included
    order = np.lexsort((np.arange(n - r), -w, np.isnan(weights[: n - r])))
    return np.concatenate([np.sort(order[: k - r]), np.arange(n - r, n)]).astype(np.int64)


def logprobs(x, token, top):
    """(logprob, entropy, ids, their log probabilities) of one row."""
    x = np.asarray(x, dtype=np.float64)
    ids = np.full(top, -1, dtype=np.int64)
    lp = np.full(top, np.nan)
    m = x.max()
    if not np.isfinite(m):
        return np.nan, np.nan, ids, lp
    p = np.exp(x - m)
    z = p.sum()
    lz = np.log(z)
    with np.errstate(invalid="ignore"):
        terms = np.where(p > 0, p * (x - m), 0.0)
    order = np.lexsort((np.arange(len(x)), -x))[:top]
    ids[: len(order)] = order
    lp[: len(order)] = x[order] - m - lz
    return x[token] - m - lz if 0 <= token < len(x) else np.nan, lz - terms.sum() / z, ids, lp
