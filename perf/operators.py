"""The serving operators around the denoise step, as cases to time and compare.

Four operators: the report of token log probabilities over the step's logits, the write of keys and values into a
paged cache of 4-bit codes, the attention of a block's queries over that cache (with the attention weight every
cached token receives, where asked for), and the eviction of a cache's least attended tokens.  ``run`` computes them
either in plain torch operations in 32 bits (``own`` false) or through the package's entry points (``own`` true).

The cache's format, shared by all sides: a pool of pages, each ``page`` tokens of every key/value head; a page of one
head holds the key codes [page][D/2], the key parameters [page][D/32] of 16 bits, then the same two for the values.
A group of 32 channels has a step s of 4 significant bits and a zero point z: code u stands for s * (u - z), which 8
significant bits hold exactly.  Its parameter is 16 s as an fp16 pattern (the low 7 bits of the significand are
zero) with z in the low 4 bits.  A 32-bit word holds 8 channels; channels 2i and 2i + 1 are its bits [4i, 4i + 4) and
[16 + 4i, 16 + 4i + 4).
"""
import math

import numpy as np
import torch

own = False

GROUP = 32
F32 = torch.float32


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one finished token of one request, its five best alternatives: the smallest report, where latency counts
        {"name": "logprobs_one", "op": "logprobs", "rows": 1, "of": 32, "V": 126464, "ldv": 126464, "top": 5,
         "dtype": "bf16"},
        # a few blocks' tokens over a 32-bit LM head with an odd vocabulary
        {"name": "logprobs_odd_f32", "op": "logprobs", "rows": 37, "of": 64, "V": 32003, "ldv": 32008, "top": 20,
         "dtype": "f32"},
        # the masked positions of a batch of 128 blocks of 32, a Dream-sized vocabulary: the step's own batch
        {"name": "logprobs_batch", "op": "logprobs", "rows": 1851, "of": 4096, "V": 151936, "ldv": 151936, "top": 20,
         "dtype": "bf16"},
        # the current blocks of a small batch go into the cache once per denoise step
        {"name": "write_block", "op": "write", "B": 16, "W": 32, "ragged": False, "heads": 4, "D": 128, "page": 32,
         "lens": 5},
        # 64 left-padded prompts of 64 to 1024 tokens, keys and values of 32 heads out of a fused projection
        {"name": "write_prompts", "op": "write", "B": 64, "W": 1024, "ragged": True, "heads": 32, "D": 128,
         "page": 64, "lens": 6},
        # one token per request over short caches, grouped heads: a decode step of a small batch
        {"name": "attend_token", "op": "attend", "B": 8, "L": 1, "q_heads": 28, "heads": 4, "D": 128, "page": 32,
         "low": 0, "high": 1280, "lens": 7, "weights": False},
        # one token per request over long caches
        {"name": "attend_token_long", "op": "attend", "B": 16, "L": 1, "q_heads": 28, "heads": 4, "D": 128,
         "page": 64, "low": 8191, "high": 32768, "lens": 8, "weights": False},
        # blocks of 32 with a key/value head for every head: LLaDA's attention over prompts and committed blocks
        {"name": "attend_block_mha", "op": "attend", "B": 64, "L": 32, "q_heads": 32, "heads": 32, "D": 128,
         "page": 64, "low": 96, "high": 1280, "lens": 9, "weights": False},
        # blocks of 32, seven query heads to each key/value head: the batch of 128 requests of the denoise benchmark;
        # the block's last step, which also gives the weights by which the cache is thinned
        {"name": "attend_block_gqa", "op": "attend", "B": 128, "L": 32, "q_heads": 28, "heads": 4, "D": 128,
         "page": 32, "low": 96, "high": 1280, "lens": 10, "weights": True},
        # two long contexts, just before they are thinned
        {"name": "attend_block_long", "op": "attend", "B": 2, "L": 32, "q_heads": 28, "heads": 4, "D": 128,
         "page": 64, "low": 100003, "high": 131072, "lens": 11, "weights": True},
        # short caches thinned to half between two blocks
        {"name": "evict_short", "op": "evict", "B": 16, "heads": 4, "D": 128, "page": 32, "low": 96, "high": 1280,
         "lens": 12, "keep": 0.5, "recent": 32},
        # long caches thinned to a quarter
        {"name": "evict_long", "op": "evict", "B": 8, "heads": 4, "D": 128, "page": 64, "low": 40000, "high": 65536,
         "lens": 13, "keep": 0.25, "recent": 64},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logprobs", "write", "attend", "attend", "attend", "evict"])
    if op == "logprobs":
        V = _log_int(rng, 1000, 152000)
        dtype = rng.choice(["bf16", "bf16", "f32"])
        rows = _log_int(rng, 1, 1024 if dtype == "f32" else 2048)
        return {"op": op, "rows": rows, "of": rows + rng.randrange(0, 64), "V": V, "ldv": -(-V // 8) * 8,
                "top": rng.choice([0, 1, 5, 20, 32]), "dtype": dtype}
    heads, group = rng.choice([(1, 8), (2, 5), (4, 7), (8, 4), (8, 1), (32, 1), (3, 3)])
    common = {"heads": heads, "D": rng.choice([64, 128, 128]), "page": rng.choice([16, 32, 64, 128]),
              "lens": rng.randrange(1 << 20)}
    if op == "write":
        W = _log_int(rng, 1, 1024)
        B = max(1, min(_log_int(rng, 1, 64), 2 ** 21 // (W * heads)))
        return {"op": op, "B": B, "W": W, "ragged": rng.random() < 0.5, **common}
    if op == "attend":
        L = rng.choice([1, 1, 4, 8, 16, 32, 32, 64, rng.randrange(2, 64)])
        high = _log_int(rng, 64, 65536)
        rows = heads * group * L
        most = min(2 ** 33 // (rows * high), 2 ** 31 // (heads * high * 128 * 4))   # scores and keys of the plain form
        B = max(1, min(_log_int(rng, 1, 64), most // 4))
        return {"op": op, "B": B, "L": L, "q_heads": heads * group, "low": rng.choice([0, high // 2, high]),
                "high": high, "weights": rng.random() < 0.4, **common}
    high = _log_int(rng, 64, 65536)
    B = max(1, min(_log_int(rng, 1, 16), 2 ** 21 // (heads * high)))
    return {"op": op, "B": B, "low": rng.choice([0, high // 2, high]), "high": high,
            "keep": rng.choice([0.1, 0.25, 0.5, 0.9]), "recent": rng.choice([0, 1, 32, 64]), **common}


def _lens(case, low, high):
    """The requests' lengths: of the case, whatever the inputs' seed."""
    return np.random.RandomState(case["lens"]).randint(low, high + 1, size=case["B"]).astype(np.int32)


def _keep(case):
    return np.ceil(_lens(case, case["low"], case["high"]) * case["keep"]).astype(np.int32)


def _write_counts(case):
    if not case["ragged"]:
        return np.full(case["B"], case["W"], dtype=np.int32)
    return _lens(case, min(64, case["W"]), case["W"])


def work(case):
    op = case["op"]
    if op == "logprobs":
        size = 2 if case["dtype"] == "bf16" else 4
        n = case["rows"] * case["V"]
        return {"bytes": n * size + case["rows"] * (8 + 8 + 8 * case["top"]), "flops": 6 * n}
    D, heads = case["D"], case["heads"]
    token = D + D // 8   # bytes of one token of one head, keys and values
    if op == "write":
        n = int(_write_counts(case).sum()) * heads
        return {"bytes": n * (2 * D * 2 + token + 2 * D * 2), "flops": n * 2 * D * 8}
    if op == "attend":
        n = int(_lens(case, case["low"], case["high"]).sum())
        rows = case["L"] * case["q_heads"]
        nbytes = n * heads * token + case["B"] * rows * (D * 2 * 2 + 4)
        flops = 4 * n * rows * D
        if case["weights"]:   # the weights need every score again once its row's sum is known
            nbytes += n * heads * 8
            flops += 2 * n * rows * D
        return {"bytes": nbytes, "flops": flops}
    n = int(_lens(case, case["low"], case["high"]).sum()) * heads
    k = int(_keep(case).sum()) * heads
    return {"bytes": n * 4 + k * (2 * token + 4 + 4), "flops": n}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _quantise(x):
    """Codes [..., D/2] (uint8) and parameters [..., D/32] (int16 patterns) of x [..., D]; 32-bit arithmetic."""
    D = x.shape[-1]
    g = x.to(F32).reshape(*x.shape[:-1], D // GROUP, GROUP)
    low, high = g.amin(-1, keepdim=True).clamp(max=0), g.amax(-1, keepdim=True).clamp(min=0)
    step = (high - low) * 16 / torch.full_like(low, 15.0)   # by a tensor: rounded once, as the definition has it
    step = ((step.view(torch.int32) + 0xFFFFF) & ~0xFFFFF).view(F32).clamp(2.0 ** -14, 12288.0)   # up to 4 bits
    s = step / 16
    z = torch.round(-low / s).clamp(0, 15)
    u = (torch.round(g / s) + z).clamp(0, 15).to(torch.uint8)
    n = u.reshape(*x.shape[:-1], D // 8, 4, 2).transpose(-1, -2).reshape(*x.shape[:-1], D // 2, 2)
    par = step.to(torch.float16).view(torch.int16) | z.to(torch.int16)
    return n[..., 0] | (n[..., 1] << 4), par[..., 0]


def _values(codes, par):
    """What codes [..., D/2] and parameters [..., D/32] stand for, in 32 bits."""
    D = codes.shape[-1] * 2
    n = torch.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], D // 8, 2, 4)
    u = n.transpose(-1, -2).reshape(*codes.shape[:-1], D // GROUP, GROUP).to(F32)
    s = (par & 0x7F80).view(torch.float16).to(F32) / 16
    return (s[..., None] * (u - (par & 15).to(F32)[..., None])).reshape(*codes.shape[:-1], D)


def _parts(pages, page, D):
    """The four parts of pages [..., bytes]: key codes and parameters, value codes and parameters, as bytes."""
    a, b = page * D // 2, page * D // 16
    lead = pages.shape[:-1]
    return (pages[..., :a].reshape(*lead, page, D // 2), pages[..., a:a + b].reshape(*lead, page, D // 16),
            pages[..., a + b:2 * a + b].reshape(*lead, page, D // 2),
            pages[..., 2 * a + b:].reshape(*lead, page, D // 16))


def _params(raw):
    """Parameters [..., D/32] of their bytes [..., D/16]."""
    return raw.contiguous().view(torch.int16)


def _made_pages(x, y, page):
    """Pages [n, heads, bytes] of keys x and values y [n, heads, page, D]."""
    n, heads, _, D = x.shape
    pieces = []
    for t in (x, y):
        codes, par = _quantise(t)
        pieces += [codes.reshape(n, heads, -1), par.contiguous().view(torch.uint8).reshape(n, heads, -1)]
    return torch.cat(pieces, -1)


def _table(gen, B, max_pages, dev, spare=0):
    """Page numbers [B, max_pages] in random order, no page twice, out of B * max_pages + spare."""
    return torch.randperm(B * max_pages + spare, generator=gen, device=dev)[:B * max_pages].to(torch.int32).reshape(
        B, max_pages)


def _pool(gen, n, heads, page, D, dev):
    """A pool whose keys have a few strong channels, as rotated keys have, and a common offset."""
    chan = torch.exp(0.5 * torch.randn(heads, 1, D, generator=gen, device=dev))
    shift = 0.5 * torch.randn(heads, 1, D, generator=gen, device=dev)
    pages = torch.empty(n, heads, page * (D + D // 8), dtype=torch.uint8, device=dev)
    at = max(1, 2 ** 26 // (heads * page * D))
    for k in range(0, n, at):
        c = min(at, n - k)
        x = torch.randn(c, heads, page, D, generator=gen, device=dev).mul_(chan).add_(shift).to(torch.bfloat16)
        y = torch.randn(c, heads, page, D, generator=gen, device=dev).to(torch.bfloat16)
        pages[k:k + c] = _made_pages(x, y, page)
    return pages


def _t(a, dev):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dev)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed * 1000003 + 17)
    op = case["op"]
    s = {"case": case}
    if op == "logprobs":
        dtype = torch.bfloat16 if case["dtype"] == "bf16" else F32
        V, ldv, of, rows = case["V"], case["ldv"], case["of"], case["rows"]
        s["logits"] = torch.empty(of, ldv, dtype=dtype, device=dev)
        for k in range(0, of, 256):
            c = min(256, of - k)
            s["logits"][k:k + c] = torch.randn(c, ldv, generator=gen, device=dev)
        peak = torch.randint(0, V, (of, 1), generator=gen, device=dev)   # a planted best token, as confident as comes
        s["logits"].scatter_(1, peak, (4.0 + 12.0 * torch.rand(of, 1, generator=gen, device=dev)).to(dtype))
        s["logits"][:, V // 2] = -math.inf                               # a token that may not be said
        s["rows"] = torch.sort(torch.randperm(of, generator=gen, device=dev)[:rows])[0].to(torch.int32)
        other = torch.randint(0, V, (rows,), generator=gen, device=dev)
        best = torch.rand(rows, generator=gen, device=dev) < 0.7
        s["tokens"] = torch.where(best, peak[s["rows"].long(), 0], other).to(torch.int32)
        return s
    B, heads, D, page = case["B"], case["heads"], case["D"], case["page"]
    if op == "write":
        W = case["W"]
        n = _write_counts(case)
        pos = np.random.RandomState(case["lens"] + 1).randint(0, 1024, size=B).astype(np.int32)
        most = -(-(1024 + W) // page)
        qkv = torch.randn(B, W, 3, heads, D, generator=gen, device=dev)  # keys and values out of a fused projection
        qkv *= torch.exp(0.5 * torch.randn(3, heads, D, generator=gen, device=dev))
        qkv = qkv.to(torch.bfloat16)
        s.update(k=qkv[:, :, 1], v=qkv[:, :, 2], first=_t(W - n, dev), pos=_t(pos, dev),
                 table=_table(gen, B, most, dev), count=_t(n, dev),
                 pages=torch.zeros(B * most, heads, page * (D + D // 8), dtype=torch.uint8, device=dev),
                 k_out=torch.zeros(B, W, heads, D, dtype=torch.bfloat16, device=dev),
                 v_out=torch.zeros(B, W, heads, D, dtype=torch.bfloat16, device=dev))
        return s
    lens = _lens(case, case["low"], case["high"])
    most = max(1, -(-case["high"] // page))
    if op == "attend":
        s["table"] = _table(gen, B, most, dev, 3)
        s["pages"] = _pool(gen, B * most + 3, heads, page, D, dev)
        s["lens"] = _t(lens, dev)
        s["q"] = torch.randn(B, case["L"], case["q_heads"], D, generator=gen, device=dev).to(torch.bfloat16)
        if case["weights"]:
            s["prior"] = torch.rand(B * most + 3, heads, page, generator=gen, device=dev)
            s["weights"] = torch.zeros_like(s["prior"])
        return s
    dst = max(1, -(-int(_keep(case).max()) // page))
    both = torch.randperm(B * (most + dst), generator=gen, device=dev).to(torch.int32)
    s["table"], s["dst_table"] = both[:B * most].reshape(B, most), both[B * most:].reshape(B, dst)
    s["pages"] = _pool(gen, B * (most + dst), heads, page, D, dev)
    w = torch.rand(B * (most + dst), heads, page, generator=gen, device=dev)
    w = torch.exp(6.0 * w * w)                                          # few tokens draw most of the weight
    s["weights"] = torch.where(torch.rand(w.shape, generator=gen, device=dev) < 0.05, torch.zeros_like(w), w)
    s["lens"], s["keep"] = _t(lens, dev), _t(_keep(case), dev)
    return s


# ---------------------------------------------------------------------------
# the operators
# ---------------------------------------------------------------------------
def run(state):
    case = state["case"]
    return (_run_own if own else _run_plain)[case["op"]](case, state)


def _plain_logprobs(case, s):
    x = s["logits"][s["rows"].long(), :case["V"]].to(F32)
    m = x.amax(-1, keepdim=True)
    d = x - m
    e = torch.exp(d)
    z = e.sum(-1, keepdim=True)
    entropy = (torch.log(z) - torch.where(e > 0, e * d, torch.zeros_like(d)).sum(-1, keepdim=True) / z)[:, 0]
    logz = torch.log(z)
    out = {"logprob": (d.gather(1, s["tokens"].long()[:, None]) - logz)[:, 0], "entropy": entropy}
    if case["top"]:
        # the largest values, ties to the lowest token: by keys that are all different
        bits = x.contiguous().view(torch.int32).long()
        key = torch.where(bits >= 0, bits, -2 ** 31 - bits - 1) * 2 ** 20 + (2 ** 20 - 1) - torch.arange(
            case["V"], device=x.device)
        ids = (2 ** 20 - 1) - (torch.topk(key, case["top"], dim=-1)[0] & (2 ** 20 - 1))
        out["top_ids"] = ids.to(torch.int32)
        out["top_logprobs"] = d.gather(1, ids) - logz
    return out


def _plain_write(case, s):
    B, W, page, D = case["B"], case["W"], case["page"], case["D"]
    col = torch.arange(W, device=s["k"].device)[None]
    valid = (col >= s["first"][:, None]) & (col < (s["first"] + s["count"])[:, None])
    pos = (s["pos"][:, None] + col - s["first"][:, None]).clamp(min=0).long()
    at = valid.nonzero(as_tuple=True)
    where = s["table"].gather(1, pos // page).long()[at], (pos % page)[at]
    parts = _parts(s["pages"], page, D)   # views: a page's parts are contiguous ranges of it
    out = {"pages": s["pages"]}
    k_codes, k_par = _quantise(s["k"][at])
    v_codes, v_par = _quantise(s["v"][at])
    parts[0][where[0], :, where[1]] = k_codes
    parts[1][where[0], :, where[1]] = k_par.contiguous().view(torch.uint8)
    parts[2][where[0], :, where[1]] = v_codes
    parts[3][where[0], :, where[1]] = v_par.contiguous().view(torch.uint8)
    s["k_out"][at] = _values(k_codes, k_par).to(torch.bfloat16)
    s["v_out"][at] = _values(v_codes, v_par).to(torch.bfloat16)
    return {**out, "k": s["k_out"], "v": s["v_out"]}


def _plain_attend(case, s):
    B, L, H, heads, D, page = case["B"], case["L"], case["q_heads"], case["heads"], case["D"], case["page"]
    got = s["pages"][s["table"].long()]                                  # [B, max_pages, heads, bytes]
    kc, kp, vc, vp = (t.transpose(1, 2).reshape(B, heads, -1, t.shape[-1]) for t in _parts(got, page, D))
    K, V = _values(kc, _params(kp)), _values(vc, _params(vp))            # [B, heads, S, D]
    n = K.shape[2]
    valid = (torch.arange(n, device=K.device)[None] < s["lens"][:, None])[:, None, None]
    q = s["q"].to(F32).reshape(B, L, heads, H // heads, D).permute(0, 2, 1, 3, 4).reshape(B, heads, -1, D)
    x = (q @ K.transpose(-1, -2) / math.sqrt(D)).masked_fill(~valid, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(x - m)
    z = p.sum(-1, keepdim=True)
    o = (p @ V) / torch.where(z > 0, z, torch.ones_like(z))
    back = lambda t: t.reshape(B, heads, L, H // heads, -1).permute(0, 2, 1, 3, 4).reshape(B, L, H, -1)  # noqa: E731
    out = {"out": back(o).to(torch.bfloat16), "lse": back(m + torch.log(z))[..., 0]}
    if case["weights"]:
        w = (p / torch.where(z > 0, z, torch.ones_like(z))).sum(2)       # [B, heads, S]
        w = w.reshape(B, heads, -1, page).transpose(1, 2)
        at = s["table"].long()
        valid = valid.reshape(B, 1, -1, page).transpose(1, 2)
        s["weights"][at] = torch.where(valid, s["prior"][at] + w, s["weights"][at])
        out["weights"] = s["weights"]
    return out


def _plain_evict(case, s):
    B, heads, D, page = case["B"], case["heads"], case["D"], case["page"]
    n, dst = s["table"].shape[1] * page, s["dst_table"].shape[1] * page
    dev = s["pages"].device
    table = s["table"].long()
    w = s["weights"][table].transpose(1, 2).reshape(B, heads, n)
    j = torch.arange(n, device=dev)
    lens = s["lens"][:, None, None]
    k = torch.minimum(s["keep"], s["lens"])[:, None, None]
    r = k.clamp(max=case["recent"])
    order = torch.where(j >= lens, -math.inf, torch.where(j >= lens - r, math.inf, w))
    rank = torch.sort(torch.sort(order, dim=-1, descending=True, stable=True)[1], dim=-1)[1]   # the inverse order
    kept = rank < k
    # kept positions first, in their order
    src = torch.sort(torch.where(kept, j, j + n), dim=-1)[0][..., :dst]
    if dst > n:
        src = torch.cat([src, src.new_full((B, heads, dst - n), 2 * n)], -1)
    used = src < n
    src = torch.where(used, src, torch.zeros_like(src))
    b, h, i = used.nonzero(as_tuple=True)
    f = src[b, h, i]
    fp, tp = table[b, f // page], s["dst_table"].long()[b, i // page]
    for part in _parts(s["pages"], page, D):
        part[tp, h, i % page] = part[fp, h, f % page]
    s["weights"][tp, h, i % page] = s["weights"][fp, h, f % page]
    src = torch.where(used, src, torch.full_like(src, -1)).to(torch.int32)
    return {"pages": s["pages"], "weights": s["weights"], "lens": k[:, 0, 0].to(torch.int32), "src": src}


def _own_logprobs(case, s):
    import denoise_step_token_gb300 as dllm

    return dllm.token_logprobs(s["logits"], s["tokens"], V=case["V"], top=case["top"], rows=s["rows"])


def _own_write(case, s):
    import denoise_step_token_gb300 as dllm

    dllm.kv4_write(s["k"], s["v"], s["pages"], s["table"], s["pos"], first=s["first"], count=s["count"],
                   k_out=s["k_out"], v_out=s["v_out"])
    return {"pages": s["pages"], "k": s["k_out"], "v": s["v_out"]}


def _own_attend(case, s):
    import denoise_step_token_gb300 as dllm

    return dllm.kv4_attend(s["q"], s["pages"], s["table"], s["lens"], prior=s.get("prior"), weights=s.get("weights"))


def _own_evict(case, s):
    import denoise_step_token_gb300 as dllm

    out = dllm.kv4_evict(s["pages"], s["weights"], s["table"], s["lens"], s["keep"], s["dst_table"],
                         recent=case["recent"])
    return {"pages": s["pages"], "weights": s["weights"], "lens": out["lens"], "src": out["src"]}


_run_plain = {"logprobs": _plain_logprobs, "write": _plain_write, "attend": _plain_attend, "evict": _plain_evict}
_run_own = {"logprobs": _own_logprobs, "write": _own_write, "attend": _own_attend, "evict": _own_evict}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
_CHANNEL = [(c // 2 + 4 * (c % 2)) * 4 for c in range(8)]   # channel c's first bit in its word


def _exact_values(raw_codes, raw_par):
    """64-bit values [..., D] of code bytes [..., D/2] and parameter bytes [..., D/16]."""
    word = raw_codes.contiguous().view(torch.int32)
    bits = torch.tensor(_CHANNEL, device=word.device)
    u = ((word[..., None] >> bits) & 15).reshape(*word.shape[:-1], -1)
    par = raw_par.contiguous().view(torch.int16).int().repeat_interleave(GROUP, -1)
    s = (1 + ((par >> 7) & 7).double() / 8) * torch.exp2((par >> 10).double() - 19)
    return (u - (par & 15)) * s


def _exact_logprobs(case, s):
    logprob, entropy, top = [], [], []
    for r, tok in zip(s["rows"].tolist(), s["tokens"].tolist()):
        x = s["logits"][r, :case["V"]].double()
        lse = torch.logsumexp(x, 0)
        p = torch.exp(x - lse)
        logprob.append(x[tok] - lse)
        entropy.append(-torch.special.xlogy(p, p).sum())
        if case["top"]:
            top.append(torch.sort(x, descending=True)[0][:case["top"]] - lse)
    out = {"logprob": torch.stack(logprob), "entropy": torch.stack(entropy)}
    if case["top"]:
        out.update(top_ids=None, top_logprobs=torch.stack(top))
    return out


def _exact_write(case, s):
    out = {"pages": None}
    for name in ("k", "v"):
        x = s[name].double()
        B, W, heads, D = x.shape
        g = x.reshape(B, W, heads, D // GROUP, GROUP)
        low, high = g.min(-1, keepdim=True)[0].clamp(max=0), g.max(-1, keepdim=True)[0].clamp(min=0)
        need = (high - low).clamp(min=2.0 ** -60) / 15
        e = torch.floor(torch.log2(need)) - 3                            # the step: up to 4 significant bits
        step = (torch.ceil(need / torch.exp2(e)) * torch.exp2(e)).clamp(2.0 ** -18, 768.0)
        z = (-low / step).round().clamp(0, 15)
        y = (((g / step).round() + z).clamp(0, 15) - z) * step
        y = y.reshape(B, W, heads, D)
        col = torch.arange(W, device=x.device)[None]
        valid = (col >= s["first"][:, None]) & (col < (s["first"] + s["count"])[:, None])
        out[name] = torch.where(valid[:, :, None, None], y, torch.zeros_like(y))
    return out


def _exact_attend(case, s):
    B, L, H, heads, D, page = case["B"], case["L"], case["q_heads"], case["heads"], case["D"], case["page"]
    dev = s["q"].device
    out = torch.zeros(B, L, H, D, dtype=torch.float64, device=dev)
    lse = torch.full((B, L, H), -math.inf, dtype=torch.float64, device=dev)
    weights = s["weights"].double() if case["weights"] else None
    a = page * D // 2
    for b, n in enumerate(s["lens"].tolist()):
        if n <= 0:
            continue
        ids = s["table"][b, :-(-n // page)].long()
        for h in range(heads):
            raw = s["pages"][ids, h]
            cut = [raw[:, i:j].reshape(len(ids) * page, -1)[:n] for i, j in (
                (0, a), (a, a + a // 8), (a + a // 8, 2 * a + a // 8), (2 * a + a // 8, 2 * a + a // 4))]
            K, V = _exact_values(cut[0], cut[1]), _exact_values(cut[2], cut[3])
            mine = slice(h * (H // heads), (h + 1) * (H // heads))
            q = s["q"][b, :, mine].double().reshape(-1, D)
            x = q @ K.T / math.sqrt(D)
            z = torch.logsumexp(x, -1)
            p = torch.exp(x - z[:, None])
            out[b, :, mine] = (p @ V).reshape(L, -1, D)
            lse[b, :, mine] = z.reshape(L, -1)
            if weights is not None:
                j = torch.arange(n, device=dev)
                weights[ids[j // page], h, j % page] = s["prior"][ids[j // page], h, j % page].double() + p.sum(0)
    got = {"out": out, "lse": lse}
    return {**got, "weights": weights} if weights is not None else got


def exact(case, seed):
    if case["op"] == "evict":   # moves values, and computes none
        return None
    s = prepare(case, seed)
    return {"logprobs": _exact_logprobs, "write": _exact_write, "attend": _exact_attend}[case["op"]](case, s)
