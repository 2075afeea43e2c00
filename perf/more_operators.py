"""More serving operators around the denoise step, as cases to time and compare.

Three groups: drawing tokens from the step's logits (temperature, top-k, min-p and top-p, by given random numbers); the
pages of a cache (forking requests, growing them, freeing, copying pages to another pool, closing a pool's gaps); and
the product that makes the logits, in 8-bit floating point with a scale for each block of 128.  ``run`` computes them
either in plain torch operations (``own`` false) or through the package's entry points (``own`` true).
"""
import math

import numpy as np
import torch

own = False

BLOCK = 128
F32, F64 = torch.float32, torch.float64
E4M3 = torch.float8_e4m3fn


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one token of one request: the smallest draw, where latency counts
        {"name": "sample_one", "op": "sample", "rows": 1, "of": 32, "V": 126464, "ldv": 126464, "kind": "mixed",
         "lens": 1},
        # a few blocks over an odd vocabulary with a padded row, every filter in use
        {"name": "sample_odd", "op": "sample", "rows": 37, "of": 64, "V": 32003, "ldv": 32008, "kind": "mixed",
         "lens": 2},
        # the masked positions of a batch of 64 blocks of 32, temperature alone: nothing may be left out of a row
        {"name": "sample_plain", "op": "sample", "rows": 987, "of": 2048, "V": 126464, "ldv": 126464, "kind": "plain",
         "lens": 3},
        # the masked positions of a batch of 128 blocks of 32, requests of every kind together
        {"name": "sample_batch", "op": "sample", "rows": 1851, "of": 4096, "V": 151936, "ldv": 151936,
         "kind": "mixed", "lens": 4},
        # one request's cache forked three ways for a try each, grown by a block and given back
        {"name": "fork_one", "op": "fork", "B": 8, "forks": 3, "layers": 2, "heads": 4, "D": 128, "page": 32,
         "high": 1280, "grow": 32, "lens": 5},
        # 64 requests of a batch, four tries each, all layers' pools
        {"name": "fork_batch", "op": "fork", "B": 384, "forks": 256, "layers": 16, "heads": 4, "D": 128, "page": 64,
         "high": 1280, "grow": 32, "lens": 6},
        # a request's pages are parked in another pool
        {"name": "copy_pages", "op": "copy", "pages": 700, "n_pages": 2048, "layers": 16, "heads": 4, "D": 128,
         "page": 32, "lens": 7},
        # a small pool's gaps are closed
        {"name": "compact_small", "op": "compact", "B": 16, "n_pages": 700, "layers": 2, "heads": 4, "D": 128,
         "page": 32, "used": 0.4, "lens": 8},
        # a pool of a serving batch, a third in use, all layers
        {"name": "compact_large", "op": "compact", "B": 128, "n_pages": 16384, "layers": 16, "heads": 4, "D": 128,
         "page": 32, "used": 0.33, "lens": 9},
        # the logits of one block's masked positions: the whole head is read for a few rows
        {"name": "head_block", "op": "head", "rows": 21, "of": 32, "K": 4096, "N": 126464},
        # an odd vocabulary, and a width that ends inside a block of scales
        {"name": "head_odd", "op": "head", "rows": 300, "of": 333, "K": 2000, "N": 32003},
        # the masked positions of a batch of 128 blocks of 32
        {"name": "head_batch", "op": "head", "rows": 1851, "of": 4096, "K": 3584, "N": 151936},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sample", "sample", "sample", "fork", "copy", "compact", "head", "head", "weights"])
    if op == "sample":
        rows, V = _log_int(rng, 1, 1851), _log_int(rng, 1000, 151936)
        return {"op": op, "rows": rows, "of": rows + rng.randrange(0, 64), "V": V, "ldv": -(-V // 8) * 8,
                "kind": rng.choice(["mixed", "mixed", "plain"]), "lens": rng.randrange(1 << 20)}
    if op == "head":
        rows = _log_int(rng, 1, 1851)
        return {"op": op, "rows": rows, "of": rows + rng.randrange(0, 64), "K": 16 * _log_int(rng, 8, 256),
                "N": _log_int(rng, 1000, 126464)}
    if op == "weights":
        return {"op": op, "K": 16 * _log_int(rng, 8, 256), "N": _log_int(rng, 100, 32000)}
    pool = {"op": op, "layers": rng.randrange(1, 17), "heads": rng.choice([1, 2, 3, 4, 8]),
            "D": rng.choice([64, 128, 128]), "page": rng.choice([16, 32, 64, 128]), "lens": rng.randrange(1 << 20)}
    if op == "fork":
        forks = _log_int(rng, 1, 128)
        return {**pool, "B": forks + rng.randrange(1, 64), "forks": forks, "high": _log_int(rng, 16, 2048),
                "grow": rng.choice([1, 8, 32, 200])}
    n_pages = max(2, min(_log_int(rng, 40, 8192), 2 ** 27 // (pool["heads"] * pool["page"] * pool["D"])))
    if op == "copy":
        return {**pool, "n_pages": n_pages, "pages": max(1, int(n_pages * rng.uniform(0.01, 0.9)))}
    return {**pool, "B": min(_log_int(rng, 1, 64), n_pages), "n_pages": n_pages, "used": rng.uniform(0.05, 0.95)}


def _fork_plan(case):
    """Sources, destinations, lengths of all requests and their pages, whatever the inputs' seed."""
    r = np.random.RandomState(case["lens"])
    B, forks, page = case["B"], case["forks"], case["page"]
    old = B - forks                                        # requests that hold pages; the rest are free rows
    lens = np.zeros(B, dtype=np.int32)
    lens[:old] = r.randint(1, case["high"] + 1, size=old)
    rows = r.permutation(B).astype(np.int32)               # live and free rows lie mixed in the batch
    lens[rows] = lens.copy()
    src = rows[:old][(np.arange(forks) // 4 if case["forks"] > 3 else np.zeros(forks, dtype=np.int64)) % old]
    return src.astype(np.int32), rows[old:], lens, -(-lens // page)


def _compact_plan(case):
    """Held pages of each request, and how many that makes."""
    r = np.random.RandomState(case["lens"])
    used = max(case["B"], int(case["n_pages"] * case["used"]))
    cut = np.sort(r.choice(used + 1, case["B"] - 1, replace=True)) if case["B"] > 1 else np.zeros(0, dtype=np.int64)
    return np.diff(np.concatenate([[0], cut, [used]])).astype(np.int32), used


def _page_bytes(case):
    """Bytes of one page over all layers: codes and weights."""
    return case["layers"] * case["heads"] * case["page"] * (case["D"] + case["D"] // 8 + 4)


def work(case):
    op = case["op"]
    if op == "sample":
        n = case["rows"] * case["V"]
        return {"bytes": n * 2 + case["rows"] * (4 * 5 + 4 + 8), "flops": 4 * n}
    if op == "fork":
        src, _, lens, _ = _fork_plan(case)
        tails = int((lens[src] % case["page"] != 0).sum())
        entries = int((-(-(lens[src] + case["grow"]) // case["page"])).sum())
        return {"bytes": 2 * tails * _page_bytes(case) + 24 * entries, "flops": 0}
    if op == "copy":
        return {"bytes": 2 * case["pages"] * _page_bytes(case) + 8 * case["pages"], "flops": 0}
    if op == "compact":
        held, used = _compact_plan(case)
        moved = int((_used_pages(case) >= used).sum())
        return {"bytes": 2 * moved * _page_bytes(case) + 12 * case["n_pages"] + 8 * int(held.sum()), "flops": 0}
    blocks = -(-case["K"] // BLOCK)
    if op == "weights":
        return {"bytes": case["N"] * case["K"] * 3 + 4 * blocks * -(-case["N"] // BLOCK),
                "flops": 2 * case["N"] * case["K"]}
    M, N, K = case["rows"], case["N"], case["K"]
    return {"bytes": M * K * 2 + N * K + 4 * blocks * -(-N // BLOCK) + M * N * 2, "flops": 2 * M * N * K}


def _used_pages(case):
    """Which pages of the pool are in use, in the order in which they were taken."""
    _, used = _compact_plan(case)
    return np.random.RandomState(case["lens"] + 1).permutation(case["n_pages"])[:used]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _t(a, dev):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dev)


def _pools(gen, case, n_pages, dev):
    """Every layer's codes [n_pages, heads, bytes] and attention weights [n_pages, heads, page]."""
    heads, page, D = case["heads"], case["page"], case["D"]
    made = []
    for _ in range(case["layers"]):
        words = torch.randint(-2 ** 31, 2 ** 31, (n_pages, heads, page * (D + D // 8) // 4), dtype=torch.int32,
                              generator=gen, device=dev)
        made += [words.view(torch.uint8), torch.rand(n_pages, heads, page, generator=gen, device=dev)]
    return made


def _weights(gen, N, K, dev):
    """8-bit weights [N, K] and scales [N/128, K/128]: rows of their own size, as a trained head's tokens have."""
    codes = torch.empty(N, K, dtype=E4M3, device=dev)
    scale = torch.empty(-(-N // BLOCK), -(-K // BLOCK), device=dev)
    at = BLOCK * max(1, 2 ** 26 // (K * BLOCK))
    for k in range(0, N, at):
        c = min(at, N - k)
        w = torch.randn(c, K, generator=gen, device=dev)
        w *= torch.exp(0.3 * torch.randn(c, 1, generator=gen, device=dev)) / math.sqrt(K)
        codes[k:k + c], scale[k // BLOCK:-(-(k + c) // BLOCK)] = _quantise(w.to(torch.bfloat16), BLOCK)
    return codes, scale


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed * 1000003 + 29)
    op = case["op"]
    s = {"case": case}
    if op == "sample":
        V, ldv, of, rows = case["V"], case["ldv"], case["of"], case["rows"]
        x = s["logits"] = torch.empty(of, ldv, dtype=torch.bfloat16, device=dev)
        for k in range(0, of, 256):
            c = min(256, of - k)
            spread = 1.0 + 2.0 * torch.rand(c, 1, generator=gen, device=dev)
            x[k:k + c] = torch.randn(c, ldv, generator=gen, device=dev) * spread
        peak = torch.randint(0, V, (of, 3), generator=gen, device=dev)   # a few likely tokens, as sure as comes
        x.scatter_(1, peak, (6.0 + 14.0 * torch.rand(of, 3, generator=gen, device=dev)).to(torch.bfloat16))
        x[:, V // 2] = -math.inf                                         # a token that may not be said
        s["rows"] = torch.sort(torch.randperm(of, generator=gen, device=dev)[:rows])[0].to(torch.int32)
        s["u"] = torch.rand(rows, generator=gen, device=dev)
        r = np.random.RandomState(case["lens"])                          # the requests' settings: of the case
        s["temperature"] = _t(r.choice([0.6, 0.8, 1.0, 1.0, 1.3], rows).astype(np.float32), dev)
        if case["kind"] == "mixed":
            s["temperature"] = torch.where(_t(r.rand(rows) < 0.05, dev), 0.0, s["temperature"])   # greedy ones
            s["top_k"] = _t(r.choice([0, 0, 1, 20, 50, 1000], rows).astype(np.int32), dev)
            s["top_p"] = _t(r.choice([1.0, 1.0, 0.95, 0.9, 0.5], rows).astype(np.float32), dev)
            s["min_p"] = _t(r.choice([0.0, 0.0, 0.0, 0.02, 0.1], rows).astype(np.float32), dev)
        return s
    if op == "head":
        of, K = case["of"], case["K"]
        x = torch.randn(of, K, generator=gen, device=dev)
        x *= torch.exp(0.7 * torch.randn(K, generator=gen, device=dev))   # a few strong channels
        s["x"] = x.to(torch.bfloat16)
        s["rows"] = torch.sort(torch.randperm(of, generator=gen, device=dev)[:case["rows"]])[0].to(torch.int32)
        s["w"], s["w_scale"] = _weights(gen, case["N"], K, dev)
        return s
    if op == "weights":
        w = torch.randn(case["N"], case["K"], generator=gen, device=dev)
        w *= torch.exp(0.3 * torch.randn(case["N"], 1, generator=gen, device=dev)) / math.sqrt(case["K"])
        s["w"] = w.to(torch.bfloat16)
        return s
    if op == "copy":
        n, n_pages = case["pages"], case["n_pages"]
        s["pools"], s["parked"] = _pools(gen, case, n_pages, dev), _pools(gen, case, n, dev)
        s["src"] = torch.randperm(n_pages, generator=gen, device=dev)[:n].to(torch.int32)
        s["dst"] = torch.randperm(n, generator=gen, device=dev).to(torch.int32)
        return s
    if op == "fork":
        src, dst, lens, held = _fork_plan(case)
        most = -(-(case["high"] + case["grow"]) // case["page"])
        need = int((-(-(lens[src] + case["grow"]) // case["page"])).sum())
        n_pages = int(held.sum()) + need + 5
        order = torch.randperm(n_pages, generator=gen, device=dev).to(torch.int32)
        own_pages = torch.arange(most, device=dev)[None] < _t(held, dev)[:, None]
        s["table"] = torch.zeros(case["B"], most, dtype=torch.int32, device=dev)
        s["table"][own_pages] = order[:int(held.sum())]
        s["refs"] = torch.zeros(n_pages, dtype=torch.int32, device=dev)
        s["refs"][order[:int(held.sum())].long()] = 1
        s.update(src=_t(src, dev), dst=_t(dst, dev), lens=_t(lens, dev), held=_t(held, dev),
                 pools=_pools(gen, case, n_pages, dev))
        return s
    held, used = _compact_plan(case)
    pages = _used_pages(case).astype(np.int32)
    most = int(held.max())
    table = np.zeros((case["B"], most), dtype=np.int32)
    table[np.arange(most)[None] < held[:, None]] = pages
    refs = np.zeros(case["n_pages"], dtype=np.int32)
    refs[pages] = 1
    s.update(table=_t(table, dev), refs=_t(refs, dev), held=_t(held, dev), pools=_pools(gen, case, case["n_pages"], dev))
    s["scattered"] = s["table"].clone(), s["refs"].clone()
    return s


# ---------------------------------------------------------------------------
# the operators
# ---------------------------------------------------------------------------
def run(state):
    case = state["case"]
    return (_run_own if own else _run_plain)[case["op"]](case, state)


def _plain_sample(case, s):
    # in 64 bits: a draw lies next to one of V borders
    x, at = torch.sort(s["logits"][s["rows"].long(), :case["V"]].to(F32) + 0.0, dim=-1, descending=True, stable=True)
    T = s["temperature"].to(F64)[:, None]
    w = torch.exp((x - x[:, :1].to(F64)) / torch.where(T > 0, T, torch.ones_like(T)))
    j = torch.arange(case["V"], device=x.device)
    left = torch.where(T > 0, case["V"], 1)
    if case["kind"] == "mixed":
        k = s["top_k"].long()[:, None]
        left = torch.minimum(left, torch.where(k > 0, k, case["V"]))
        left = torch.minimum(left, (w >= s["min_p"].to(F64)[:, None]).sum(-1, keepdim=True))
    c = torch.cumsum(torch.where(j < left, w, torch.zeros_like(w)), -1)
    if case["kind"] == "mixed":
        p = s["top_p"].to(F64)[:, None]
        left = torch.where(p < 1, torch.minimum(left, (c < p * c[:, -1:]).sum(-1, keepdim=True) + 1), left)
    mass = c.gather(1, left - 1)
    i = torch.minimum((c <= s["u"].to(F64)[:, None] * mass).sum(-1, keepdim=True), left - 1)
    return {"tokens": at.gather(1, i)[:, 0].to(torch.int32), "prob": (w.gather(1, i) / mass)[:, 0].to(F32)}


def _plain_take(refs, need):
    """Free pages, lowest first, for requests that need some each: [requests, most needed], and which are theirs."""
    free = torch.nonzero(refs == 0)[:, 0]
    j = torch.arange(max(1, int(need.max())), device=refs.device)[None]
    theirs = j < need[:, None]
    return free[((torch.cumsum(need, 0) - need)[:, None] + j).clamp(max=free.numel() - 1)], theirs


def _plain_fork(case, s):
    page, refs, table, src, dst = case["page"], s["refs"], s["table"], s["src"].long(), s["dst"].long()
    s["lens"][dst] = s["lens"][src]
    full, tail = s["lens"][src] // page, s["lens"][src] % page != 0
    fresh = _plain_take(refs, tail.long())[0][:, 0]
    j = torch.arange(table.shape[1], device=refs.device)[None]
    shared = j < full[:, None]
    old = table[src].long()
    refs.index_add_(0, old[shared], torch.ones_like(old[shared], dtype=torch.int32))
    rows = torch.where(shared, old, table[dst].long())
    at = torch.nonzero(tail)[:, 0]
    rows[at, full.long()[at]] = fresh[at]
    table[dst] = rows.to(torch.int32)
    refs[fresh[at]] = 1
    for pool in s["pools"]:
        pool[fresh[at]] = pool[old[at, full.long()[at]]]
    held = full + tail
    # each copy grows
    more = -(-(s["lens"][dst] + case["grow"]) // page) - held
    new, theirs = _plain_take(refs, more.long())
    b, k = torch.nonzero(theirs, as_tuple=True)
    table[dst[b], (held[b] + k)] = new[b, k].to(torch.int32)
    refs[new[b, k]] = 1
    forked = table.clone(), refs.clone()
    # and gives its pages back
    held = held + more
    mine = table[dst].long()[j < held[:, None]]
    refs.index_add_(0, mine, -torch.ones_like(mine, dtype=torch.int32))
    s["held"][dst] = 0
    fresh = torch.where(tail, fresh, -torch.ones_like(fresh)).to(torch.int32)
    return {"table": forked[0], "refs": forked[1], "fresh": fresh, "freed": refs, "held": s["held"], "lens": s["lens"],
            "pools": s["pools"]}


def _plain_copy(case, s):
    for a, b in zip(s["pools"], s["parked"]):
        b[s["dst"].long()] = a[s["src"].long()]
    return s["parked"]


def _plain_compact(case, s):
    s["table"].copy_(s["scattered"][0])
    s["refs"].copy_(s["scattered"][1])
    refs, table = s["refs"], s["table"]
    used = refs > 0
    n = used.sum()
    at = torch.arange(refs.numel(), device=refs.device)
    movers, holes = at[used & (at >= n)], at[~used & (at < n)]
    new = torch.where(used, at, -torch.ones_like(at))
    new[movers] = holes
    mine = torch.arange(table.shape[1], device=refs.device)[None] < s["held"][:, None]
    table[mine] = new[table[mine].long()].to(torch.int32)
    refs[holes] = refs[movers]
    refs[movers] = 0
    for pool in s["pools"]:
        pool[holes] = pool[movers]
    return {"table": table, "refs": refs, "used": n.to(torch.int32).reshape(1), "map": new.to(torch.int32),
            "pools": s["pools"]}


def _quantise(x, block_rows):
    """Codes of x [n, K] and a scale for every 128 columns of `block_rows` rows, in 32 bits."""
    n, K = x.shape
    rows, cols = -(-n // block_rows), -(-K // BLOCK)
    g = torch.nn.functional.pad(x.to(F32), (0, cols * BLOCK - K, 0, rows * block_rows - n))
    g = g.reshape(rows, block_rows, cols, BLOCK)
    top = g.abs().amax((1, 3), keepdim=True)
    scale = (top / torch.full_like(top, 448.0)).clamp(min=2.0 ** -126)   # by a tensor: rounded once
    codes = (g / scale).clamp(-448, 448).reshape(rows * block_rows, cols * BLOCK)[:n, :K].to(E4M3)
    return codes, scale[:, 0, :, 0]


def _widen(codes, scale, block_rows):
    """The values of codes [n, K], in 32 bits."""
    n, K = codes.shape
    return codes.to(F32) * scale.repeat_interleave(block_rows, 0)[:n].repeat_interleave(BLOCK, 1)[:, :K]


def _plain_head(case, s):
    codes, scale = _quantise(s["x"][s["rows"].long()], 1)
    y = (_widen(codes, scale, 1) @ _widen(s["w"], s["w_scale"], BLOCK).T).to(torch.bfloat16)
    return {"logits": torch.nn.functional.pad(y, (0, -case["N"] % 8)), "scale": scale}


def _plain_weights(case, s):
    codes, scale = _quantise(s["w"], BLOCK)
    return {"codes": codes, "scale": scale}


def _own_sample(case, s):
    import denoise_step_token_gb300 as dllm

    return dllm.sample(s["logits"], s["u"], V=case["V"], rows=s["rows"], temperature=s["temperature"],
                       top_k=s.get("top_k"), top_p=s.get("top_p"), min_p=s.get("min_p"))


def _own_fork(case, s):
    import denoise_step_token_gb300 as dllm

    page = case["page"]
    fresh = dllm.page_fork(s["pools"], s["refs"], s["table"], s["held"], s["lens"], s["src"], s["dst"], page_size=page)
    dllm.page_grow(s["refs"], s["table"], s["held"], s["lens"], s["dst"], case["grow"], page_size=page)
    forked = s["table"].clone(), s["refs"].clone()
    dllm.page_free(s["refs"], s["table"], s["held"], s["dst"])
    return {"table": forked[0], "refs": forked[1], "fresh": fresh, "freed": s["refs"], "held": s["held"],
            "lens": s["lens"], "pools": s["pools"]}


def _own_copy(case, s):
    import denoise_step_token_gb300 as dllm

    dllm.page_copy(s["pools"], s["parked"], s["src"], s["dst"])
    return s["parked"]


def _own_compact(case, s):
    import denoise_step_token_gb300 as dllm

    s["table"].copy_(s["scattered"][0])
    s["refs"].copy_(s["scattered"][1])
    out = dllm.page_compact(s["pools"], s["refs"], s["table"], s["held"])
    return {"table": s["table"], "refs": s["refs"], "used": out["used"], "map": out["map"], "pools": s["pools"]}


def _own_head(case, s):
    import denoise_step_token_gb300 as dllm

    codes, scale = dllm.fp8_quantize(s["x"], rows=s["rows"])
    return {"logits": dllm.fp8_matmul(codes, scale, s["w"], s["w_scale"]), "scale": scale}


def _own_weights(case, s):
    import denoise_step_token_gb300 as dllm

    codes, scale = dllm.fp8_quantize(s["w"], block_rows=BLOCK)
    return {"codes": codes, "scale": scale}


_run_plain = {"sample": _plain_sample, "fork": _plain_fork, "copy": _plain_copy, "compact": _plain_compact,
              "head": _plain_head, "weights": _plain_weights}
_run_own = {"sample": _own_sample, "fork": _own_fork, "copy": _own_copy, "compact": _own_compact, "head": _own_head,
            "weights": _own_weights}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_sample(case, s):
    """The probability with which each row's token was drawn; the tokens themselves are whole numbers."""
    prob = []
    off = {"top_k": 0, "top_p": 1.0, "min_p": 0.0}
    setting = {k: s[k].double().tolist() if k in s else [v] * case["rows"] for k, v in off.items()}
    for i, (r, T, u) in enumerate(zip(s["rows"].tolist(), s["temperature"].double().tolist(), s["u"].double().tolist())):
        if T == 0:
            prob.append(1.0)
            continue
        x = s["logits"][r, :case["V"]].double()
        value = torch.sort(x, descending=True)[0]
        w = torch.softmax(value / T, 0)
        n = int(min(setting["top_k"][i] or case["V"], int((w >= setting["min_p"][i] * w[0]).sum())))
        c = torch.cumsum(w[:n], 0)
        if setting["top_p"][i] < 1:
            n = min(n, int(torch.searchsorted(c, setting["top_p"][i] * c[-1])) + 1)
        mass = c[n - 1]
        k = min(int(torch.searchsorted(c[:n], u * mass, right=True)), n - 1)
        prob.append(float(w[k] / mass))
    return {"tokens": None, "prob": torch.tensor(prob, dtype=F64)}


def _exact_codes(x, block_rows):
    """Values [n, K] that the codes stand for, and the scales, by the format: 3 bits behind the leading one, steps of
    2^-9 below 2^-6."""
    n, K = x.shape
    at = torch.arange(n, device=x.device) // block_rows
    scale = torch.zeros(int(at[-1]) + 1, -(-K // BLOCK), dtype=F64, device=x.device)
    y = torch.empty(n, K, dtype=F64, device=x.device)
    for c in range(scale.shape[1]):
        part = x[:, c * BLOCK:(c + 1) * BLOCK].double()
        top = torch.zeros(scale.shape[0], dtype=F64, device=x.device)
        top.index_reduce_(0, at, part.abs().amax(1), "amax")
        scale[:, c] = (top / 448).clamp(min=2.0 ** -126)
        v = part / scale[at, c, None]
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
        y[:, c * BLOCK:(c + 1) * BLOCK] = (v / step).round() * step
    return y, scale


def _exact_head(case, s):
    K = case["K"]
    q, scale = _exact_codes(s["x"][s["rows"].long()], 1)
    for c in range(scale.shape[1]):
        q[:, c * BLOCK:(c + 1) * BLOCK] *= scale[:, c, None]
    y = torch.zeros(case["rows"], -(-case["N"] // 8) * 8, dtype=F64, device=q.device)
    of = s["w_scale"].double()
    for n in range(0, case["N"], 64 * BLOCK):
        m = min(case["N"], n + 64 * BLOCK)
        w = s["w"][n:m].double()
        row = torch.arange(n, m, device=q.device) // BLOCK
        y[:, n:m] = q @ (w * of[row][:, torch.arange(K, device=q.device) // BLOCK]).T
    return {"logits": y, "scale": scale}


def _exact_weights(case, s):
    y, scale = _exact_codes(s["w"], BLOCK)
    return {"codes": y, "scale": scale}


def exact(case, seed):
    if case["op"] in ("fork", "copy", "compact"):   # these move values, and compute none
        return None
    s = prepare(case, seed)
    return {"sample": _exact_sample, "head": _exact_head, "weights": _exact_weights}[case["op"]](case, s)
