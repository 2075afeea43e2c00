"""The 4-bit cache on the GPU against its definition in 64 bits.

Tolerances, from the operators' own roundings:
- what is written, read and moved: exact (codes, parameters, values, choices);
- a score: its products are exact, its sum is held in 32 bits over D/16 steps
  of the tensor cores, which may cut rather than round: within 2^-19 of
  sum |q k| scale, and 2^-21 of its own size through the base-2 scale; lse and
  the tokens' weights inherit that, the weights with 2^-20 for the
  exponentials and their 32-bit sums;
- the output: softmax weights rounded to fp16 (2^-11 of each, and 2^-25 of the
  row's largest for those below fp16's normal range), values exact, the sum
  rounded to bf16 (8 significant bits: 2^-8)."""
import numpy as np
import pytest

import kv4_reference as ref

pytestmark = pytest.mark.gpu


def score_tol(size, lse):
    return 2.0 ** -19 * size + 2.0 ** -21 * np.abs(np.where(np.isfinite(lse), lse, 0.0)) + 2.0 ** -21


class Cache:
    """A random cache: pages in random order, slots past the lengths full of NaN."""

    def __init__(self, rng, lens, heads, D, page, extra=2, q_scale=1.0, spare=2):
        self.lens = np.asarray(lens, dtype=np.int32)
        self.page, self.D, self.heads = page, D, heads
        B = len(lens)
        most = max(1, -(-int(self.lens.max(initial=0)) // page)) + extra
        n = B * most + spare
        k = rng.standard_normal((n, heads, page, D)) * np.exp(0.5 * rng.standard_normal((heads, 1, D)))
        v = rng.standard_normal((n, heads, page, D))
        self.k = ref.from_bf16(ref.to_bf16(k))
        self.v = ref.from_bf16(ref.to_bf16(v))
        self.table = rng.permutation(n)[: B * most].reshape(B, most).astype(np.int32)
        for b, ln in enumerate(self.lens):
            for j in range(int(ln), most * page):
                self.k[self.table[b, j // page], :, j % page] = np.nan
                self.v[self.table[b, j // page], :, j % page] = np.nan
        self.pages = ref.pages_of(self.k, self.v, page)

    def upload(self, dev):
        import torch
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
        return t(self.pages), t(self.table), t(self.lens)


def bf16(x, dev):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16).to(dev)


def run_attend(dllm, cache, q, *, scale=None, weights=False, strided=False):
    import torch
    dev = torch.device("cuda", 0)
    pages, table, lens = cache.upload(dev)
    B, L, H, D = q.shape
    if strided:   # a slice of a fused projection
        fused = torch.full((B, L, 3 * H, D), float("nan"), dtype=torch.bfloat16, device=dev)
        fused[:, :, H:2 * H] = bf16(q, dev)
        tq = fused[:, :, H:2 * H]
    else:
        tq = bf16(q, dev)
    prior = w = None
    if weights:
        prior = torch.rand(pages.shape[0], cache.heads, cache.page, device=dev)
        w = torch.full_like(prior, 77.0)
    out = dllm.kv4_attend(tq, pages, table, lens, scale=scale, prior=prior, weights=w)
    assert dllm.get_device_error(dev) == 0
    got = {k: v.float().cpu().numpy() for k, v in out.items()}
    return got, None if prior is None else prior.cpu().numpy()


def check_attend(dllm, cache, q, *, scale=None, weights=False, strided=False):
    q = ref.from_bf16(ref.to_bf16(q))
    got, prior = run_attend(dllm, cache, q, scale=scale, weights=weights, strided=strided)
    D, page = cache.D, cache.page
    s = D ** -0.5 if scale is None else scale
    want_w = None if prior is None else np.full(prior.shape, 77.0)
    tol_w = None if prior is None else np.zeros(prior.shape)
    for b, n in enumerate(cache.lens):
        k, v = ref.tokens_of(cache.pages, cache.table[b], int(n), page, D)
        out, lse, w, size, spread = ref.attend(q[b], k, v, s)
        tol = score_tol(size, lse)
        assert np.array_equal(np.isneginf(lse), np.isneginf(got["lse"][b]))
        fin = np.isfinite(lse)
        assert (np.abs(got["lse"][b][fin] - lse[fin]) <= tol[fin]).all(), (b, n)
        bound = 2.0 ** -8 * 1.01 * np.abs(out) + (2.0 ** -11 + 2 * tol[..., None]) * spread + 2.0 ** -24 * n * 4
        assert (np.abs(got["out"][b] - out) <= bound).all(), (b, n, np.abs(got["out"][b] - out).max())
        if prior is not None:
            for j in range(int(n)):
                p = cache.table[b, j // page]
                want_w[p, :, j % page] = prior[p, :, j % page].astype(np.float64) + w[:, j]
                tol_w[p, :, j % page] = w[:, j] * (2 * tol.max(initial=0) + 2.0 ** -20) + 2.0 ** -23 * want_w[p, :, j % page]
    if prior is not None:
        assert (np.abs(got["weights"] - want_w) <= tol_w).all()
    return got


# name: (lengths, L, query heads, heads, D, page)
SHAPES = {
    "one": ([1], 1, 1, 1, 128, 16),
    "empty": ([0, 5, 0], 3, 2, 1, 64, 16),
    "token": ([0, 1, 15, 16, 17, 31, 33, 700], 1, 28, 4, 128, 32),
    "token_mha": ([5, 127, 128, 129], 1, 6, 6, 64, 16),
    "token_wide_group": ([300, 2049], 1, 24, 1, 128, 64),
    "block_mha": ([32, 33, 95, 640], 32, 3, 3, 128, 64),
    "block_gqa": ([32, 127, 129, 511, 2], 32, 14, 2, 128, 32),
    "block_gqa_64": ([64, 128, 300], 32, 8, 1, 64, 128),
    "block_odd": ([77, 256], 5, 9, 3, 128, 256),
    "block_129_rows": ([257, 131], 43, 3, 1, 128, 16),
    "block_long_rows": ([150], 100, 7, 1, 128, 32),
    "split": ([5000, 1, 3], 4, 4, 2, 128, 64),
    "split_rows": ([4111], 32, 7, 1, 128, 16),
}


@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("name", SHAPES)
def test_attend(dllm, name, weights):
    lens, L, H, heads, D, page = SHAPES[name]
    rng = np.random.default_rng(len(name) + sum(lens))
    cache = Cache(rng, lens, heads, D, page)
    check_attend(dllm, cache, rng.standard_normal((len(lens), L, H, D)), weights=weights, strided=weights)


@pytest.mark.parametrize("L", [2, 32])
@pytest.mark.parametrize("factor", [0.0, 1e-20, 1e-3, 40.0, 1e6, 1e20])
def test_attend_query_sizes(dllm, factor, L):
    """Queries of any size: equal weights (0), subnormal in fp16 without their
    scale, one token taking all (40 and beyond)."""
    rng = np.random.default_rng(9)
    cache = Cache(rng, [200, 45], 2, 128, 32)
    q = rng.standard_normal((2, L, 8, 128)) * factor
    scale = 128 ** -0.5 if factor < 1e3 else 40.0 / factor
    check_attend(dllm, cache, q, scale=scale, weights=True)


@pytest.mark.parametrize("L,H", [(1, 4), (32, 14)])
def test_attend_scores_that_grow(dllm, L, H):
    """Every tile's scores exceed the last one's: the running offset moves each
    time, and what came before fades to nothing."""
    rng = np.random.default_rng(10)
    n = 900
    cache = Cache(rng, [n], 2, 128, 32)
    d = np.ones(128) / 8
    for sign in (1, -1):
        ramp = sign * np.linspace(-30, 30, n)
        for j in range(n):
            cache.k[cache.table[0, j // 32], :, j % 32] = ramp[j] * d
        cache.pages = ref.pages_of(cache.k, cache.v, 32)
        check_attend(dllm, cache, np.broadcast_to(8 * d, (1, L, H, 128)), scale=1.0, weights=True)


def test_attend_negative_scale_and_aliased_prior(dllm):
    import torch
    rng = np.random.default_rng(11)
    cache = Cache(rng, [70, 130], 2, 64, 16)
    q = rng.standard_normal((2, 6, 4, 64))
    check_attend(dllm, cache, q, scale=-0.3)
    dev = torch.device("cuda", 0)
    pages, table, lens = cache.upload(dev)
    w = torch.rand(pages.shape[0], 2, 16, device=dev)
    apart = dllm.kv4_attend(bf16(q, dev), pages, table, lens, prior=w.clone(), weights=torch.zeros_like(w))["weights"]
    fresh = dllm.kv4_attend(bf16(q, dev), pages, table, lens, weights=torch.zeros_like(w))["weights"]
    before = w.clone()
    dllm.kv4_attend(bf16(q, dev), pages, table, lens, prior=w, weights=w)
    for b, n in enumerate(cache.lens):
        for j in range(int(n)):
            at = (int(cache.table[b, j // 16]), slice(None), j % 16)
            assert torch.equal(w[at], apart[at])
            assert torch.equal(before[at] + fresh[at], apart[at])


@pytest.mark.parametrize("L,H,heads", [(1, 4, 2), (32, 14, 2)])
def test_attend_nan_stays_with_its_request(dllm, L, H, heads):
    """A NaN key, value or query makes its own rows NaN and no others'."""
    rng = np.random.default_rng(12)
    cache = Cache(rng, [100, 100, 100, 100], heads, 128, 16)
    cache.k[cache.table[0, 2], 0, 3, 40] = np.nan      # request 0, head 0
    cache.v[cache.table[1, 1], 1, 5, 77] = np.inf      # request 1, head 1: one group of channels
    cache.pages = ref.pages_of(cache.k, cache.v, 16)
    q = rng.standard_normal((4, L, H, 128))
    q[2, L - 1, 1, 9] = np.nan
    got, _ = run_attend(dllm, cache, q)
    G = H // heads
    nan = np.isnan(got["out"])
    assert nan[0, :, :G].all() and not nan[0, :, G:].any()
    assert nan[1, :, G:, 64:96].all() and not nan[1, :, :G].any() and not nan[1, :, G:, :64].any()
    assert nan[2, L - 1, 1].all() and not nan[2, : L - 1].any() and not nan[2, L - 1, 2:].any()
    assert not nan[3].any()


@pytest.mark.parametrize("L,H", [(1, 8), (32, 14)])
def test_attend_shared_prefix_equal_bits_and_streams(dllm, L, H):
    """Two requests over the same pages are both right; equal calls give equal
    bits, on another stream too."""
    import torch
    rng = np.random.default_rng(13)
    cache = Cache(rng, [3000, 3000], 2, 128, 64)
    cache.table[1] = cache.table[0]
    q = rng.standard_normal((1, L, H, 128))
    dev = torch.device("cuda", 0)
    pages, table, lens = cache.upload(dev)
    tq = bf16(np.concatenate([q, q]), dev)
    a = dllm.kv4_attend(tq, pages, table, lens)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c = dllm.kv4_attend(tq, pages, table, lens)
    side.synchronize()
    b = dllm.kv4_attend(tq, pages, table, lens)
    for k in a:
        assert torch.equal(a[k], b[k]) and torch.equal(a[k], c[k])
    kv = ref.tokens_of(cache.pages, cache.table[0], 3000, 64, 128)
    _, lse, _, size, _ = ref.attend(ref.from_bf16(ref.to_bf16(q))[0], *kv, 128 ** -0.5)
    for i in range(2):
        assert (np.abs(a["lse"][i].cpu().numpy() - lse) <= score_tol(size, lse)).all()


@pytest.mark.parametrize("L,H", [(1, 4), (32, 14)])
def test_attend_errors_the_device_sees(dllm, L, H):
    """A page number outside the pool and a length beyond the table are
    recorded; the other requests' results stand."""
    import torch
    rng = np.random.default_rng(14)
    cache = Cache(rng, [100, 100, 50], 2, 128, 16, extra=0)
    q = rng.standard_normal((3, L, H, 128))
    good, _ = run_attend(dllm, cache, q)
    dev = torch.device("cuda", 0)
    for kind in ("page", "negative", "length"):
        pages, table, lens = cache.upload(dev)
        if kind == "length":
            lens[0] = 7 * 16 + 1
        else:
            table[0, 3] = pages.shape[0] if kind == "page" else -1
        w = torch.zeros(pages.shape[0], 2, 16, device=dev)
        out = dllm.kv4_attend(bf16(q, dev), pages, table, lens, weights=w)
        assert dllm.get_device_error(dev) == 5
        assert dllm.get_device_error(dev) == 0
        np.testing.assert_array_equal(out["out"].float().cpu().numpy()[1:], good["out"][1:])


# ---------------------------------------------------------------------------
# the write
# ---------------------------------------------------------------------------
def write_case(rng, B, W, heads, D, kind):
    x = rng.standard_normal((B, W, 2, heads, D)).astype(np.float32)
    if kind == "zeros":
        x[:, ::2] = 0.0
    elif kind == "one_sided":
        x = np.abs(x) + 3
        x[:, 1::2] *= -1
    elif kind == "sizes":
        x *= np.exp2(rng.integers(-40, 12, (B, W, 2, heads, D // 32, 1))).repeat(32, -1).reshape(x.shape).astype(np.float32)
    elif kind == "grid":   # quotients that fall on halves
        x = np.round(x * 4) / 4
        x[..., 0::32], x[..., 1::32] = -3.75, 3.75
    elif kind == "nan":
        x[rng.random(x.shape) < 0.002] = np.nan
        x[rng.random(x.shape) < 0.002] = np.inf
        x[rng.random(x.shape) < 0.002] = -np.inf
    return ref.from_bf16(np.where(np.isfinite(x), ref.to_bf16(np.nan_to_num(x, posinf=0, neginf=0)),
                                  (np.ascontiguousarray(x).view(np.uint32) >> 16).astype(np.uint16)))


@pytest.mark.parametrize("kind", ["plain", "zeros", "one_sided", "sizes", "grid", "nan"])
@pytest.mark.parametrize("B,W,heads,D,page", [(1, 1, 1, 64, 16), (3, 32, 4, 128, 32), (2, 77, 3, 64, 16),
                                              (5, 50, 2, 128, 256)])
def test_write(dllm, kind, B, W, heads, D, page):
    import torch
    dev = torch.device("cuda", 0)
    rng = np.random.default_rng(B * 100 + W)
    x = write_case(rng, B, W, heads, D, kind)
    first = rng.integers(0, W, B).astype(np.int32)
    count = np.array([rng.integers(0, W - f + 1) for f in first], dtype=np.int32)
    first[0], count[0] = 0, W
    pos = rng.integers(0, 70, B).astype(np.int32)
    most = -(-(70 + W) // page)
    table = rng.permutation(B * most + 1)[: B * most].reshape(B, most).astype(np.int32)
    before = rng.integers(0, 256, (B * most + 1, heads, page * (D + D // 8)), dtype=np.uint8)
    fused = bf16(np.where(np.isfinite(x), x, 0), dev)
    raw = torch.from_numpy(np.ascontiguousarray(x).view(np.uint32).__rshift__(16).astype(np.uint16).view(np.int16))
    fused.view(torch.int16).copy_(raw.to(dev))   # NaN and infinite patterns as they are
    pages = torch.from_numpy(before.copy()).to(dev)
    outs = [torch.full((B, W, heads, D), 5.0, dtype=torch.bfloat16, device=dev) for _ in range(2)]
    t = lambda a: torch.from_numpy(a).to(dev)  # noqa: E731
    dllm.kv4_write(fused[:, :, 0], fused[:, :, 1], pages, t(table), t(pos), first=t(first), count=t(count),
                   k_out=outs[0], v_out=outs[1])
    assert dllm.get_device_error(dev) == 0
    # expected: the definition, one token at a time
    made = ref.pages_of(*(x[:, :, i].reshape(B * W, heads, 1, D) for i in range(2)), 1)
    vals = ref.values_of(made, 1, D)
    want = before.copy()
    wo = [np.full((B, W, heads, D), 5.0) for _ in range(2)]
    cuts = [(0, D // 2), (D // 2, D // 16), (D // 2 + D // 16, D // 2), (D + D // 16, D // 16)]
    for b in range(B):
        for c in range(first[b], first[b] + count[b]):
            j = pos[b] + c - first[b]
            for at, size in cuts:
                o = page * at + (j % page) * size
                want[table[b, j // page], :, o:o + size] = made[b * W + c, :, at:at + size]
            for i in range(2):
                wo[i][b, c] = vals[i][b * W + c, :, 0]
    np.testing.assert_array_equal(pages.cpu().numpy(), want)
    for i in range(2):
        np.testing.assert_array_equal(outs[i].float().cpu().numpy(), wo[i])
    # the step bounds the error: half a step, one at the range's ends
    g = x[:, :, 0].reshape(B, W, heads, -1, 32).astype(np.float64)
    ok = np.isfinite(g).all(-1)
    _, step, _ = ref.quantise(x[:, :, 0])
    err = np.abs(vals[0].reshape(g.shape) - g)
    inside = ok & (np.abs(g).max(-1, initial=0) < 11000)
    assert (err[inside] <= step[inside][..., None]).all()


def test_write_defaults_saturation_and_errors(dllm):
    import torch
    dev = torch.device("cuda", 0)
    pages, _ = dllm.kv4_pages(6, 2, 16, 128, dev)
    table = torch.tensor([[4, 1], [0, 3]], dtype=torch.int32, device=dev)
    k = torch.randn(2, 20, 2, 128, device=dev).to(torch.bfloat16)
    k[0, 0, 0, 0] = 1e38
    k[0, 0, 0, 1] = -1e38
    pos = torch.tensor([3, 12], dtype=torch.int32, device=dev)
    ko = torch.empty_like(k)
    dllm.kv4_write(k, k, pages, table, pos, k_out=ko)                 # all columns from 0
    assert dllm.get_device_error(dev) == 0
    vals = ref.values_of(pages.cpu().numpy(), 16, 128)
    # saturates on both sides: the zero point is rint(7.5 up to 4 bits of step) of the whole range
    assert vals[0][4, 0, 3, 1] < -768 * 6 and vals[0][4, 0, 3, 0] > 768 * 6
    np.testing.assert_array_equal(vals[1][3, :, 15], ko[1, 19].float().cpu().numpy())
    was = pages.clone()
    for p, f, c in ((13, 0, 20), (-1, 0, 4), (0, 1, 20), (0, -1, 3)):           # past the table, before it, past W, before 0
        one = lambda v: torch.tensor([v, 0], dtype=torch.int32, device=dev)  # noqa: E731
        dllm.kv4_write(k, k, pages, table, one(p), first=one(f), count=one(c))
        assert dllm.get_device_error(dev) == 5
        assert torch.equal(pages, was), (p, f, c)
    table[0, 1] = 6
    dllm.kv4_write(k, k, pages, table, pos)
    assert dllm.get_device_error(dev) == 5


# ---------------------------------------------------------------------------
# eviction
# ---------------------------------------------------------------------------
EVICTIONS = {
    "one": ([1], [1], 0), "none_kept": ([40, 7], [0, -3], 5), "all_kept": ([40, 7, 0], [40, 99, 3], 2),
    "half": ([100, 33, 1024, 1025], [50, 16, 512, 513], 8), "recent_only": ([300, 20], [10, 30], 64),
    "no_recent": ([2500, 1023], [700, 1022], 0), "long": ([9000], [3001], 33),
}


@pytest.mark.parametrize("kind", ["random", "ties", "equal", "zeros", "signed", "special"])
@pytest.mark.parametrize("name", EVICTIONS)
def test_evict(dllm, name, kind):
    import torch
    dev = torch.device("cuda", 0)
    lens, keep, recent = EVICTIONS[name]
    rng = np.random.default_rng(len(name) * 7 + len(kind))
    heads, D, page = (3, 64, 16) if len(lens) > 2 else (2, 128, 32)
    B = len(lens)
    cap = max(1, -(-max(min(k, n) for k, n in zip(keep, lens)) // page))
    cache = Cache(rng, lens, heads, D, page, extra=1, spare=B * cap)
    free = np.setdiff1d(np.arange(len(cache.pages)), cache.table)
    dst = rng.permutation(free)[: B * cap].reshape(B, cap).astype(np.int32)
    shape = (len(cache.pages), heads, page)
    w = rng.random(shape).astype(np.float32)
    if kind == "ties":
        w = np.round(w * 4) / 4
    elif kind == "equal":
        w[:] = 0.25
    elif kind == "zeros":
        w[rng.random(shape) < 0.9] = 0
    elif kind == "signed":
        w = w - 0.5
    elif kind == "special":
        w[rng.random(shape) < 0.2] = np.nan
        w[rng.random(shape) < 0.2] = np.inf
        w[rng.random(shape) < 0.2] = -np.inf
        w[rng.random(shape) < 0.2] = -0.0
    w = w.astype(np.float32)
    pages, table, tl = cache.upload(dev)
    tw, td = torch.from_numpy(w.copy()).to(dev), torch.from_numpy(dst).to(dev)
    out = dllm.kv4_evict(pages, tw, table, tl, torch.tensor(keep, dtype=torch.int32, device=dev), td, recent=recent)
    assert dllm.get_device_error(dev) == 0
    src, new = out["src"].cpu().numpy(), out["lens"].cpu().numpy()
    got_p, got_w = pages.cpu().numpy(), tw.cpu().numpy()
    want_p, want_w = cache.pages.copy(), w.copy()
    cuts = [(0, D // 2), (D // 2, D // 16), (D // 2 + D // 16, D // 2), (D + D // 16, D // 16)]
    for b, n in enumerate(lens):
        assert new[b] == min(max(keep[b], 0), n)
        for h in range(heads):
            mine = np.array([w[cache.table[b, j // page], h, j % page] for j in range(n)], dtype=np.float32)
            stay = ref.evict(mine, keep[b], recent)
            np.testing.assert_array_equal(src[b, h, : len(stay)], stay)
            assert (src[b, h, len(stay):] == -1).all()
            for i, j in enumerate(stay):
                p, q = cache.table[b, j // page], dst[b, i // page]
                for at, size in cuts:
                    f, t = page * at + (j % page) * size, page * at + (i % page) * size
                    want_p[q, h, t:t + size] = cache.pages[p, h, f:f + size]
                want_w[q, h, i % page] = w[p, h, j % page]
    np.testing.assert_array_equal(got_p, want_p)
    np.testing.assert_array_equal(got_w.view(np.uint32), want_w.view(np.uint32))


def test_evict_errors_the_device_sees(dllm):
    import torch
    dev = torch.device("cuda", 0)
    rng = np.random.default_rng(20)
    cache = Cache(rng, [60, 60], 2, 64, 16, extra=0, spare=8)
    free = np.setdiff1d(np.arange(len(cache.pages)), cache.table)
    for kind in ("length", "source", "target", "room"):
        pages, table, lens = cache.upload(dev)
        dst = torch.from_numpy(free[:4].reshape(2, 2).astype(np.int32)).to(dev)
        keep = torch.tensor([20, 20], dtype=torch.int32, device=dev)
        if kind == "length":
            lens[0] = 65
        elif kind == "source":
            table[0, 1] = len(cache.pages)
        elif kind == "target":
            dst[0, 1] = -5
        else:
            keep[0] = 33
        w = torch.rand(pages.shape[0], 2, 16, device=dev)
        out = dllm.kv4_evict(pages, w, table, lens, keep, dst)
        assert dllm.get_device_error(dev) == 5
        assert out["lens"].cpu().tolist() == [32 if kind == "room" else 20, 20]
        stay = ref.evict(np.array([w[int(table[1, j // 16]), 0, j % 16].item() for j in range(60)]), 20, 0)
        np.testing.assert_array_equal(out["src"][1, 0, :20].cpu().numpy(), stay)


# ---------------------------------------------------------------------------
# together, and at the far end of a pool
# ---------------------------------------------------------------------------
def test_pool_beyond_32_bits(dllm):
    """A pool of 4.5 GB: the pages used sit past 2^32 bytes."""
    import torch
    dev = torch.device("cuda", 0)
    heads, page, D = 4, 64, 128
    n = (9 << 29) // (heads * page * (D + D // 8))
    pages = torch.zeros((n, heads, page * (D + D // 8)), dtype=torch.uint8, device=dev)
    weights = torch.zeros((n, heads, page), dtype=torch.float32, device=dev)
    B, W = 2, 150
    rng = np.random.default_rng(21)
    x = ref.from_bf16(ref.to_bf16(rng.standard_normal((B, W, 2, heads, D))))
    table = torch.tensor([[n - 1, n - 5, n - 3], [n - 2, n - 4, n - 6]], dtype=torch.int32, device=dev)
    dst = torch.tensor([[n - 7], [n - 8]], dtype=torch.int32, device=dev)
    fused = bf16(x, dev)
    lens = torch.tensor([W, W], dtype=torch.int32, device=dev)
    dllm.kv4_write(fused[:, :, 0], fused[:, :, 1], pages, table, torch.zeros(B, dtype=torch.int32, device=dev))
    for L, H in ((1, 4), (32, 28)):
        q = ref.from_bf16(ref.to_bf16(rng.standard_normal((B, L, H, D))))
        out = dllm.kv4_attend(bf16(q, dev), pages, table, lens, weights=weights)
        for b in range(B):
            k, v = (ref.dequantise(*ref.quantise(x[b, :, i])).transpose(1, 0, 2) for i in range(2))
            o, lse, w, size, spread = ref.attend(q[b], k, v, D ** -0.5)
            assert (np.abs(out["lse"][b].cpu().numpy() - lse) <= score_tol(size, lse)).all()
            assert np.abs(out["out"][b].float().cpu().numpy() - o).max() <= 0.02
    ev = dllm.kv4_evict(pages, weights, table, lens, torch.tensor([60, 64], dtype=torch.int32, device=dev), dst, recent=4)
    assert dllm.get_device_error(dev) == 0
    src = ev["src"].cpu().numpy()
    kept = ref.values_of(pages[n - 8].cpu().numpy(), page, D)
    for h in range(heads):
        want = ref.dequantise(*ref.quantise(x[1, :, 1, h]))[src[1, h, :64]]
        np.testing.assert_array_equal(kept[1][h], want)


def test_refusals(dllm):
    import torch
    dev = torch.device("cuda", 0)
    pages, weights = dllm.kv4_pages(4, 2, 16, 128, dev)
    table = torch.zeros(1, 2, dtype=torch.int32, device=dev)
    lens = torch.ones(1, dtype=torch.int32, device=dev)
    q = torch.zeros(1, 2, 4, 128, dtype=torch.bfloat16, device=dev)
    k = torch.zeros(1, 2, 2, 128, dtype=torch.bfloat16, device=dev)
    dllm.kv4_attend(q, pages, table, lens)
    with pytest.raises(TypeError):
        dllm.kv4_attend(q.half(), pages, table, lens)
    with pytest.raises(TypeError):
        dllm.kv4_attend(q, pages, table, lens.long())
    with pytest.raises(TypeError):
        dllm.kv4_attend(q, pages, table, lens, weights=weights[:3].contiguous())
    with pytest.raises(ValueError):
        dllm.kv4_attend(q, pages, torch.zeros(2, 2, dtype=torch.int32, device=dev), lens)
    with pytest.raises(ValueError):
        dllm.kv4_attend(q[..., :64], pages[:, :, :1000].contiguous(), table, lens)
    with pytest.raises(ValueError):
        dllm.kv4_attend(q, pages.cpu(), table, lens)
    for bad in (q[:, :, :3], torch.zeros(1, 1025, 2, 128, dtype=torch.bfloat16, device=dev)):
        with pytest.raises(dllm.DllmError):
            dllm.kv4_attend(bad, pages, table, lens)
    with pytest.raises(dllm.DllmError):
        dllm.kv4_attend(q, pages, table, lens, scale=float("nan"))
    with pytest.raises(dllm.DllmError):     # prior without weights
        dllm.kv4_attend(q, pages, table, lens, prior=weights)
    with pytest.raises(dllm.DllmError):     # a workspace too small
        dllm.kv4_attend(q, pages, table, lens, workspace=torch.zeros(256, dtype=torch.uint8, device=dev))
    with pytest.raises(dllm.DllmError):     # off a 16-byte boundary
        dllm.kv4_attend(torch.zeros(1, 2, 4, 136, dtype=torch.bfloat16, device=dev)[..., 4:132], pages, table, lens)
    with pytest.raises(TypeError):
        dllm.kv4_write(k.float(), k.float(), pages, table, lens)
    with pytest.raises(ValueError):
        dllm.kv4_write(k[:, :, :1], k[:, :, :1], pages, table, lens)
    with pytest.raises(TypeError):
        dllm.kv4_write(k, k, pages, table, lens.long())
    with pytest.raises(TypeError):
        dllm.kv4_write(k, k, pages, table, lens, k_out=k[:, :1].contiguous())
    with pytest.raises(TypeError):
        dllm.kv4_evict(pages, weights[:2].contiguous(), table, lens, lens, table)
    with pytest.raises(dllm.DllmError):
        dllm.kv4_evict(pages, weights, table, lens, lens, table, recent=-1)
    with pytest.raises(ValueError):
        dllm.kv4_pages(4, 2, 24, 128, dev)
    # nothing to do is not an error
    none = torch.zeros(0, 2, dtype=torch.int32, device=dev)
    empty = torch.zeros(0, dtype=torch.int32, device=dev)
    assert dllm.kv4_attend(q[:0], pages, none, empty)["out"].shape[0] == 0
    dllm.kv4_write(k[:0], k[:0], pages, none, empty)
    assert dllm.kv4_evict(pages, weights, none, empty, empty, none)["lens"].numel() == 0
    assert dllm.get_device_error(dev) == 0


@pytest.mark.parametrize("L,H,heads", [(32, 2, 2), (32, 7, 1), (40, 8, 1), (1, 4, 1)])
def test_attend_many_short_requests(dllm, L, H, heads):
    """Hundreds of requests of one or two tiles, empty ones among them: every
    CTA runs through several, its warps items apart."""
    rng = np.random.default_rng(30)
    lens = rng.choice([0, 1, 100, 128, 129, 250, 257], 700)
    lens[:200] = rng.choice([0, 128], 200)
    cache = Cache(rng, lens, heads, 64, 64, extra=0)
    check_attend(dllm, cache, rng.standard_normal((700, L, H, 64)), weights=True)


def test_attend_one_long_among_short(dllm):
    """One request far longer than the others is cut over the CTAs."""
    rng = np.random.default_rng(31)
    lens = [64] * 40 + [20000] + [300] * 3
    cache = Cache(rng, lens, 1, 64, 256, extra=0)
    check_attend(dllm, cache, rng.standard_normal((44, 33, 4, 64)), weights=True)
    check_attend(dllm, cache, rng.standard_normal((44, 33, 1, 64)), weights=True)
    check_attend(dllm, cache, rng.standard_normal((44, 1, 4, 64)), weights=True)
