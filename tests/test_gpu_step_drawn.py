"""step_sampled: the step over given tokens and confidences, where tokens are missing, confidences lie on a threshold,
and calls run side by side."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def dev():
    import torch
    return torch.device("cuda", 0)


def test_calls_at_once(dllm):
    """Batches of several shapes on streams of their own, beside plain steps and replayed graphs, one of which was captured
    before any other call of its size: everyone gets its own results."""
    import torch
    rng = np.random.default_rng(2)
    d = dev()
    work = []
    for B, L, V in ((300, 32, 500), (7, 700, 2000), (64, 100, 1000), (1, 1, 9)):
        ids = torch.from_numpy(np.where(rng.random((B, L)) < 0.7, V, 3).astype(np.int32)).to(d)
        tok = torch.from_numpy(rng.integers(0, V, B * L).astype(np.int32)).to(d)
        conf = torch.from_numpy(rng.random(B * L).astype(np.float32) * 0.9 + 0.1).to(d)
        thr = torch.from_numpy(rng.random(B).astype(np.float32)).to(d)
        work.append((ids, tok, conf, thr, V))

    def turn(w):
        ids, tok, conf, thr, V = w
        thr = thr[:len(ids)]
        mine, cs = ids.clone(), torch.full(ids.shape, float("nan"), device=d)
        out = dllm.step_sampled(tok, conf, mine, thr, cs, V=V, mask_id=V, debug=True)
        return [mine, cs, *(out[k] for k in sorted(out))]

    turn([t[:1] if k < 1 else t[:32] if k < 3 else t for k, t in enumerate(work[0])])   # loads the kernels: not while capturing
    graphs, replayed = [], []
    for w in work:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            replayed.append(turn(w))
        graphs.append(g)
    want = [turn(w) for w in work]
    B, L, V = 64, 32, 4000
    logits = torch.from_numpy(rng.standard_normal((B * L, V)) * 3).to(torch.bfloat16).to(d)
    blocks = torch.full((B, L), V, dtype=torch.int32, device=d)
    thr = torch.full((B,), 0.3, device=d)

    def plain():
        ids, cs = blocks.clone(), torch.full((B, L), float("nan"), device=d)
        return ids, cs, dllm.step(logits, ids, thr, cs, V=V, mask_id=V)["n_new"]
    plain_want = plain()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(8)]
    got, steps = [], []
    for _ in range(10):
        for k, w in enumerate(work):
            with torch.cuda.stream(streams[k]):
                got.append((k, turn(w)))
            with torch.cuda.stream(streams[4 + k]):
                graphs[k].replay()
        steps.append(plain())
    torch.cuda.synchronize()
    same = lambda a, b: all(x.equal(y) or torch.equal(x.nan_to_num(-5), y.nan_to_num(-5)) for x, y in zip(a, b))  # noqa: E731
    for k, o in got + list(enumerate(replayed)):
        assert same(o, want[k])
    assert all(same(o, plain_want) for o in steps)
    assert dllm.get_device_error(d) == 0


def test_a_caller_s_workspace(dllm):
    import torch
    d = dev()
    ids = torch.full((3, 8), 50, dtype=torch.int32, device=d)
    tok, conf = torch.arange(24, dtype=torch.int32, device=d), torch.linspace(0.1, 0.9, 24, device=d)
    thr, cs = torch.full((3,), 0.5, device=d), torch.zeros(3, 8, device=d)
    ws = torch.zeros(dllm.step_workspace_size(3, 8, 50), dtype=torch.uint8, device=d)
    out = dllm.step_sampled(tok, conf, ids, thr, cs, V=50, mask_id=50, workspace=ws)
    assert out["n_new"].tolist() == [1, 4, 8] and out["done"].tolist() == [0, 0, 1]
    for bad in (ws[:100], ws[1:]):
        with pytest.raises(dllm.DllmError):
            dllm.step_sampled(tok, conf, ids, thr, cs, V=50, mask_id=50, workspace=bad)
    with pytest.raises(ValueError):
        dllm.step_sampled(tok, conf, ids, thr, cs, V=50, mask_id=50, workspace=ws.cpu())
    assert dllm.get_device_error(d) == 0


def expected(ids, tok, conf, thr, quota, mask):
    """(ids, n_new, done) by the rules of include/dllm.h, over the masked positions that have a token."""
    ids = ids.copy()
    n_new, done = [], []
    for b in range(len(ids)):
        at = np.flatnonzero((ids[b] == mask) & (tok[b] >= 0))
        order = at[np.argsort(-conf[b, at], kind="stable")]
        if quota is not None:
            take = order[:max(int(quota[b]), 0)]
        else:
            over = at[conf[b, at] > thr[b]]
            take = over if len(over) else order[:1]
        ids[b, take] = tok[b, take]
        n_new.append(len(take))
        done.append(int(not (ids[b] == mask).any()))
    return ids, n_new, done


def run(dllm, ids, tok, conf, thr, quota, mask, V, **kw):
    import torch
    t = lambda x: None if x is None else torch.from_numpy(np.ascontiguousarray(x)).to(dev())  # noqa: E731
    g_ids, cs = t(ids), torch.full(ids.shape, float("nan"), device=dev())
    out = dllm.step_sampled(t(tok.ravel()), t(conf.ravel()), g_ids, t(thr), cs, V=V, mask_id=mask, quota=t(quota),
                            debug=True, **kw)
    assert dllm.get_device_error(dev()) == 0
    return g_ids.cpu().numpy(), cs.cpu().numpy(), {k: v.cpu().numpy() for k, v in out.items()}


@pytest.mark.parametrize("L", [1, 5, 32, 33, 100, 700])
@pytest.mark.parametrize("rule", ["threshold", "negative threshold", "quota", "quota beyond"])
def test_positions_without_a_token_stay_masked(dllm, rule, L):
    """Some, then all, of a block's masked positions have no token: they are not unmasked by any rule, count for nothing,
    and the block is not done."""
    rng = np.random.default_rng(L)
    B, V = 9, 50
    mask = V
    ids = np.where(rng.random((B, L)) < 0.7, mask, 3).astype(np.int32)
    ids[0], ids[1], ids[2] = mask, mask, 3
    tok = rng.integers(0, V, (B, L)).astype(np.int32)
    conf = rng.random((B, L)).astype(np.float32)
    none = rng.random((B, L)) < 0.4
    none[0] = True                                       # a block without a token at all
    none[1] = np.arange(L) > 0                           # a block with one
    none[3] = False
    tok[none] = np.where(rng.random(none.sum()) < 0.8, -1, -7)
    conf[none] = np.where(rng.random(none.sum()) < 0.5, np.nan, 0.9)
    conf[4] *= 0.1                                       # nothing passes: the surest one that has a token
    thr = np.full(B, -1.0 if rule.startswith("negative") else 0.5, dtype=np.float32)
    quota = None
    if rule.startswith("quota"):
        quota = np.full(B, L + 3 if "beyond" in rule else 2, dtype=np.int32)
    want, n_new, done = expected(ids, tok, conf, thr, quota, mask)
    got, cs, out = run(dllm, ids, tok, conf, None if quota is not None else thr, quota, mask, V)
    np.testing.assert_array_equal(got, want)
    assert (got >= 0).all() and got[0].tolist() == [mask] * L
    assert out["n_new"].tolist() == n_new and out["done"].tolist() == done
    assert out["accept_len"].tolist() == [L * d for d in done]
    fresh = (ids == mask) & (want != mask)
    np.testing.assert_array_equal(cs[fresh], conf[fresh])
    assert np.isnan(cs[~fresh]).all()
    np.testing.assert_array_equal(out["tok"], np.where(ids == mask, np.maximum(tok, -1), -1))
    import torch
    cs0 = np.where(ids == mask, np.float32("nan"), rng.random((B, L)).astype(np.float32))
    t = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(dev())  # noqa: E731
    g_ids, g_cs = t(ids), t(cs0)
    again = dllm.step_sampled(t(tok.ravel()), t(conf.ravel()), g_ids, None if quota is not None else t(thr), g_cs, V=V,
                              mask_id=mask, quota=None if quota is None else t(quota))
    np.testing.assert_array_equal(g_ids.cpu().numpy(), want)
    feats = dllm.features(g_ids, g_cs, mask_id=mask)
    np.testing.assert_array_equal(again["feats"].cpu().numpy(), feats.cpu().numpy())
    assert np.isfinite(again["feats"][1:].cpu().numpy()[(want[1:] != mask).any(1)]).all()


def test_confidences_are_taken_as_they_are(dllm):
    """Confidences next to their threshold, on either side and on it: compared and recorded bit for bit."""
    rng = np.random.default_rng(1)
    B, L, V = 200, 32, 50
    mask = V
    p = rng.random((B, L)).astype(np.float32)
    thr = rng.random(B).astype(np.float32)
    side = rng.integers(0, 3, (B, L))
    p = np.where(side == 0, thr[:, None], np.where(side == 1, np.nextafter(thr[:, None], np.float32(2)), p))
    p = np.where(p > thr[:, None], np.nextafter(thr[:, None], np.float32(2)), p).astype(np.float32)
    p[5], p[6, ::2], p[7] = 1e-42, 0.0, np.float32(2.0 ** -149)      # subnormal ones count too
    ids = np.full((B, L), mask, dtype=np.int32)
    tok = rng.integers(0, V, (B, L)).astype(np.int32)
    want, n_new, _ = expected(ids, tok, p, thr, None, mask)
    got, cs, out = run(dllm, ids, tok, p, thr, None, mask, V)
    np.testing.assert_array_equal(out["conf"], p)
    np.testing.assert_array_equal(got, want)
    assert out["n_new"].tolist() == n_new
    np.testing.assert_array_equal(cs[want != mask], p[want != mask])


@pytest.mark.parametrize("quota", [False, True])
@pytest.mark.parametrize("L,V", [(8, 500), (32, 30011), (5, 126464)])
def test_greedy_rows_decode_as_the_step_does(dllm, quota, L, V):
    """At temperature 0 (and top-k 1) the draw and its conf are the step's argmax and confidence: the same positions are
    unmasked, in a batch where other requests are sampled.  Requests where a confidence lies within 1e-5 of what decides (the
    step's own tolerance) are left out; few do."""
    import torch
    rng = np.random.default_rng(L)
    B, mask = 24, V
    ldv = -(-V // 8) * 8
    x = rng.standard_normal((B * L, ldv)) * 2
    x[np.arange(B * L), rng.integers(0, V, B * L)] += rng.random(B * L) * (8 + np.log(V))
    logits = torch.from_numpy(x).to(torch.bfloat16).to(dev())
    ids0 = np.where(rng.random((B, L)) < 0.7, mask, 3).astype(np.int32)
    ids0[0] = 3
    thr = torch.full((B,), 0.6, device=dev())
    left = torch.full((B,), 2, dtype=torch.int32, device=dev()) if quota else None
    ids, cs = torch.from_numpy(ids0).to(dev()), torch.full((B, L), float("nan"), device=dev())
    mine, mine_cs = ids.clone(), cs.clone()
    want = dllm.step(logits, ids, thr, cs, V=V, mask_id=mask, quota=left, debug=True)
    masked = torch.from_numpy(ids0.ravel() == mask).to(dev())
    rows = torch.where(masked, torch.arange(B * L, dtype=torch.int32, device=dev()), -1).to(torch.int32)
    T = torch.zeros(B * L, device=dev())
    k = torch.zeros(B * L, dtype=torch.int32, device=dev())
    T[B * L // 2:], k[B * L // 2:] = 0.9, 1                  # the other greedy requests, by top-k
    T[:L * 3], k[:L * 3] = 1.0, 0                            # three sampled ones
    d = dllm.sample(logits, torch.rand(B * L, device=dev()), V=V, rows=rows, temperature=T, top_k=k, conf=True)
    out = dllm.step_sampled(d["tokens"], d["conf"], mine, thr, mine_cs, V=V, mask_id=mask, quota=left, debug=True)
    assert dllm.get_device_error(dev()) == 0
    p, conf = want["conf"].cpu().numpy(), out["conf"].cpu().numpy()
    compared = 0
    for b in range(3, B):
        at = ids0[b] == mask
        np.testing.assert_array_equal(want["tok"][b].cpu().numpy()[at], out["tok"][b].cpu().numpy()[at])
        np.testing.assert_allclose(conf[b, at], p[b, at], rtol=0, atol=1e-5)
        order = np.sort(p[b, at])
        if not at.any() or np.abs(p[b, at] - 0.6).min() < 1e-5 or (len(order) > 1 and np.diff(order).min() < 1e-5):
            continue
        compared += 1
        assert torch.equal(mine[b], ids[b]) and int(out["n_new"][b]) == int(want["n_new"][b])
        assert int(out["done"][b]) == int(want["done"][b])
        fresh = (ids0[b] == mask) & (ids[b].cpu().numpy() != mask)
        np.testing.assert_allclose(mine_cs[b].cpu().numpy()[fresh], cs[b].cpu().numpy()[fresh], rtol=0, atol=1e-5)
    assert compared >= B // 2
