"""token_logprobs on the GPU against the definition in 64 bits.

Tolerance: the framework's 1e-5 max(1, |value|) for log sums.  The sums run
over at most ~V / 256 values per thread in 32 bits (rounding 2^-24 each, of
random sign) with exponentials good to 2^-22, so for the V here the error of
ln z stays under 1e-6; a log probability adds roundings of its own size."""
import numpy as np
import pytest

import kv4_reference as ref

pytestmark = pytest.mark.gpu

TOL = 1e-5


def rows(rng, n, V, dtype, kind):
    x = rng.standard_normal((n, V)).astype(np.float32) * 3
    if kind == "peaked":
        x[np.arange(n), rng.integers(0, V, n)] += 20
    elif kind == "ties":
        x = np.round(x)
    elif kind == "equal":
        x[:] = 1.5
    elif kind == "ascending":
        x = np.broadcast_to(np.linspace(-8, 8, V, dtype=np.float32), (n, V)).copy()
    elif kind == "masked":
        x[:, rng.random(V) < 0.7] = -np.inf
        x[:, rng.random(V) < 0.1] = -3.3895313892515355e38   # bf16's lowest
        x[:, V // 2] = 0.5
    elif kind == "lowest":
        x[:] = -3.3895313892515355e38
    elif kind == "signed_zero":
        x = np.where(rng.random((n, V)) < 0.5, -0.0, 0.0).astype(np.float32)
    return ref.from_bf16(ref.to_bf16(x)) if dtype == "bf16" else x


def upload(x, dtype, ldv, dev):
    import torch
    t = torch.full((x.shape[0], ldv), float("nan"), dtype=torch.float32)
    t[:, : x.shape[1]] = torch.from_numpy(x)
    return t.to(torch.bfloat16 if dtype == "bf16" else torch.float32).to(dev)


def check(dllm, x, tokens, top, dtype, ldv, row_of=None):
    import torch
    dev = torch.device("cuda", 0)
    logits = upload(x, dtype, ldv, dev)
    idx = np.arange(len(tokens)) if row_of is None else row_of
    out = dllm.token_logprobs(logits, torch.tensor(tokens, dtype=torch.int32, device=dev), V=x.shape[1], top=top,
                              rows=None if row_of is None else torch.tensor(row_of, dtype=torch.int32, device=dev))
    got = {k: v.cpu().numpy() for k, v in out.items()}
    for i, r in enumerate(idx):
        lp, ent, ids, tlp = ref.logprobs(x[r], tokens[i], top)
        np.testing.assert_allclose(got["logprob"][i], lp, rtol=TOL, atol=TOL)
        np.testing.assert_allclose(got["entropy"][i], ent, rtol=TOL, atol=TOL)
        if top:
            np.testing.assert_array_equal(got["top_ids"][i], ids)
            np.testing.assert_allclose(got["top_logprobs"][i], tlp, rtol=TOL, atol=TOL)
    return got


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,V,top", [(1, 1, 1), (1, 7, 32), (2, 8, 5), (3, 31, 20), (5, 1000, 5), (1, 8191, 20),
                                     (1, 8192, 32), (2, 8193, 1), (4, 40961, 32), (3, 126464, 0), (600, 513, 3),
                                     (2100, 33, 2)])
def test_sizes(dllm, dtype, n, V, top):
    rng = np.random.default_rng(V + n)
    x = rows(rng, n, V, dtype, "plain")
    check(dllm, x, rng.integers(0, V, n).tolist(), top, dtype, -(-V // 8) * 8 + 8)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["peaked", "ties", "equal", "ascending", "masked", "lowest", "signed_zero"])
@pytest.mark.parametrize("n,top", [(2, 20), (700, 32)])
def test_values(dllm, dtype, kind, n, top):
    """700 rows go a row to a CTA, 2 rows are cut: ties, adversarial orders and
    masks through both."""
    V = 30011
    rng = np.random.default_rng(5)
    x = rows(rng, n if n < 8 else 4, V, dtype, kind)
    idx = np.arange(n) % len(x)
    tokens = rng.integers(0, V, len(x))[idx]
    if n < 8:
        check(dllm, x, tokens.tolist(), top, dtype, 30016)
    else:
        import torch
        dev = torch.device("cuda", 0)
        out = dllm.token_logprobs(upload(x, dtype, 30016, dev), torch.tensor(tokens, dtype=torch.int32, device=dev), V=V,
                                  top=top, rows=torch.tensor(idx, dtype=torch.int32, device=dev))
        got = {k: v.cpu().numpy() for k, v in out.items()}
        for r in range(4):   # every entry of a row says the same, and it is right
            lp, ent, ids, tlp = ref.logprobs(x[r], tokens[r], top)
            mine = idx == r
            np.testing.assert_array_equal(got["top_ids"][mine], np.broadcast_to(ids, (mine.sum(), top)))
            for name, want in (("logprob", lp), ("entropy", ent), ("top_logprobs", tlp)):
                np.testing.assert_allclose(got[name][mine], np.broadcast_to(want, got[name][mine].shape), rtol=TOL,
                                           atol=TOL)


def test_rows_without_a_finite_maximum(dllm):
    V = 5000
    rng = np.random.default_rng(2)
    x = rows(rng, 5, V, "f32", "plain")
    x[0] = -np.inf
    x[1, 4999] = np.nan
    x[2, 17] = np.inf
    x[3, :] = -np.inf
    x[3, 4321] = 2.0   # one finite value: certain
    import torch
    dev = torch.device("cuda", 0)
    out = dllm.token_logprobs(upload(x, "f32", V, dev), torch.tensor([1, 1, 17, 4321, -1], dtype=torch.int32, device=dev),
                              V=V, top=3)
    got = {k: v.cpu().numpy() for k, v in out.items()}
    assert np.isnan(got["logprob"][[0, 1, 2, 4]]).all() and got["logprob"][3] == 0.0
    assert np.isnan(got["entropy"][:3]).all() and got["entropy"][3] == 0.0
    assert (got["top_ids"][:3] == -1).all() and np.isnan(got["top_logprobs"][:3]).all()
    np.testing.assert_array_equal(got["top_ids"][3], [4321, 0, 1])      # -inf tokens follow, lowest first
    assert got["top_logprobs"][3, 0] == 0.0 and np.isneginf(got["top_logprobs"][3, 1:]).all()
    np.testing.assert_allclose(got["entropy"][4], ref.logprobs(x[4], 0, 0)[1], rtol=TOL)   # nothing asked, still told


def test_rows_out_of_range_and_repeated(dllm):
    import torch
    dev = torch.device("cuda", 0)
    rng = np.random.default_rng(3)
    x = rows(rng, 3, 9000, "bf16", "plain")
    out = dllm.token_logprobs(upload(x, "bf16", 9000, dev), torch.tensor([5, 6, 5, 8999, 9000], dtype=torch.int32, device=dev),
                              V=9000, top=2, rows=torch.tensor([2, -1, 2, 3, 0], dtype=torch.int32, device=dev))
    got = {k: v.cpu().numpy() for k, v in out.items()}
    for i in (1, 3):
        assert np.isnan(got["logprob"][i]) and np.isnan(got["entropy"][i]) and (got["top_ids"][i] == -1).all()
    assert np.isnan(got["logprob"][4]) and np.isfinite(got["entropy"][4])
    for k in got:
        np.testing.assert_array_equal(got[k][0], got[k][2])


def test_equal_calls_give_equal_bits_and_leave_the_workspace_ready(dllm):
    import torch
    dev = torch.device("cuda", 0)
    rng = np.random.default_rng(4)
    V = 100003
    logits = upload(rows(rng, 3, V, "bf16", "plain"), "bf16", 100008, dev)
    tok = torch.tensor([3, 1, 2], dtype=torch.int32, device=dev)
    first = dllm.token_logprobs(logits, tok, V=V, top=20)
    few = dllm.token_logprobs(logits, tok[:1].contiguous(), V=V, top=32)     # another split, same workspace
    again = dllm.token_logprobs(logits, tok, V=V, top=20)
    for k in first:
        assert torch.equal(first[k], again[k]), k
    assert torch.equal(few["top_ids"][0, :20], first["top_ids"][0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        there = dllm.token_logprobs(logits, tok, V=V, top=20)
    side.synchronize()
    for k in first:
        assert torch.equal(first[k], there[k]), k


def test_no_entries(dllm):
    import torch
    dev = torch.device("cuda", 0)
    out = dllm.token_logprobs(torch.zeros(4, 16, dtype=torch.bfloat16, device=dev),
                              torch.zeros(0, dtype=torch.int32, device=dev), top=2)
    assert out["logprob"].numel() == 0 and out["top_ids"].shape == (0, 2)


def test_refusals(dllm):
    import torch
    dev = torch.device("cuda", 0)
    x = torch.zeros(4, 16, dtype=torch.bfloat16, device=dev)
    t = torch.zeros(4, dtype=torch.int32, device=dev)
    with pytest.raises(TypeError):
        dllm.token_logprobs(x.half(), t)
    with pytest.raises(TypeError):
        dllm.token_logprobs(x, t.long())
    with pytest.raises(ValueError):
        dllm.token_logprobs(x, torch.zeros(5, dtype=torch.int32, device=dev))
    with pytest.raises(ValueError):
        dllm.token_logprobs(x.cpu(), t)
    for kw in ({"V": 17}, {"V": 0}, {"top": 33}):
        with pytest.raises(dllm.DllmError):
            dllm.token_logprobs(x, t, **kw)
    with pytest.raises(dllm.DllmError):   # 12 values of 2 bytes: rows off 16-byte boundaries
        dllm.token_logprobs(x[:, :12].contiguous(), t)
