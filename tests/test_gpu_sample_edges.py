"""dllm_sample at the ends of its ranges: u of 1 and more, weights that hardly count, large vocabularies."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def dev():
    import torch
    return torch.device("cuda", 0)


def draw(dllm, x, u, V=None, **kw):
    import torch
    if x.shape[1] % 8:
        V, x = x.shape[1], torch.nn.functional.pad(x, (0, -x.shape[1] % 8), value=float("nan"))
    t = {k: torch.tensor(v, device=dev()) for k, v in kw.items()}
    out = dllm.sample(x, torch.tensor(u, dtype=torch.float32, device=dev()), V=V, **t)
    assert dllm.get_device_error(dev()) == 0
    return out["tokens"].tolist(), out["prob"].double().tolist()


@pytest.mark.parametrize("V", [8, 5003, 126464])
@pytest.mark.parametrize("low", [-33.0, -36.0, -42.0])
def test_u_of_one_takes_the_last_kept_token(dllm, V, low):
    """One token of weight 1, two of 2^-46 to 2^-61, the rest below 2^-62 (exp(-42.98)): the last of the kept ones is drawn
    with u >= 1, whatever its weight does to sums; filters move the end forward."""
    import torch
    x = torch.full((1, V), low - 10.0, device=dev())
    x[0, V // 2], x[0, 1], x[0, V - 2] = 0.0, low, low + 1.0
    x = x.to(torch.bfloat16)
    one = lambda v, t: np.array([v], dtype=t)  # noqa: E731
    for u in (1.0, 7.0, float("inf")):
        assert draw(dllm, x, [u])[0] == [1]
        assert draw(dllm, x, [u], top_k=one(2, np.int32))[0] == [V - 2]
        assert draw(dllm, x, [u], top_k=one(3, np.int32))[0] == [1]
        assert draw(dllm, x, [u], top_k=one(10 ** 9, np.int32))[0] == [1]
        assert draw(dllm, x, [u], min_p=one(2.0 ** -61, np.float32))[0] == [1]
        assert draw(dllm, x, [u], min_p=one(2.0 ** -10, np.float32))[0] == [V // 2]
        assert draw(dllm, x, [u], top_p=one(0.9, np.float32))[0] == [V // 2]
        assert draw(dllm, x, [u], top_p=one(0.9, np.float32), top_k=one(2, np.int32))[0] == [V // 2]
        assert draw(dllm, x, [u], temperature=one(0.0, np.float32))[0] == [V // 2]
    assert draw(dllm, x, [0.999])[0] == [V // 2]


def test_u_of_one_with_ties_and_wide_values(dllm):
    """The last of equal tokens; rows whose values only the wide path tells apart.  A weight is held to 2^-62 of the
    largest, and so is its probability where the largest token is the mass."""
    import torch
    x = torch.full((3, 9000), -40.0, device=dev())
    x[0, [5, 77, 8001]] = 0.0
    x[1, 4000], x[1, [3, 8999]] = 300.0, 262.0            # wide
    x[1, 17] = 264.0
    x[2, ::2] = float("-inf")
    x[2, 11] = 0.0
    x = x.to(torch.bfloat16)
    tokens, prob = draw(dllm, x, [1.0, 1.0, 2.0])
    assert tokens == [8999, 8999, 8999]
    np.testing.assert_allclose(prob, [np.exp(-40) / 3, np.exp(-38), np.exp(-40)], rtol=1e-7, atol=2.0 ** -62)


def test_large_vocabulary(dllm):
    """2^24 and some tokens, peaked and flat.  The unit of a mass is 2^-37 of the largest weight there; each of the row's
    different values may be off by half of one: a draw is compared where u is further than that from a border."""
    import torch
    import sample_reference
    V = 2 ** 24 + 5
    gen = torch.Generator(device=dev())
    gen.manual_seed(7)
    x = torch.randn(2, V + 3, generator=gen, device=dev()) * 1.5
    x[0, 12345678] = 18.0                                  # half of the row's mass
    x = x.to(torch.bfloat16)
    host = x[:, :V].float().cpu().numpy().astype(np.float64)
    for u, kw in (([0.25, 0.61803], {}),
                  ([0.95, 0.3], {"top_k": np.full(2, 3000000, dtype=np.int32), "top_p": np.full(2, 0.95, dtype=np.float32)})):
        tokens, prob = draw(dllm, x, u, V=V, **kw)
        for i in range(2):
            want, p, margin = sample_reference.sample(host[i], float(np.float32(u[i])),
                                                      top_k=int(kw["top_k"][i]) if kw else 0,
                                                      top_p=float(kw["top_p"][i]) if kw else 1.0)
            top = 1.0 / np.exp(host[i] - host[i].max()).sum()           # the largest weight's share
            if margin > len(np.unique(host[i])) * 2.0 ** -38 * top + V * 2.0 ** -53:   # and the reference's own sums
                assert tokens[i] == want
                np.testing.assert_allclose(prob[i], p, rtol=1e-6)
            else:
                assert abs(host[i][tokens[i]] - host[i][want]) < 0.1


@pytest.mark.parametrize("kind", ["plain", "flat", "peaked", "masked", "zeros", "tiny", "huge", "edges", "lowest", "signed_zero"])
@pytest.mark.parametrize("n,V", [(1, 126464), (3, 30011), (160, 5000), (700, 999), (2, 1)])
def test_confidence(dllm, kind, n, V):
    """conf against the softmax in 64 bits, whatever the draw's settings: a quotient of masses good to 1e-11 rounded once
    to 32 bits (2^-24), weights held to 2^-62 of the largest.  Everything else is as without it."""
    import torch
    from test_gpu_sample import rows, settings
    rng = np.random.default_rng(n)
    x = rows(rng, n, V, kind)
    if n > 2:
        x[1] = -np.inf
    u = rng.random(n)
    logits = torch.full((n, -(-V // 8) * 8), float("nan"))
    logits[:, :V] = torch.from_numpy(x.astype(np.float32))
    logits = logits.to(torch.bfloat16).to(dev())
    given = {k: torch.from_numpy(v).to(dev()) for k, v in settings(rng, n).items()}
    given["temperature"][0] = -1.0 if n > 1 else 1.0
    at = torch.from_numpy(np.where(rng.random(n) < 0.1, -1, np.arange(n)).astype(np.int32)).to(dev())
    t = torch.from_numpy(u.astype(np.float32)).to(dev())
    plain = dllm.sample(logits, t, V=V, rows=at, **given)
    out = dllm.sample(logits, t, V=V, rows=at, conf=True, **given)
    assert dllm.get_device_error(dev()) == 0
    assert torch.equal(plain["tokens"], out["tokens"]) and torch.equal(plain["prob"].nan_to_num(-1), out["prob"].nan_to_num(-1))
    tokens, conf = out["tokens"].cpu().numpy(), out["conf"].double().cpu().numpy()
    for i in range(n):
        if tokens[i] < 0:
            assert np.isnan(conf[i])
            continue
        w = np.exp(x[i].astype(np.float64) - x[i].max())
        np.testing.assert_allclose(conf[i], w[tokens[i]] / w.sum(), rtol=1e-7, atol=2.0 ** -62)
