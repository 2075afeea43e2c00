"""dllm_sample on the GPU against its definition in 64 bits.

Tokens are compared for equality wherever the definition's u is further than
1e-10 of the kept mass from a border (the header promises 2^-40 = 9e-13; the
64-bit sums of 152 thousand terms are good to 2e-11), which hardly any entry is
not; where values tie, borders are hit exactly and both sides hold them exactly.
Probabilities: a quotient of masses good to 1e-11, rounded once to 32 bits, so
2^-24 relative and a little: 1e-7."""
import numpy as np
import pytest

import kv4_reference as ref
import sample_reference

pytestmark = pytest.mark.gpu

KINDS = ["plain", "flat", "peaked", "ties", "equal", "masked", "lowest", "zeros", "tiny", "huge", "ramp", "signed_zero",
         "edges"]


def rows(rng, n, V, kind):
    x = rng.standard_normal((n, V)) * 3
    if kind == "flat":
        x = rng.standard_normal((n, V)) * 0.3
    elif kind == "peaked":
        x[np.arange(n), rng.integers(0, V, n)] += 20
    elif kind == "ties":
        x = np.round(x)
    elif kind == "equal":
        x[:] = 1.5
    elif kind == "masked":
        x[:, rng.random(V) < 0.7] = -np.inf
        x[:, rng.random(V) < 0.1] = -3.3895313892515355e38
        x[:, V // 2] = 0.5
    elif kind == "lowest":
        x[:] = -3.3895313892515355e38
    elif kind == "zeros":
        x[:, ::2] = 0.0
    elif kind == "tiny":
        x *= 2.0 ** -30
    elif kind == "huge":
        x *= 200
    elif kind == "ramp":
        x = np.broadcast_to(np.linspace(-8, 8, V), (n, V)).copy()
    elif kind == "signed_zero":
        x = np.where(rng.random((n, V)) < 0.5, -0.0, 0.0)
    elif kind == "edges":   # values at the borders of what the counters hold
        x = rng.choice(np.array([256.0, -256.0, 255.0, -255.0, 2.0 ** -28, -2.0 ** -28, 2.0 ** -27, 1e-38, 9.2e-41]), (n, V))
    return ref.from_bf16(ref.to_bf16(x.astype(np.float32)))


def settings(rng, n):
    return {"temperature": rng.choice([0.0, 0.3, 0.7, 1.0, 1.5, 20.0], n).astype(np.float32),
            "top_k": rng.choice([0, 0, 1, 2, 50, 1000, 10 ** 9], n).astype(np.int32),
            "top_p": rng.choice([1.0, 1.0, 0.95, 0.5, 0.1, 0.0], n).astype(np.float32),
            "min_p": rng.choice([0.0, 0.0, 0.01, 0.2, 1.0], n).astype(np.float32)}


def check(dllm, x, u, given=None, row_of=None, ldv=None):
    import torch
    dev = torch.device("cuda", 0)
    V = x.shape[1]
    ldv = -(-V // 8) * 8 if ldv is None else ldv
    logits = torch.full((x.shape[0], ldv), float("nan"), dtype=torch.float32)
    logits[:, :V] = torch.from_numpy(np.asarray(x, dtype=np.float32))
    logits = logits.to(torch.bfloat16).to(dev)
    t = {k: torch.from_numpy(v).to(dev) for k, v in (given or {}).items()}
    out = dllm.sample(logits, torch.from_numpy(u.astype(np.float32)).to(dev), V=V,
                      rows=None if row_of is None else torch.tensor(row_of, dtype=torch.int32, device=dev), **t)
    assert dllm.get_device_error(dev) == 0
    tokens, prob = out["tokens"].cpu().numpy(), out["prob"].cpu().numpy()
    near = 0
    for i in range(len(u)):
        r = i if row_of is None else row_of[i]
        g = {k: float(v[i]) for k, v in (given or {}).items()}
        if not 0 <= r < x.shape[0]:
            assert tokens[i] == -1 and np.isnan(prob[i])
            continue
        want, p, margin = sample_reference.sample(x[r], float(np.float32(u[i])), T=g.get("temperature", 1.0),
                                                  top_k=int(g.get("top_k", 0)), top_p=g.get("top_p", 1.0),
                                                  min_p=g.get("min_p", 0.0))
        if margin < 1e-10 and x[r][tokens[i]] != x[r][want]:
            near += 1
            continue
        assert tokens[i] == want, (i, g, u[i], margin, x[r][want], x[r][tokens[i]])
        np.testing.assert_allclose(prob[i], p, rtol=1e-7)
    assert near <= 1 + len(u) // 100
    return out


@pytest.mark.parametrize("n,V", [(1, 1), (3, 2), (1, 7), (5, 8), (2, 9), (4, 100), (3, 4095), (2, 4096), (2, 4097),
                                 (1, 8192), (1, 30011), (7, 65537), (1, 126464), (9, 126464), (40, 32003), (160, 5000),
                                 (700, 999)])
def test_sizes(dllm, n, V):
    """Clusters of 1 to 8 CTAs, rows that leave some of them nothing, more rows than the grid holds."""
    rng = np.random.default_rng(V + n)
    check(dllm, rows(rng, n, V, "plain"), rng.random(n))
    check(dllm, rows(rng, n, V, "plain"), rng.random(n), settings(rng, n), ldv=-(-V // 8) * 8 + 16)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n,V", [(3, 30011), (330, 3001)])
def test_values(dllm, kind, n, V):
    rng = np.random.default_rng(KINDS.index(kind))
    x = rows(rng, n, V, kind)
    check(dllm, x, rng.random(n))
    check(dllm, x, rng.random(n), settings(rng, n))
    check(dllm, x, rng.random(n), {"temperature": np.full(n, 3e38, dtype=np.float32)})


def test_many_equal_tokens(dllm):
    """More tokens of the drawn value than are gathered at once, from the first to the last."""
    n, V = 6, 126465
    x = np.full((n, V), 2.0)
    x[:, 7] = -1.0
    u = np.array([0.0, 0.25, 0.5, 0.75, 1 - 2.0 ** -24, 2.0])
    check(dllm, x, u)
    rng = np.random.default_rng(1)
    x = rng.choice([0.0, -0.0, -1.0], (n, V))
    check(dllm, x, u)


def test_random_numbers_out_of_range(dllm):
    rng = np.random.default_rng(2)
    x = rows(rng, 5, 2000, "plain")
    check(dllm, x, np.array([-1.0, -1e-9, 1.0, 7.0, np.inf]))
    import torch
    dev = torch.device("cuda", 0)
    out = dllm.sample(torch.from_numpy(x).to(torch.bfloat16).to(dev), torch.full((5,), float("nan"), device=dev))
    assert out["tokens"].tolist() == [int(r.argmax()) for r in x]


def test_rows_that_give_none(dllm):
    """NaN, infinity and nothing at all, wherever in the row; entries without a row; temperatures that are none."""
    n, V = 8, 50000
    rng = np.random.default_rng(3)
    x = rows(rng, n, V, "plain")
    x[0, 0], x[1, V - 1], x[2, 33333] = np.nan, np.nan, np.inf
    x[3] = -np.inf
    x[4, :] = -np.inf
    x[4, 49999] = -3.0
    check(dllm, x, rng.random(n))
    order = [5, -1, 4, 8, 2, 2 ** 31 - 1, 7, 0, 5, -2 ** 31]
    check(dllm, x, rng.random(10), row_of=order)
    given = {"temperature": np.array([1, -1, np.nan, 1, np.inf, np.inf, 1e-45, -0.0], dtype=np.float32)}
    check(dllm, x, rng.random(n), given)


def test_temperatures_far_out(dllm):
    rng = np.random.default_rng(4)
    n = 12
    x = rows(rng, n, 9000, "plain")
    T = np.array([1e-45, 1e-38, 1e-20, 1e-6, 0.01, 3, 50, 1e4, 1e20, 3e38, np.inf, 0.1], dtype=np.float32)
    check(dllm, x, rng.random(n), {"temperature": T})
    check(dllm, rows(rng, n, 9000, "huge"), rng.random(n), {"temperature": T})


def test_frequencies(dllm):
    """Draws with u over an even grid give each token its share, to a grid step."""
    import torch
    dev = torch.device("cuda", 0)
    x = torch.tensor([[1.0, 0.0, 2.0, -1.0, 2.0, 0.5, -3.0, 1.0]], device=dev).to(torch.bfloat16)
    n = 4096
    u = (torch.arange(n, device=dev, dtype=torch.float32) + 0.5) / n
    out = dllm.sample(x, u, rows=torch.zeros(n, dtype=torch.int32, device=dev))
    p = torch.softmax(x.double()[0], 0)
    got = torch.bincount(out["tokens"].long(), minlength=8).double() / n
    assert float((got - p).abs().max()) <= 1.0 / n


def test_equal_calls_batches_and_graphs(dllm):
    """A row's draw does not depend on its batch; a captured call replays; another stream gives the same."""
    import torch
    dev = torch.device("cuda", 0)
    rng = np.random.default_rng(5)
    n, V = 400, 20000
    x = torch.from_numpy(rows(rng, n, V, "flat")).to(torch.bfloat16).to(dev)
    u = torch.rand(n, device=dev)
    whole = dllm.sample(x, u)
    for k in (0, 1, 17, 399):
        one = dllm.sample(x, u[k:k + 1].contiguous(), rows=torch.tensor([k], dtype=torch.int32, device=dev))
        assert one["tokens"][0] == whole["tokens"][k] and one["prob"][0] == whole["prob"][k]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = dllm.sample(x, u)
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out["tokens"], whole["tokens"]) and torch.equal(out["prob"], whole["prob"])
        u.copy_(torch.rand(n, device=dev))
        whole = dllm.sample(x, u)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out = dllm.sample(x, u)
    torch.cuda.synchronize()
    assert torch.equal(out["tokens"], whole["tokens"])
    assert dllm.get_device_error(dev) == 0


def test_calls_at_once(dllm):
    """Calls of one row (a cluster of CTAs) and of many, on streams of their own and in graphs replayed side by side, and
    products between them: everyone gets its own draws."""
    import torch
    dev = torch.device("cuda", 0)
    rng = np.random.default_rng(6)
    work = []
    for n, V in ((1, 126464), (3, 40000), (200, 9000), (37, 32003)):
        x = torch.from_numpy(rows(rng, n, V, "plain")).to(torch.bfloat16).to(dev)
        x = torch.nn.functional.pad(x, (0, -V % 8)).contiguous()
        work.append((x, torch.rand(n, device=dev), V))
    want = [dllm.sample(x, u, V=V) for x, u, V in work]
    a, sa = dllm.fp8_quantize(torch.randn(300, 512, device=dev).to(torch.bfloat16))
    b, sb = dllm.fp8_quantize(torch.randn(2000, 512, device=dev).to(torch.bfloat16), block_rows=128)
    product = dllm.fp8_matmul(a, sa, b, sb)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for x, u, V in work:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append((dllm.sample(x, u, V=V), dllm.fp8_matmul(a, sa, b, sb)))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(8)]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for k, (x, u, V) in enumerate(work):
            with torch.cuda.stream(streams[k]):
                got.append((k, dllm.sample(x, u, V=V)))
            with torch.cuda.stream(streams[4 + k]):
                graphs[k].replay()
    torch.cuda.synchronize()
    for k, o in got + [(k, o[0]) for k, o in enumerate(outs)]:
        assert torch.equal(o["tokens"], want[k]["tokens"]) and torch.equal(o["prob"], want[k]["prob"])
    assert all(torch.equal(o[1], product) for o in outs)
    assert dllm.get_device_error(dev) == 0
