"""examples/block_cache.py: the operators around the step, together."""
import importlib.util
import os

import numpy as np
import pytest

from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("block_cache", os.path.join(ROOT, "examples", "block_cache.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("L,budget", [(8, 48), (1, 30), (33, 100)])
def test_block_cache(dllm, example, L, budget):
    """Blocks fill, caches stay within their budget, reports say what 64 bits say of
    the logits, and a second run gives the same bits."""
    prompts = [range(5, 12), range(100, 140), [1]]
    runs = [example.decode(prompts, L=L, blocks=4, budget=budget, say=lambda s: None) for _ in range(2)]
    tokens, lens, reports = runs[0]
    assert dllm.get_device_error() == 0
    assert tokens.shape == (3, 4 * L) and int(tokens.min()) >= 0 and int(tokens.max()) < 2000
    want = [len(p) for p in prompts]
    for _ in range(4):
        want = [n + L for n in want]
        if max(want) > budget:
            want = [min(n, budget) for n in want]
    assert lens.tolist() == want
    for i, r in enumerate(reports):
        x = r["logits"].double().cpu().numpy()
        lp = x - x.max(1, keepdims=True)
        lp -= np.log(np.exp(lp).sum(1, keepdims=True))
        asked = tokens[:, i * L:(i + 1) * L].reshape(-1).cpu().numpy()
        np.testing.assert_allclose(r["logprob"].cpu().numpy(), lp[np.arange(len(asked)), asked], rtol=1e-5, atol=1e-5)
        np.testing.assert_allclose(r["entropy"].cpu().numpy(), -(np.exp(lp) * lp).sum(1), rtol=1e-5, atol=1e-5)
        np.testing.assert_array_equal(r["top_ids"][:, 0].cpu().numpy(), x.argmax(1))
        assert bool(r["lse"].isfinite().all())
    for a, b in zip(reports, runs[1][2]):
        for k in a:
            assert (a[k] == b[k]).all(), k
    assert (runs[1][0] == tokens).all()
