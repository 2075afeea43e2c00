"""examples/several_tries.py, and the step over drawn tokens."""
import importlib.util
import os

import numpy as np
import pytest

from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("several_tries", os.path.join(ROOT, "examples", "several_tries.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("tries,L", [(3, 8), (1, 16), (5, 5)])
def test_several_tries(dllm, example, tries, L):
    """Blocks fill, every page is counted by those who hold it, the pool ends without gaps, and a second run gives the
    same tokens."""
    prompts = [range(5, 12), range(100, 140), [1]]
    runs = [example.decode(prompts, tries=tries, L=L, say=lambda s: None) for _ in range(2)]
    tokens, (refs, table, held, lens) = runs[0]
    assert dllm.get_device_error() == 0
    assert tokens.shape == (3, 3 * L) and int(tokens.min()) >= 0 and int(tokens.max()) < 2000
    assert lens[:3].tolist() == [len(p) + 3 * L for p in prompts]
    assert held[:3].tolist() == [-(-(len(p) + 3 * L) // 16) for p in prompts] and not held[3:].any()
    used = int(held.sum())
    count = np.zeros(len(refs), dtype=np.int32)
    for b, h in enumerate(held.tolist()):
        np.add.at(count, table[b, :h].cpu().numpy(), 1)
    np.testing.assert_array_equal(refs.cpu().numpy(), count)
    assert (count[:used] == 1).all() and not count[used:].any()
    assert (runs[1][0] == tokens).all()


@pytest.mark.parametrize("quota", [False, True])
def test_step_over_drawn_tokens(dllm, quota):
    """At temperature 0 the draw is the argmax with probability 1: all masked positions go at once.  Otherwise the
    positions whose draws pass the threshold, or the surest one."""
    import torch
    dev = torch.device("cuda", 0)
    rng = np.random.default_rng(0)
    B, L, V = 6, 8, 500
    mask = V
    logits = torch.from_numpy(rng.standard_normal((B * L, 504)) * 3).to(torch.bfloat16).to(dev)
    ids0 = torch.from_numpy(np.where(rng.random((B, L)) < 0.6, mask, 3).astype(np.int32)).to(dev)
    ids0[0] = 3                                   # nothing masked
    rows = torch.where(ids0.view(-1) == mask, torch.arange(B * L, dtype=torch.int32, device=dev), -1).to(torch.int32)
    thr = torch.full((B,), 0.5, device=dev)
    left = torch.full((B,), 2, dtype=torch.int32, device=dev) if quota else None
    for T in (0.0, 0.7):
        d = dllm.sample(logits, torch.rand(B * L, device=dev), V=V, rows=rows,
                        temperature=torch.full((B * L,), T, device=dev))
        ids, conf = ids0.clone(), torch.full((B, L), float("nan"), device=dev)
        out = dllm.step_sampled(d["tokens"], d["prob"], ids, thr, conf, V=V, mask_id=mask, quota=left, debug=True)
        assert dllm.get_device_error(dev) == 0
        p, t = d["prob"].view(B, L).cpu().numpy(), d["tokens"].view(B, L).cpu().numpy()
        masked = (ids0 == mask).cpu().numpy()
        for b in range(B):
            at = np.flatnonzero(masked[b])
            order = at[np.argsort(-p[b, at], kind="stable")]
            take = order[:2] if quota else order[p[b, order] > 0.5] if (p[b, at] > 0.5).any() else order[:1]
            want = ids0[b].cpu().numpy().copy()
            want[take] = t[b, take]
            np.testing.assert_array_equal(ids[b].cpu().numpy(), want)
            assert int(out["n_new"][b]) == len(take)
            np.testing.assert_allclose(conf[b].cpu().numpy()[take], p[b, take], rtol=2.0 ** -22)   # two quotients
            assert int(out["done"][b]) == int(len(take) == len(at))
