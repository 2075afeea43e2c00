"""token_logprobs on the GPU: whole rows of several rounds, maxima where the
arithmetic changes, and vocabularies near the largest.

Tolerance: that of test_gpu_logprobs.py, 1e-5 max(1, |value|)."""
import numpy as np
import pytest

import kv4_reference as ref
from test_gpu_logprobs import TOL, check, rows, upload

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("size", [16383.7, 16380.3, 16384.0])
def test_maxima_where_the_arithmetic_changes(dllm, size, sign):
    """Sums begun under a maximum within 16384 and ended under one beyond it, and
    the reverse: both forms of c x - c m stand for the same numbers."""
    V = 40009
    rng = np.random.default_rng(8)
    x = np.full((4, V), sign * size, dtype=np.float32)
    x[0, V // 2:] = sign * size + 0.6       # later values pass the bound, or come back within it
    x[1, : V // 2] = sign * size + 0.6
    x[2] += rng.uniform(-1, 1, V).astype(np.float32)
    x[3] = np.sort(x[2])
    check(dllm, x, [3, V - 1, 17, 0], 4, "f32", 40016)


@pytest.mark.parametrize("dtype,V", [("f32", 2 ** 30 + 1003), ("bf16", 2 ** 31 - 1)])
def test_vocabularies_near_the_largest(dllm, dtype, V):
    """Byte counts and ends of rounds that pass 32 bits: one row of 4 GB."""
    import torch
    dev = torch.device("cuda", 0)
    ldv = -(-V // 8) * 8
    logits = torch.full((1, ldv), float("-inf"), dtype=torch.float32 if dtype == "f32" else torch.bfloat16, device=dev)
    logits[0, V:] = float("nan")
    at = np.array([0, 5, 1500, 2040, 4095, 4096, V // 3, V - 4097, V - 700, V - 1])
    vals = np.array([1.5, 3.0, 7.0, -2.0, 6.5, 0.25, 2.0, 4.0, 5.0, 6.0], dtype=np.float32)
    logits[0, torch.from_numpy(at).to(dev)] = torch.from_numpy(vals).to(dev).to(logits.dtype)
    out = dllm.token_logprobs(logits, torch.tensor([1500], dtype=torch.int32, device=dev), V=V, top=12)
    got = {k: v.cpu().numpy()[0] for k, v in out.items()}
    lp, ent, order, tlp = ref.logprobs(vals, 2, 10)
    np.testing.assert_allclose(got["logprob"], lp, rtol=TOL, atol=TOL)
    np.testing.assert_allclose(got["entropy"], ent, rtol=TOL, atol=TOL)
    np.testing.assert_array_equal(got["top_ids"][:10], at[order])
    np.testing.assert_allclose(got["top_logprobs"][:10], tlp, rtol=TOL, atol=TOL)
    # the rest are the lowest tokens of probability 0
    rest = [v for v in range(12) if v not in at][:2]
    np.testing.assert_array_equal(got["top_ids"][10:], rest)
    assert np.isneginf(got["top_logprobs"][10:]).all()
    assert dllm.get_device_error(dev) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["peaked", "ties", "equal", "ascending", "masked", "lowest", "signed_zero"])
@pytest.mark.parametrize("top", [0, 3, 32])
def test_whole_rows_of_several_rounds(dllm, dtype, kind, top):
    """At most six CTAs run on an SM, so with 18 rows to each SM a CTA has two
    whole rows or more, 8 (bf16) or 15 (f32) rounds each: lists, floors and sums
    are used again from row to row."""
    import torch
    dev = torch.device("cuda", 0)
    V = 30011
    n = 18 * torch.cuda.get_device_properties(dev).multi_processor_count
    x = rows(np.random.default_rng(6), 5, V, dtype, kind)
    rng = np.random.default_rng(7)
    idx = rng.integers(0, 5, n)
    tokens = rng.integers(0, V, 5)
    out = dllm.token_logprobs(upload(x, dtype, 30016, dev), torch.tensor(tokens[idx], dtype=torch.int32, device=dev), V=V,
                              top=top, rows=torch.tensor(idx, dtype=torch.int32, device=dev))
    got = {k: v.cpu().numpy() for k, v in out.items()}
    for r in range(5):
        mine = idx == r
        lp, ent, ids, tlp = ref.logprobs(x[r], tokens[r], top)
        want = {"logprob": lp, "entropy": ent}
        if top:
            np.testing.assert_array_equal(got["top_ids"][mine], np.broadcast_to(ids, (mine.sum(), top)))
            want["top_logprobs"] = tlp
        for name, w in want.items():
            np.testing.assert_allclose(got[name][mine], np.broadcast_to(w, got[name][mine].shape), rtol=TOL, atol=TOL)
    assert dllm.get_device_error(dev) == 0
