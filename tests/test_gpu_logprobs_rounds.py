"""token_logprobs on the GPU: whole rows of several rounds, maxima where the
arithmetic changes, and vocabularies near the largest.

Tolerance: that of test_gpu_logprobs.py, 1e-5 max(1, |value|)."""
import numpy as np
import pytest


from test_gpu_logprobs import check

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
