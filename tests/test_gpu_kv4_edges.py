"""The 4-bit cache on the GPU where ranges, paddings and sharing end.

Tolerances are those of test_gpu_kv4.py; what is compared for equality is exact
by the operators' definitions."""
import numpy as np
import pytest

from test_gpu_kv4 import Cache, bf16

pytestmark = pytest.mark.gpu


def test_calls_of_several_threads_on_one_stream(dllm):
    """Threads that call on the same stream, with requests, lengths and rows of
    their own, get their own results."""
    import threading
    import torch
    dev = torch.device("cuda", 0)
    rng = np.random.default_rng(60)
    work = []
    for B, L in ((1, 40), (64, 40), (7, 70), (30, 1)):
        cache = Cache(rng, rng.integers(1, 400, B), 1, 64, 16)
        args = (bf16(rng.standard_normal((B, L, 2, 64)), dev), *cache.upload(dev))
        work.append((args, dllm.kv4_attend(*args)))
    torch.cuda.synchronize()
    stream = torch.cuda.current_stream()
    wrong = []

    def run(args, want):
        with torch.cuda.stream(stream):
            outs = [dllm.kv4_attend(*args) for _ in range(40)]
            stream.synchronize()
            wrong.extend(k for o in outs for k in want if not torch.equal(o[k], want[k]))
    threads = [threading.Thread(target=run, args=w) for w in work * 2]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    assert dllm.get_device_error(dev) == 0
