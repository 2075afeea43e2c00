"""The 4-bit cache on the GPU where ranges, paddings and sharing end.

Tolerances are those of test_gpu_kv4.py; what is compared for equality is exact
by the operators' definitions."""
import numpy as np
import pytest

import kv4_reference as ref
from test_gpu_kv4 import Cache, bf16, check_attend

pytestmark = pytest.mark.gpu

BIG = 3.3895313892515355e38   # bf16's largest


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


def operators(dllm, dev, seed):
    """Calls of both operators that take a workspace, the attention at few and at
    many rows, and their outputs."""
    import torch
    rng = np.random.default_rng(seed)
    cache = Cache(rng, [3000, 700, 1], 2, 128, 32)
    pages, table, lens = cache.upload(dev)
    few, many = (bf16(rng.standard_normal((3, L, 14, 128)), dev) for L in (1, 16))
    logits = bf16(rng.standard_normal((9, 40000)), dev)
    tokens = torch.arange(9, dtype=torch.int32, device=dev)
    w = torch.zeros(pages.shape[0], 2, 32, device=dev)

    def call():
        return [dllm.token_logprobs(logits, tokens, top=7), dllm.kv4_attend(few, pages, table, lens, weights=w),
                dllm.kv4_attend(many, pages, table, lens)]
    return call


def test_captured_in_graphs(dllm):
    """Graphs captured one after the other replay in any order, between eager
    calls and side by side, with the bits of the eager calls."""
    import torch
    dev = torch.device("cuda", 0)
    calls = [operators(dllm, dev, s) for s in (50, 51, 52)]
    want = [[{k: t.clone() for k, t in o.items()} for o in c()] for c in calls]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(c())
        graphs.append(g)

    def same(i):
        torch.cuda.synchronize()
        for got, exp in zip(outs[i], want[i]):
            for k in exp:
                assert torch.equal(got[k], exp[k]), (i, k)
                got[k].zero_()
    for i in (2, 0, 1, 1, 0):
        graphs[i].replay()
        calls[1]()
        same(i)
    side = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for g, s in zip(graphs, side):
        with torch.cuda.stream(s):
            g.replay()
    for i in range(3):
        same(i)
    assert dllm.get_device_error(dev) == 0


@pytest.mark.parametrize("low,high", [(-2e38, 2e38), (-3.3e38, 3.3e38), (-BIG, BIG), (-BIG, 1.0), (0.0, BIG),
                                      (-1.0, BIG), (-BIG, 2e38), (-12000.0, 12000.0), (-20000.0, 300.0)])
def test_write_ranges_that_saturate(dllm, low, high):
    """Steps past their largest, up to ranges that no 32-bit number holds: codes,
    parameters and values are those of the definition."""
    import torch
    dev = torch.device("cuda", 0)
    rng = np.random.default_rng(40)
    x = rng.uniform(-0.5, 0.5, (1, 8, 2, 2, 64)) * min(abs(high - low), 1e38)
    x[..., 0::32], x[..., 17::32] = low, high
    x[0, 3, :, :, 5] = 0.0
    x = ref.from_bf16(ref.to_bf16(np.clip(x, low, high)))
    pages, _ = dllm.kv4_pages(1, 2, 16, 64, dev)
    t = bf16(x, dev)
    out = [torch.empty((1, 8, 2, 64), dtype=torch.bfloat16, device=dev) for _ in range(2)]
    zero = torch.zeros(1, dtype=torch.int32, device=dev)
    dllm.kv4_write(t[:, :, 0], t[:, :, 1], pages, zero[None], zero, k_out=out[0], v_out=out[1])
    assert dllm.get_device_error(dev) == 0
    rows = np.zeros((2, 1, 2, 16, 64))
    rows[:, 0, :, :8] = x[0].transpose(1, 2, 0, 3)
    want = ref.pages_of(rows[0], rows[1], 16)
    got = pages.cpu().numpy()
    for at, size in ((0, 32), (16 * 32, 4), (16 * 36, 32), (16 * 68, 4)):   # the eight tokens written
        np.testing.assert_array_equal(got[..., at:at + 8 * size], want[..., at:at + 8 * size])
    vals = ref.values_of(want, 16, 64)
    for i in range(2):
        np.testing.assert_array_equal(out[i][0].float().cpu().numpy(), vals[i][0].transpose(1, 0, 2)[:8])


def fill_shared_memory(dllm, dev, seed):
    """Other kernels' data in every SM's shared memory: logits of any bits."""
    import torch
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    bits = torch.randint(-2 ** 15, 2 ** 15, (2048, 30016), dtype=torch.int16, generator=gen, device=dev)
    dllm.token_logprobs(bits.view(torch.bfloat16), torch.zeros(2048, dtype=torch.int32, device=dev))


# rows that fill no warp: 56 and 100 (two streams share them), 234 of 256, and 700 in blocks of 234, 234 and 232
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("L,H", [(8, 7), (25, 4), (39, 6), (100, 7)])
def test_attend_equal_bits_with_rows_that_fill_no_warp(dllm, L, H, D):
    """Equal calls give equal bits whatever ran before them, and whichever item
    a CTA had before."""
    import torch
    dev = torch.device("cuda", 0)
    rng = np.random.default_rng(41)
    lens = rng.integers(100, 1500, 40)
    cache = Cache(rng, lens, 1, D, 32)
    q = rng.standard_normal((40, L, H, D)) * np.exp2(rng.integers(-3, 4, (40, L, H, 1)))
    pages, table, tl = cache.upload(dev)
    tq = bf16(q, dev)
    want = dllm.kv4_attend(tq, pages, table, tl)
    for i in range(8):
        fill_shared_memory(dllm, dev, i)
        got = dllm.kv4_attend(tq, pages, table, tl)
        for k in want:
            assert torch.equal(got[k], want[k]), (k, i)


def test_refused_workspaces(dllm):
    """A workspace on the host, of another type, misaligned or in pieces is
    refused before anything is launched."""
    import torch
    dev = torch.device("cuda", 0)
    pages, _ = dllm.kv4_pages(2, 1, 16, 64, dev)
    table = torch.zeros(1, 2, dtype=torch.int32, device=dev)
    one = torch.ones(1, dtype=torch.int32, device=dev)
    q = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16, device=dev)
    n = 64 << 20
    good = torch.zeros(n, dtype=torch.uint8, device=dev)
    calls = (lambda w: dllm.kv4_attend(q, pages, table, one, workspace=w),
             lambda w: dllm.token_logprobs(torch.zeros(1, 64, device=dev), one, workspace=w))
    for call in calls:
        call(good)
        for bad in (torch.zeros(n, dtype=torch.uint8), good[::2], torch.zeros(n // 4, device=dev)):
            with pytest.raises((ValueError, TypeError)):
                call(bad)
        with pytest.raises(dllm.DllmError):
            call(good[16:])
    assert dllm.get_device_error(dev) == 0


def test_refused_shapes(dllm):
    """Wrong numbers of dimensions, and none at all, are refused by name."""
    import torch
    dev = torch.device("cuda", 0)
    pages, weights = dllm.kv4_pages(2, 1, 16, 64, dev)
    table = torch.zeros(1, 2, dtype=torch.int32, device=dev)
    one = torch.ones(1, dtype=torch.int32, device=dev)
    q = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16, device=dev)
    for flat in (pages[0], pages.reshape(-1)):
        with pytest.raises((TypeError, ValueError)):
            dllm.kv4_attend(q, flat, table, one)
        with pytest.raises((TypeError, ValueError)):
            dllm.kv4_write(q, q, flat, table, one)
        with pytest.raises((TypeError, ValueError)):
            dllm.kv4_evict(flat, weights, table, one, one, table)
    with pytest.raises((TypeError, ValueError)):
        dllm.kv4_attend(q[..., :0], pages, table, one)
    with pytest.raises((TypeError, ValueError)):
        dllm.kv4_write(q[..., :0], q[..., :0], pages, table, one)
    with pytest.raises((TypeError, ValueError)):
        dllm.kv4_evict(pages, weights[:, :, :0].contiguous(), table, one, one, table)


# query rows per key/value head at the edges of the kernels' rules, with the tokens' weights
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("L,H", [(8, 4), (11, 3), (16, 7), (32, 4), (43, 3), (32, 8), (33, 8), (64, 8), (257, 1), (100, 7)])
def test_attend_rows_at_the_rules_edges(dllm, L, H, D):
    """32, 33, 112, 128, 129, 256, 264, 512, 257 and 700 rows: of 257, the second
    block's rows leave a stream without any."""
    rng = np.random.default_rng(42)
    lens = [0, 1, 128, 129, 400, 1300]
    cache = Cache(rng, lens, 1, D, 32)
    check_attend(dllm, cache, rng.standard_normal((len(lens), L, H, D)), weights=True)


def test_evict_reports_pages_far_into_a_long_cache(dllm):
    """A table entry outside the pool is recorded wherever its tokens lie, kept or
    not; the other requests' choices stand."""
    import torch
    dev = torch.device("cuda", 0)
    heads, page, n = 80, 256, 13 * 1024
    per = n // page
    pages, weights = dllm.kv4_pages(2 * per + 2, heads, page, 64, dev)
    weights.copy_(1 + torch.rand(weights.shape, device=dev))
    table = torch.arange(2 * per, dtype=torch.int32, device=dev).reshape(2, per)
    dst = torch.tensor([[2 * per], [2 * per + 1]], dtype=torch.int32, device=dev)
    lens, keep = (torch.full((2,), x, dtype=torch.int32, device=dev) for x in (n, 40))
    good = dllm.kv4_evict(pages, weights.clone(), table, lens, keep, dst)
    assert dllm.get_device_error(dev) == 0
    for where in (0, 30, per - 2):
        for entry in (-1, 2 * per + 2):
            bad = table.clone()
            bad[0, where] = entry
            out = dllm.kv4_evict(pages, weights.clone(), bad, lens, keep, dst)
            assert dllm.get_device_error(dev) == 5, (where, entry)
            assert torch.equal(out["src"][1], good["src"][1])


@pytest.mark.parametrize("first", [-1, -5, -2 ** 31])
def test_write_first_columns_below_zero(dllm, first):
    """Recorded however far below, with the columns counted or not; nothing is
    written for that request."""
    import torch
    dev = torch.device("cuda", 0)
    pages, _ = dllm.kv4_pages(4, 1, 16, 64, dev)
    table = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device=dev)
    k = torch.randn(2, 4, 1, 64, device=dev).to(torch.bfloat16)
    pos = torch.zeros(2, dtype=torch.int32, device=dev)
    start = torch.tensor([first, 1], dtype=torch.int32, device=dev)
    for count in (None, torch.tensor([3, 3], dtype=torch.int32, device=dev)):
        pages.zero_()
        dllm.kv4_write(k, k, pages, table, pos, first=start, count=count)
        assert dllm.get_device_error(dev) == 5
        assert not pages[:2].any() and pages[2].any()
