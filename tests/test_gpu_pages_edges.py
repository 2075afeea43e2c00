"""dllm_pages_*: forks of requests whose tables name pages outside the pool, and sums at the limits."""
import numpy as np
import pytest

from test_gpu_pages import State

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("entry", [-1, 200, 2 ** 31 - 1, -2 ** 31])
@pytest.mark.parametrize("length", [160, 150])   # ends with a page; inside one
@pytest.mark.parametrize("at", [0, 5, 8])
def test_fork_of_a_row_with_a_bad_page(dllm, entry, length, at):
    """A page outside the pool among the full ones: the fork is not served, takes no page and spreads nothing; the forks
    beside it are as they would be without it."""
    rng = np.random.default_rng(at)
    s = State(rng, 200, 4, 12, 16, [160, length, 33, 90], spare_rows=40)
    s.table[1, at] = entry
    s.upload()
    src, dst = [0, 1, 2, 1, 3] + [2] * 34, list(range(4, 43))
    before = [t.clone() for t in (s.g_table, s.g_refs)]
    fresh = dllm.page_fork(s.g_pools, s.g_refs, s.g_table, s.g_held, s.g_lens, s.rows(src), s.rows(dst), page_size=16)
    assert dllm.get_device_error(s.dev) == 5
    assert fresh[1] == -2 and fresh[3] == -2
    for f in (1, 3):
        assert s.g_held[dst[f]] == 0 and s.g_lens[dst[f]] == 0
        assert (s.g_table[dst[f]] == before[0][dst[f]]).all()
    good = [(a, b) for a, b in zip(src, dst) if a != 1]
    import pages_reference as ref
    want, error = ref.fork(s.pools, s.refs, s.table, s.held, s.lens, [a for a, _ in good], [b for _, b in good], 16)
    assert not error and [fresh.tolist()[b - 4] for _, b in good] == want
    s.same(dllm)


def test_forks_of_long_rows_are_checked_to_their_end(dllm):
    """Rows of thousands of pages, and more forks than a round of the deciding block."""
    import torch
    rng = np.random.default_rng(3)
    s = State(rng, 9000, 2, 4100, 1, [4000, 4100], arrays=(), spare_rows=1100)
    s.table[1, 4099] = 9000
    s.upload()
    fresh = dllm.page_fork([], s.g_refs, s.g_table, s.g_held, s.g_lens, s.rows([0, 1] * 550), s.rows(range(2, 1102)),
                           page_size=1)
    assert dllm.get_device_error(s.dev) == 5
    assert fresh.tolist() == [-1, -2] * 550
    assert s.g_held[2:].tolist() == [4000, 0] * 550
    assert torch.equal(s.g_table[2::2, :4000], s.g_table[:1, :4000].expand(550, -1))
    assert torch.equal(s.g_refs[s.g_table[0, :4000].long()], torch.full((4000,), 551, dtype=torch.int32, device=s.dev))


def test_growth_at_the_limits_of_its_sums(dllm):
    """The largest pool, full, and rounds of rows that want 2^30 pages each: nobody is served, and that is recorded."""
    import torch
    dev = torch.device("cuda", 0)
    n_pages, R, most = 2 ** 30 - 1, 2048, 2 ** 20
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 24 GB")
    refs = torch.ones(n_pages, dtype=torch.int32, device=dev)
    table = torch.empty(R, most, dtype=torch.int32, device=dev)
    held, lens = torch.zeros(R, dtype=torch.int32, device=dev), torch.full((R,), most, dtype=torch.int32, device=dev)
    rows = torch.arange(R, dtype=torch.int32, device=dev)
    taken = dllm.page_grow(refs, table, held, lens, rows, 0, page_size=1)
    assert bool((taken == -1).all()) and not held.any()
    assert dllm.get_device_error(dev) == 5
    del refs, table
    torch.cuda.empty_cache()


def test_copies_within_one_pool(dllm):
    """Source and destination in the same tensors: disjoint pages, several copies of one, skipped ones."""
    rng = np.random.default_rng(4)
    s = State(rng, 100, 2, 8, 16, [100, 17], arrays=((4096 + 48,), (16,), (3, 32)))
    order = rng.permutation(100)
    src, dst = order[:40].copy(), order[40:80].copy()
    src[7:12] = src[3]
    src[20], dst[21] = -1, -1
    dllm.page_copy(s.g_pools, s.g_pools, s.rows(src), s.rows(dst))
    for a in s.pools:
        for x, y in zip(src, dst):
            if x >= 0 and y >= 0:
                a[y] = a[x]
    s.same(dllm)


@pytest.mark.parametrize("n_pages", [40, 9000])
def test_pools_without_arrays(dllm, n_pages):
    """Tables and counts alone, where the contents are someone else's: forks, release, compaction."""
    rng = np.random.default_rng(5)
    s = State(rng, n_pages, 4, 10, 16, [40, 16, 33, 20], arrays=(), spare_rows=3)
    s.fork(dllm, [0, 2, 0], [4, 5, 6])
    s.free(dllm, [0, 1])
    s.compact(dllm)
    s.grow(dllm, [2, 4], 50)
    s.compact(dllm)
