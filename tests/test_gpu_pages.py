"""dllm_pages_* on the GPU against plain Python: whole numbers and bytes, so equality throughout."""
import numpy as np
import pytest

import pages_reference as ref

pytestmark = pytest.mark.gpu


class State:
    """A pool with requests in it, on both sides."""

    def __init__(self, rng, n_pages, B, max_pages, page, lens, arrays=((48,), (5, 16)), spare_rows=0):
        import torch
        self.dev = torch.device("cuda", 0)
        self.page = page
        self.pools = [rng.integers(0, 256, (n_pages, *s)).astype(np.uint8) for s in arrays]
        self.refs = np.zeros(n_pages, dtype=np.int32)
        self.table = rng.integers(-5, n_pages + 5, (B + spare_rows, max_pages)).astype(np.int32)
        self.lens = np.zeros(B + spare_rows, dtype=np.int32)
        self.held = np.zeros(B + spare_rows, dtype=np.int32)
        order = rng.permutation(n_pages)
        at = 0
        for b, n in enumerate(lens):
            k = -(-int(n) // page)
            self.lens[b], self.held[b] = n, k
            self.table[b, :k] = order[at:at + k]
            self.refs[order[at:at + k]] = 1
            at += k
        self.upload()

    def upload(self):
        import torch
        t = lambda x: torch.from_numpy(x.copy()).to(self.dev)  # noqa: E731
        self.g_pools = [t(a) for a in self.pools]
        self.g_refs, self.g_table, self.g_held, self.g_lens = t(self.refs), t(self.table), t(self.held), t(self.lens)

    def rows(self, r):
        import torch
        return torch.tensor(list(r), dtype=torch.int32, device=self.dev)

    def same(self, dllm, error=False):
        assert dllm.get_device_error(self.dev) == (5 if error else 0)
        for a, b in ((self.refs, self.g_refs), (self.table, self.g_table), (self.held, self.g_held), (self.lens, self.g_lens)):
            np.testing.assert_array_equal(b.cpu().numpy(), a)
        for a, b in zip(self.pools, self.g_pools):
            np.testing.assert_array_equal(b.cpu().numpy(), a)

    def fork(self, dllm, src, dst):
        want, error = ref.fork(self.pools, self.refs, self.table, self.held, self.lens, src, dst, self.page)
        got = dllm.page_fork(self.g_pools, self.g_refs, self.g_table, self.g_held, self.g_lens, self.rows(src),
                             self.rows(dst), page_size=self.page)
        assert got.tolist() == want
        self.same(dllm, error)

    def grow(self, dllm, rows, extra):
        want, error = ref.grow(self.refs, self.table, self.held, self.lens, rows, extra, self.page)
        got = dllm.page_grow(self.g_refs, self.g_table, self.g_held, self.g_lens, self.rows(rows), extra,
                             page_size=self.page)
        assert got.tolist() == want
        self.same(dllm, error)

    def free(self, dllm, rows):
        error = ref.release(self.refs, self.table, self.held, rows)
        dllm.page_free(self.g_refs, self.g_table, self.g_held, self.rows(rows))
        self.same(dllm, error)

    def compact(self, dllm):
        U, new = ref.compact(self.pools, self.refs, self.table, self.held)
        out = dllm.page_compact(self.g_pools, self.g_refs, self.g_table, self.g_held)
        assert out["used"].tolist() == [U]
        np.testing.assert_array_equal(out["map"].cpu().numpy(), new)
        self.same(dllm)


@pytest.mark.parametrize("page", [1, 16, 100])
@pytest.mark.parametrize("n_pages,B,forks", [(40, 1, 1), (300, 4, 3), (9000, 30, 70), (20000, 9, 1500)])
def test_life_of_a_pool(dllm, n_pages, B, forks, page):
    """Forks (several of one source), growth, release, compaction, and again."""
    rng = np.random.default_rng(n_pages + page)
    lens = rng.integers(0, max(2, min(10, n_pages // (4 * B)) * page), B)
    s = State(rng, n_pages, B, 40, page, lens, spare_rows=forks)
    s.fork(dllm, rng.integers(0, B, forks).tolist(), list(range(B, B + forks)))
    s.grow(dllm, rng.permutation(B + forks)[:forks].tolist(), 3 * page)
    s.free(dllm, rng.permutation(B + forks)[:(B + forks) // 2].tolist())
    s.compact(dllm)
    s.compact(dllm)
    live = [b for b in range(B + forks) if s.held[b]]
    spare = [b for b in range(B + forks) if not s.held[b]]
    if live and spare:
        s.fork(dllm, live[:1] * len(spare), spare)
    s.free(dllm, list(range(B + forks)))
    assert not s.refs.any()
    s.compact(dllm)


@pytest.mark.parametrize("arrays", [((16,),), ((4096,), (4112,), (16,)), ((3, 40000),), ((16,),) * 64, ((131072 + 48,), (48,)) * 3])
def test_contents_of_every_size(dllm, arrays):
    """Pages of 16 bytes to some hundred KB, 1 to 64 arrays: copies to another pool, forks and moves."""
    import torch
    rng = np.random.default_rng(7)
    s = State(rng, 60, 5, 8, 16, [100, 17, 16, 1, 0], arrays=arrays, spare_rows=5)
    s.fork(dllm, [0, 1, 2, 3, 4], [5, 6, 7, 8, 9])
    s.free(dllm, [1, 3, 5])
    s.compact(dllm)
    src, dst = rng.permutation(60)[:23], rng.permutation(31)[:23]
    src[3], dst[5] = -1, -1
    parked = [rng.integers(0, 256, (31, *a)).astype(np.uint8) for a in arrays]
    g = [torch.from_numpy(a.copy()).to(s.dev) for a in parked]
    dllm.page_copy(s.g_pools, g, s.rows(src), s.rows(dst))
    for k, a in enumerate(parked):
        for x, y in zip(src, dst):
            if x >= 0 and y >= 0:
                a[y] = s.pools[k][x]
        np.testing.assert_array_equal(g[k].cpu().numpy(), a)
    assert dllm.get_device_error(s.dev) == 0


def test_pools_that_run_out(dllm):
    """Too few free pages: entries in their order as far as they last; what is not served holds nothing."""
    rng = np.random.default_rng(8)
    s = State(rng, 12, 4, 10, 16, [40, 16, 33, 20], spare_rows=6)   # 9 pages taken
    s.fork(dllm, [0, 1, 2, 3, 0, 1], [4, 5, 6, 7, 8, 9])            # 0, 2 and 3 take a page; the last 0 finds none
    s.grow(dllm, [1, 0], 1)                                         # nothing is left
    s.free(dllm, [2])
    s.grow(dllm, [3, 1, 0], 32)
    s.grow(dllm, [0], 1000)                                         # beyond the table
    s.compact(dllm)


def test_rows_and_pages_outside(dllm):
    """Row and page numbers that are none are recorded, and touch nothing."""
    rng = np.random.default_rng(9)
    s = State(rng, 40, 4, 10, 16, [40, 16, 33, 20], spare_rows=3)
    s.fork(dllm, [0, -1, 99, 1], [4, 5, 6, 2 ** 31 - 1])
    s.grow(dllm, [-1, 0, 7], 40)
    s.free(dllm, [-5, 1, 7])
    s.free(dllm, [1, 1])                 # nothing is held any more
    s.free(dllm, [0, 0])                 # twice in one call: once
    for entry in (-1, 40, 2 ** 31 - 1):
        s = State(rng, 40, 4, 10, 16, [40, 16, 33, 20], spare_rows=3)
        s.g_table[0, 0] = entry
        before = [p.clone() for p in s.g_pools]
        dllm.page_free(s.g_refs, s.g_table, s.g_held, s.rows([0]))
        assert dllm.get_device_error(s.dev) == 5
        dllm.page_compact(s.g_pools, s.g_refs, s.g_table, s.g_held)
        dllm.get_device_error(s.dev)
        s.g_table[2, 2] = entry          # the page that a fork would copy
        fresh = dllm.page_fork(s.g_pools, s.g_refs, s.g_table, s.g_held, s.g_lens, s.rows([2]), s.rows([4]), page_size=16)
        assert fresh.tolist() == [-2] and dllm.get_device_error(s.dev) == 5
        assert int(s.g_held[4]) == 0
        dllm.page_copy(before, s.g_pools, s.rows([entry if entry != -1 else 40, 3]), s.rows([1, 3]))
        assert dllm.get_device_error(s.dev) == 5
        assert (s.g_pools[0][3] == before[0][3]).all()


def test_lengths_that_pages_do_not_reach(dllm):
    """lens beyond the held pages, and negative: recorded, and cut to what is there."""
    rng = np.random.default_rng(10)
    s = State(rng, 40, 3, 10, 16, [40, 16, 33], spare_rows=3)
    s.g_lens[0], s.g_lens[1] = 1000, -3
    fresh = dllm.page_fork(s.g_pools, s.g_refs, s.g_table, s.g_held, s.g_lens, s.rows([0, 1]), s.rows([3, 4]), page_size=16)
    assert dllm.get_device_error(s.dev) == 5
    assert fresh.tolist() == [-1, -1] and s.g_lens[3:5].tolist() == [48, 0] and s.g_held[3:5].tolist() == [3, 0]


def test_captured_and_on_other_streams(dllm):
    """Fork, growth, release and compaction replay in a graph; another stream gives the same."""
    import torch
    rng = np.random.default_rng(11)
    s = State(rng, 500, 6, 20, 16, [100, 30, 16, 1, 0, 77], spare_rows=4)
    src, dst = s.rows([0, 1, 5, 0]), s.rows([6, 7, 8, 9])

    def turn():
        a = dllm.page_fork(s.g_pools, s.g_refs, s.g_table, s.g_held, s.g_lens, src, dst, page_size=16)
        b = dllm.page_grow(s.g_refs, s.g_table, s.g_held, s.g_lens, dst, 20, page_size=16)
        c = s.g_table.clone(), s.g_refs.clone()
        dllm.page_free(s.g_refs, s.g_table, s.g_held, dst)
        return a, b, *c
    want = [t.clone() for t in turn()]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = turn()
    for _ in range(3):
        g.replay()
        turn()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = turn()
    torch.cuda.synchronize()
    for a, b in zip(again, want):
        assert torch.equal(a, b)
    assert dllm.get_device_error(s.dev) == 0


def test_refusals(dllm):
    import torch
    rng = np.random.default_rng(12)
    s = State(rng, 40, 3, 10, 16, [40, 16, 33], spare_rows=3)
    one = s.rows([0])
    batch = (s.g_refs, s.g_table, s.g_held)
    with pytest.raises(ValueError):
        dllm.page_fork(s.g_pools, *batch, s.g_lens, one, s.rows([3, 4]), page_size=16)
    with pytest.raises(ValueError):
        dllm.page_copy(s.g_pools, s.g_pools[:1], one, one)
    with pytest.raises(dllm.DllmError):
        dllm.page_fork([s.g_pools[0][:20]], *batch, s.g_lens, one, s.rows([3]), page_size=16)
    with pytest.raises(dllm.DllmError):
        dllm.page_fork(s.g_pools, *batch, s.g_lens, one, s.rows([3]), page_size=0)
    with pytest.raises(TypeError):
        dllm.page_free(s.g_refs.long(), s.g_table, s.g_held, one)
    with pytest.raises(TypeError):
        dllm.page_free(*batch, one.float())
    with pytest.raises(ValueError):
        dllm.page_free(s.g_refs.cpu(), s.g_table, s.g_held, one)
    with pytest.raises(ValueError):
        dllm.page_compact([s.g_pools[0][:, ::2]], *batch)
    with pytest.raises(dllm.DllmError):
        dllm.page_compact([torch.zeros(40, 8, dtype=torch.uint8, device=s.dev)], *batch)
    with pytest.raises(ValueError):
        dllm.page_compact(s.g_pools * 33, *batch)
    s.same(dllm)
