"""The default workspace of token_logprobs and kv4_attend, on the CPU.

The library is replaced by one that records the workspace each call is given,
and the checks that ask for a CUDA device are taken out: what is tested is which
memory a call gets, and who else may be using it."""
import ctypes
import threading
import time
from types import SimpleNamespace

import pytest
import torch

import denoise_step_token_gb300 as pkg


@pytest.fixture
def fake(monkeypatch):
    """Records (entry, workspace) and (exit, workspace) of every call, in order."""
    log = []
    state = SimpleNamespace(log=log, hold=0.0, seen=None)

    def call(ref, stream):
        args = ref._obj
        log.append(("in", args.workspace))
        if state.seen is not None:
            state.seen(args)
        time.sleep(state.hold)
        log.append(("out", args.workspace))
        return 0

    lib = SimpleNamespace(dllm_logprobs=call, dllm_kv4_attend=call, dllm_logprobs_workspace_size=lambda *a: 5000,
                          dllm_kv4_attend_workspace_size=lambda *a: 9000)
    monkeypatch.setattr(pkg, "_lib", lib)
    monkeypatch.setattr(pkg, "_check_tensors", lambda *a: None)
    monkeypatch.setattr(pkg, "_raw_stream", lambda *a: 7)
    monkeypatch.setattr(pkg, "_stream_ws", {})
    monkeypatch.setattr(pkg, "_size_cache", {})
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    return state


def attend():
    q = torch.zeros(1, 40, 2, 64, dtype=torch.bfloat16)
    pages = torch.zeros(2, 1, 16 * 72, dtype=torch.uint8)
    return pkg.kv4_attend(q, pages, torch.zeros(1, 2, dtype=torch.int32), torch.ones(1, dtype=torch.int32))


def logprobs():
    return pkg.token_logprobs(torch.zeros(2, 16), torch.zeros(2, dtype=torch.int32))


def test_threads_on_one_stream_do_not_share_a_workspace_in_use(fake):
    """A call's launches share one workspace; a call of another thread on the
    same stream must not come between them with the same one."""
    fake.hold = 0.005
    threads = [threading.Thread(target=f) for f in (attend, logprobs) * 4]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    in_use = set()
    for what, ws in fake.log:
        if what == "in":
            assert ws not in in_use
            in_use.add(ws)
        else:
            in_use.remove(ws)
    assert len(fake.log) == 16


def test_one_workspace_a_stream_grown_on_demand(fake):
    logprobs()
    attend()
    logprobs()
    assert len({ws for _, ws in fake.log}) == 1   # both fit the first one


def test_captured_calls_keep_to_their_graph(fake, monkeypatch):
    """A graph replays with the memory that its capture saw.  So a captured call
    leaves none for later calls, takes none of theirs, and clears its join
    counters within the graph."""
    zeroed = []

    def seen(args):
        raw = (ctypes.c_uint8 * args.workspace_bytes).from_address(args.workspace)
        zeroed.append(not any(raw[:8192]))
        raw[:8192] = b"\1" * 8192   # as if left by whatever ran before a replay
    fake.seen = seen
    before = attend() and fake.log[-1][1]
    kept = torch.empty(0)
    held = [kept]   # what the captured calls allocated, so that addresses cannot be used again
    empty, zeros = torch.empty, torch.zeros
    monkeypatch.setattr(torch, "empty", lambda *a, **k: held.append(empty(*a, **k)) or held[-1])
    monkeypatch.setattr(torch, "zeros", lambda *a, **k: held.append(zeros(*a, **k)) or held[-1])
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    first = attend() and fake.log[-1][1]
    second = logprobs() and fake.log[-1][1]
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    fake.seen = None
    after = attend() and fake.log[-1][1]
    assert len({before, first, second}) == 3
    assert after == before
    assert zeroed == [True] * 3


def test_refused_workspaces(fake):
    """Memory that a kernel cannot use as its workspace never reaches the
    library: another device's, of another type, or in pieces."""
    logits, tokens = torch.zeros(2, 16), torch.zeros(2, dtype=torch.int32)
    pkg.token_logprobs(logits, tokens, workspace=torch.zeros(9000, dtype=torch.uint8))
    assert len(fake.log) == 2
    for bad in (torch.zeros(9000, dtype=torch.uint8, device="meta"), torch.zeros(9000),
                torch.zeros(18000, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError):
            pkg.token_logprobs(logits, tokens, workspace=bad)
    assert len(fake.log) == 2


@pytest.mark.parametrize("D", [64, 128])
def test_attention_workspace_follows_the_batch(D):
    """A token's call asks for what its units (16 rows of a request's head) can
    be cut into, 64 pieces each and 4096 in all; a smaller batch never for more."""
    size = lambda B, heads, L, q_heads: int(pkg.load().dllm_kv4_attend_workspace_size(  # noqa: E731
        ctypes.byref(pkg.Kv4Cache(9, heads, 32, D, B, 7, None, None)), L, q_heads))
    piece = 16 * (D + 2) * 4
    assert size(1, 1, 1, 1) == 8192 + 64 * piece
    assert size(0, 1, 1, 8) == size(1, 1, 1, 8) == 8192 + 64 * piece
    assert size(3, 2, 5, 8) == 8192 + 3 * 2 * 2 * 64 * piece
    assert size(64, 8, 1, 8) == size(4096, 8, 1, 8) == 8192 + 4096 * piece
    for heads, group in ((1, 1), (4, 7)):
        by_batch = [size(B, heads, 1, heads * group) for B in (1, 2, 15, 16, 17, 200, 5000)]
        by_rows = [size(6, heads, L, heads * group) for L in (1, 2, 4, 5, 32, 100, 1024)]
        assert by_batch == sorted(by_batch) and by_rows == sorted(by_rows)
