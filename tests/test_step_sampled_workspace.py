"""step_sampled on the CPU: which memory a call gets as its workspace, who else may be using it, and what is refused.

The library is replaced by one that records the workspace each call is given, and the checks that ask for a CUDA device
are taken out."""
import ctypes
from types import SimpleNamespace

import pytest
import torch

import denoise_step_token_gb300 as pkg

NEED = 20000


@pytest.fixture
def fake(monkeypatch):
    state = SimpleNamespace(given=[], stream=7, capturing=False)

    def call(ref, *rest):
        args = ref._obj
        raw = (ctypes.c_uint8 * args.workspace_bytes).from_address(args.workspace)
        state.given.append((args.workspace, args.workspace_bytes, not any(raw[:NEED])))
        return 0

    lib = SimpleNamespace(dllm_step_merge=call, dllm_step_drawn=call, dllm_step_workspace_size=lambda *a: NEED)
    monkeypatch.setattr(pkg, "_lib", lib)
    monkeypatch.setattr(pkg, "_require_cuda", lambda *a: torch.device("cpu"))
    monkeypatch.setattr(pkg, "_check_tensors", lambda *a: None)
    monkeypatch.setattr(pkg, "_raw_stream", lambda *a: state.stream)
    monkeypatch.setattr(pkg, "_stream", lambda *a: ctypes.c_void_p(state.stream))
    monkeypatch.setattr(pkg, "_step_ws", pkg._Workspaces())
    monkeypatch.setattr(pkg, "_stream_ws", {})
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: state.capturing)
    monkeypatch.setattr(pkg, "_drawn_ws", {})
    return state


def step(**kw):
    B, L = 2, 4
    return pkg.step_sampled(torch.zeros(B * L, dtype=torch.int32), torch.ones(B * L), torch.zeros(B, L, dtype=torch.int32),
                            torch.zeros(B), torch.zeros(B, L), V=50, mask_id=50, **kw)


def test_every_stream_has_its_own(fake):
    step()
    step()
    fake.stream = 8
    step()
    (a, n, zero), (b, *_), (c, _, clear) = fake.given
    assert a == b != c and n >= NEED and zero and clear


def test_none_of_it_is_the_step_s(fake):
    step()
    assert fake.given[0][0] != pkg._step_ws.get(torch.device("cpu"), NEED).data_ptr()
    assert not pkg._stream_ws                      # nor that of the operators that clear their counters alone


def test_a_graph_has_its_own_cleared(fake, monkeypatch):
    empty, held = torch.empty, []   # kept, so that addresses are not used again; as dirty as memory may be
    monkeypatch.setattr(torch, "empty", lambda *a, **k: held.append(empty(*a, **k).fill_(1)) or held[-1])
    fake.capturing = True
    step()
    fake.capturing = False
    step()
    (a, n, zero), (b, *_) = fake.given
    assert a != b and zero and n >= NEED
    assert [w.buf.data_ptr() for w in pkg._drawn_ws.values()] == [b]


def test_a_caller_s_own(fake):
    own = torch.zeros(30000, dtype=torch.uint8)
    step(workspace=own)
    assert fake.given[0][:2] == (own.data_ptr(), 30000) and not pkg._drawn_ws
    for bad in (own.int(), own[::2]):
        with pytest.raises(ValueError):
            step(workspace=bad)


@pytest.mark.parametrize("kw,code", [({"B": -1}, -1), ({"L": 0}, -1), ({"L": 1025}, -1), ({"V": 0}, -1), ({"input_ids": None}, -1),
                                     ({"conf_state": None}, -1), ({"done": None}, -1), ({"thr": None}, -1),
                                     ({"tokens": None}, -1), ({"conf": None}, -1), ({"workspace": None}, -5),
                                     ({"workspace": 0x80010}, -5), ({"workspace_bytes": 64}, -5), ({"B": 1 << 16}, -6),
                                     ({"B": 0, "tokens": None, "workspace": None}, 0)])
def test_refusals(kw, code):
    lib = pkg.load()
    base = dict(B=2, L=4, V=50, mask_id=50, ldv=56, input_ids=0x10000, thr=0x20000, conf_state=0x30000, done=0x40000,
                accept_len=0x50000, n_new=0x60000, workspace=0x80000, workspace_bytes=1 << 20, tokens=0x1000, conf=0x2000)
    base.update(kw)
    tokens, conf = base.pop("tokens"), base.pop("conf")
    assert lib.dllm_step_drawn(ctypes.byref(pkg.StepArgs(**base)), tokens, conf, None, None) == code
    if "thr" in kw:
        base["workspace"] = None      # with a quota the threshold may be absent: refused for its workspace instead
        assert lib.dllm_step_drawn(ctypes.byref(pkg.StepArgs(**base)), tokens, conf, 0x3000, None) == -5
    assert lib.dllm_step_drawn(None, tokens, conf, None, None) == -1


def test_sample_conf_refusals():
    lib = pkg.load()
    a = pkg.SampleArgs(N=2, V=16, ldv=16, logits_rows=2, logits=0x10000, u=0x20000, tokens=0x30000, prob=0x40000)
    assert lib.dllm_sample_conf(ctypes.byref(a), None, None) == -1
    assert lib.dllm_sample_conf(None, 0x50000, None) == -1
    a.ldv = 20
    assert lib.dllm_sample_conf(ctypes.byref(a), 0x50000, None) == -2
    a.N, a.ldv = 0, 16
    assert lib.dllm_sample_conf(ctypes.byref(a), None, None) == 0
