"""dllm_logprobs and dllm_kv4_* without a GPU: what their host side refuses,
and with which code, before any CUDA call; sizes; empty calls."""
import ctypes

import numpy as np
import pytest

import denoise_step_token_gb300 as dllm
import kv4_reference as ref

INVAL, ALIGN, WORKSPACE, UNSUPPORTED = -1, -2, -5, -6


def cache(**kw):
    base = dict(n_pages=8, heads=2, page_size=16, head_dim=128, B=2, max_pages=4, pages=0x10000, table=0x20000)
    base.update(kw)
    return dllm.Kv4Cache(**base)


CACHE_ERRORS = [({"n_pages": 0}, INVAL), ({"heads": 0}, INVAL), ({"B": -1}, INVAL), ({"max_pages": 0}, INVAL),
                ({"page_size": 8}, UNSUPPORTED), ({"page_size": 48}, UNSUPPORTED), ({"page_size": 512}, UNSUPPORTED),
                ({"head_dim": 96}, UNSUPPORTED), ({"B": 65536}, UNSUPPORTED), ({"heads": 4097}, UNSUPPORTED),
                ({"page_size": 256, "max_pages": 1 << 23}, UNSUPPORTED), ({"pages": None}, INVAL),
                ({"table": None}, INVAL), ({"pages": 0x10008}, ALIGN)]


def write_args(c=None, **kw):
    base = dict(cache=cache() if c is None else c, W=4, k=0x30000, v=0x40000, k_stride=(ctypes.c_int64 * 3)(1024, 256, 128),
                v_stride=(ctypes.c_int64 * 3)(1024, 256, 128), pos=0x50000)
    base.update(kw)
    return dllm.Kv4WriteArgs(**base)


def attend_args(c=None, **kw):
    base = dict(cache=cache() if c is None else c, L=2, q_heads=4, scale=0.1, q=0x30000,
                q_stride=(ctypes.c_int64 * 3)(1024, 512, 128), lens=0x40000, out=0x50000, lse=0x60000,
                workspace=0x100000, workspace_bytes=1 << 30)
    base.update(kw)
    return dllm.Kv4AttendArgs(**base)


def evict_args(c=None, **kw):
    base = dict(cache=cache() if c is None else c, recent=0, dst_max_pages=2, lens=0x30000, keep=0x40000, weights=0x50000,
                dst_table=0x60000, dst_lens=0x70000, src=0x80000)
    base.update(kw)
    return dllm.Kv4EvictArgs(**base)


def logprob_args(**kw):
    base = dict(N=2, V=16, top=2, dtype=0, ldv=16, logits_rows=2, logits=0x10000, tokens=0x20000, logprob=0x30000,
                entropy=0x40000, top_ids=0x50000, top_logprobs=0x60000, workspace=0x100000, workspace_bytes=1 << 30)
    base.update(kw)
    return dllm.LogprobsArgs(**base)


@pytest.mark.parametrize("kw,code", CACHE_ERRORS)
def test_cache_is_checked_by_every_call(kw, code):
    lib = dllm.load()
    for args, fn in ((write_args, lib.dllm_kv4_write), (attend_args, lib.dllm_kv4_attend), (evict_args, lib.dllm_kv4_evict)):
        assert fn(ctypes.byref(args(cache(**kw))), None) == code


def strides(*s):
    return (ctypes.c_int64 * 3)(*s)


@pytest.mark.parametrize("kw,code", [({"W": -1}, INVAL), ({"k": None}, INVAL), ({"v": None}, INVAL), ({"pos": None}, INVAL),
                                     ({"k": 0x30002}, ALIGN), ({"v_out": 0x30004}, ALIGN),
                                     ({"v_stride": strides(1024, 257, 128)}, ALIGN)])
def test_write_refusals(kw, code):
    assert dllm.load().dllm_kv4_write(ctypes.byref(write_args(**kw)), None) == code


@pytest.mark.parametrize("kw,code", [({"L": 0}, INVAL), ({"L": 1025}, INVAL), ({"q_heads": 3}, INVAL), ({"q_heads": 0}, INVAL),
                                     ({"L": 1024, "q_heads": 2048}, UNSUPPORTED), ({"scale": float("inf")}, INVAL),
                                     ({"q": None}, INVAL), ({"lens": None}, INVAL), ({"out": None}, INVAL),
                                     ({"lse": None, "weights": 0x70000}, INVAL), ({"prior": 0x70000}, INVAL),
                                     ({"q": 0x30008}, ALIGN), ({"out": 0x50002}, ALIGN),
                                     ({"q_stride": strides(1024, 512, 100)}, ALIGN), ({"workspace": None}, WORKSPACE),
                                     ({"workspace": 0x100080}, WORKSPACE), ({"workspace_bytes": 4096}, WORKSPACE)])
def test_attend_refusals(kw, code):
    assert dllm.load().dllm_kv4_attend(ctypes.byref(attend_args(**kw)), None) == code


@pytest.mark.parametrize("kw,code", [({"recent": -1}, INVAL), ({"dst_max_pages": 0}, INVAL),
                                     ({"dst_max_pages": 1 << 28}, UNSUPPORTED), ({"lens": None}, INVAL), ({"keep": None}, INVAL),
                                     ({"weights": None}, INVAL), ({"dst_table": None}, INVAL), ({"dst_lens": None}, INVAL),
                                     ({"src": None}, INVAL)])
def test_evict_refusals(kw, code):
    assert dllm.load().dllm_kv4_evict(ctypes.byref(evict_args(**kw)), None) == code


@pytest.mark.parametrize("kw,code", [({"N": -1}, INVAL), ({"V": 0}, INVAL), ({"top": -1}, INVAL), ({"top": 33}, INVAL),
                                     ({"dtype": 2}, INVAL), ({"ldv": 15}, INVAL), ({"logits": None}, INVAL),
                                     ({"logits_rows": -1}, INVAL), ({"tokens": None}, INVAL), ({"logprob": None}, INVAL),
                                     ({"top_ids": None}, INVAL), ({"top_logprobs": None}, INVAL), ({"logits": 0x10008}, ALIGN),
                                     ({"ldv": 20}, ALIGN), ({"ldv": 18, "dtype": 1}, ALIGN), ({"workspace": None}, WORKSPACE),
                                     ({"workspace_bytes": 64}, WORKSPACE), ({"workspace": 0x100010}, WORKSPACE)])
def test_logprobs_refusals(kw, code):
    assert dllm.load().dllm_logprobs(ctypes.byref(logprob_args(**kw)), None) == code


def test_null_arguments_and_empty_calls():
    lib = dllm.load()
    for fn in (lib.dllm_logprobs, lib.dllm_kv4_write, lib.dllm_kv4_attend, lib.dllm_kv4_evict):
        assert fn(None, None) == INVAL
    assert lib.dllm_logprobs(ctypes.byref(logprob_args(N=0)), None) == 0
    none = cache(B=0, table=None)
    assert lib.dllm_kv4_write(ctypes.byref(write_args(none)), None) == 0
    assert lib.dllm_kv4_write(ctypes.byref(write_args(W=0)), None) == 0
    assert lib.dllm_kv4_attend(ctypes.byref(attend_args(none)), None) == 0
    assert lib.dllm_kv4_evict(ctypes.byref(evict_args(none)), None) == 0


def test_sizes():
    lib = dllm.load()
    for page in (16, 32, 64, 128, 256):
        for D in (64, 128):
            assert lib.dllm_kv4_page_bytes(page, D) == page * (D + D // 8)
    for page, D in ((0, 64), (24, 64), (512, 64), (16, 32), (16, 256)):
        assert lib.dllm_kv4_page_bytes(page, D) == 0
    assert lib.dllm_logprobs_workspace_size(1, 16, 32) > 0
    assert lib.dllm_logprobs_workspace_size(-1, 16, 1) == lib.dllm_logprobs_workspace_size(1, 0, 1) == 0
    assert lib.dllm_logprobs_workspace_size(1, 16, 33) == 0
    c = cache()
    assert lib.dllm_kv4_attend_workspace_size(ctypes.byref(c), 2, 4) > 0
    assert lib.dllm_kv4_attend_workspace_size(ctypes.byref(c), 2, 3) == 0
    for which, cls in ((9, dllm.LogprobsArgs), (10, dllm.Kv4Cache), (11, dllm.Kv4WriteArgs), (12, dllm.Kv4AttendArgs),
                       (13, dllm.Kv4EvictArgs)):
        assert lib.dllm_struct_size(which) == ctypes.sizeof(cls)


# ---------------------------------------------------------------------------
# the 64-bit reference itself
# ---------------------------------------------------------------------------
def test_reference_quantiser_by_hand():
    x = np.zeros(32)
    x[:4] = [-7.0, 8.0, 0.4, 0.6]       # range 15: step 1, zero point 7
    u, step, z = ref.quantise(x)
    assert step[0] == 1.0 and z[0] == 7
    np.testing.assert_array_equal(ref.dequantise(u, step, z)[:5], [-7, 8, 0, 1, 0])
    x[1] = 8.5                          # 15.5 / 15 up to 4 significant bits
    assert ref.quantise(x)[1][0] == 1.125
    assert ref.quantise(np.full(32, 3.0))[2][0] == 0          # one sided: 0 stays a code
    assert ref.quantise(np.zeros(32))[1][0] == 2.0 ** -18


def test_reference_pages_round_trip():
    rng = np.random.default_rng(0)
    k, v = rng.standard_normal((2, 3, 2, 16, 64))
    a, b = ref.values_of(ref.pages_of(k, v, 16), 16, 64)
    np.testing.assert_array_equal(a, ref.dequantise(*ref.quantise(k)))
    np.testing.assert_array_equal(b, ref.dequantise(*ref.quantise(v)))
    # every value fits bf16 and fp16 exactly
    np.testing.assert_array_equal(ref.from_bf16(ref.to_bf16(a)), a)
    np.testing.assert_array_equal(a.astype(np.float16), a)


def test_reference_eviction_by_hand():
    w = np.array([5.0, 1.0, 5.0, np.nan, 2.0, 0.0])
    np.testing.assert_array_equal(ref.evict(w, 3, 1), [0, 2, 5])
    np.testing.assert_array_equal(ref.evict(w, 5, 0), [0, 1, 2, 4, 5])
    np.testing.assert_array_equal(ref.evict(w, 2, 9), [4, 5])
    np.testing.assert_array_equal(ref.evict(w, 0, 1), [])


def test_reference_attention_against_a_plain_loop():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((2, 4, 64)), rng.standard_normal((2, 5, 64)), rng.standard_normal((2, 5, 64))
    out, lse, w, _, _ = ref.attend(q, k, v, 0.5)
    for i in range(2):
        for h in range(4):
            e = [np.exp(0.5 * float(q[i, h] @ k[h // 2, j])) for j in range(5)]
            np.testing.assert_allclose(out[i, h], sum(e[j] * v[h // 2, j] for j in range(5)) / sum(e), rtol=1e-12)
            np.testing.assert_allclose(lse[i, h], np.log(sum(e)), rtol=1e-12)
    np.testing.assert_allclose(w.sum(-1), [4.0, 4.0], rtol=1e-12)   # each row gives 1 in all
