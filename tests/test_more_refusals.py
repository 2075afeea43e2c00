"""dllm_sample, dllm_pages_* and dllm_fp8_* without a GPU: what their host side refuses, and with which code, before any
CUDA call; sizes; empty calls; the references of their GPU tests by hand."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest

import denoise_step_token_gb300 as dllm
import pages_reference
import sample_reference
from denoise_step_token_gb300 import _build

INVAL, ALIGN, CUDA, WORKSPACE, UNSUPPORTED = -1, -2, -3, -5, -6


def sample_args(**kw):
    base = dict(N=2, V=16, ldv=16, logits_rows=2, logits=0x10000, u=0x20000, tokens=0x30000, prob=0x40000)
    base.update(kw)
    return dllm.SampleArgs(**base)


@pytest.mark.parametrize("kw,code", [({"N": -1}, INVAL), ({"V": 0}, INVAL), ({"ldv": 15}, INVAL), ({"logits_rows": -1}, INVAL),
                                     ({"logits": None}, INVAL), ({"u": None}, INVAL), ({"tokens": None}, INVAL),
                                     ({"prob": None}, INVAL), ({"logits": 0x10008}, ALIGN), ({"ldv": 20}, ALIGN),
                                     ({"V": (1 << 28) + 8, "ldv": 1 << 29}, UNSUPPORTED)])
def test_sample_refusals(kw, code):
    assert dllm.load().dllm_sample(ctypes.byref(sample_args(**kw)), None) == code


def batch(**kw):
    base = dict(n_pages=8, B=2, max_pages=4, page_size=16, refs=0x10000, table=0x20000, held=0x30000)
    base.update(kw)
    return dllm.PagesBatch(**base)


def pool(n_pages=8, arrays=((0x100000, 64), (0x200000, 16))):
    p = dllm.PagesPool(n_pages, len(arrays))
    for k, (at, size) in enumerate(arrays):
        p.arrays[k], p.page_bytes[k] = at, size
    return p


def page_calls(b, p, ws=0x400000, size=1 << 20):
    """Every call that takes a batch: (with a pool?, its status)."""
    lib = dllm.load()
    b, p = ctypes.byref(b), ctypes.byref(p)
    return [(True, lambda: lib.dllm_pages_fork(b, p, 0x50000, 1, 0x60000, 0x70000, 0x80000, ws, size, None)),
            (False, lambda: lib.dllm_pages_grow(b, 0x50000, 1, 0x60000, 1, 0x80000, ws, size, None)),
            (False, lambda: lib.dllm_pages_free(b, 1, 0x60000, None)),
            (True, lambda: lib.dllm_pages_compact(b, p, 0x60000, 0x70000, ws, size, None))]


@pytest.mark.parametrize("kw,code", [({"n_pages": 0}, INVAL), ({"B": -1}, INVAL), ({"max_pages": 0}, INVAL),
                                     ({"page_size": 0}, INVAL), ({"refs": None}, INVAL), ({"table": None}, INVAL),
                                     ({"held": None}, INVAL), ({"refs": 0x10004}, ALIGN),
                                     ({"max_pages": (1 << 20) + 1}, UNSUPPORTED)])
def test_page_batches_are_checked_by_every_call(kw, code):
    for _, call in page_calls(batch(**kw), pool(kw.get("n_pages") or 8)):
        assert call() == code


@pytest.mark.parametrize("p,code", [(pool(0), INVAL), (pool(9), INVAL), (pool(8, ((None, 16),)), INVAL), (pool(8, ((0x1000, 0),)), INVAL),
                                    (pool(8, ((0x1008, 16),)), ALIGN), (pool(8, ((0x1000, 24),)), ALIGN),
                                    (pool(8, ((0x1000, 1 << 33),)), UNSUPPORTED)])
def test_page_pools_are_checked(p, code):
    lib = dllm.load()
    for takes, call in page_calls(batch(), p):
        if takes:
            assert call() == code
    if p.n_pages != 9:   # copies go between pools of any sizes
        assert lib.dllm_pages_copy(ctypes.byref(p), ctypes.byref(pool()), 1, 0x60000, 0x70000, None) == code
        assert lib.dllm_pages_copy(ctypes.byref(pool()), ctypes.byref(p), 1, 0x60000, 0x70000, None) == code


def test_page_workspaces_and_arguments():
    lib = dllm.load()
    size = lib.dllm_pages_workspace_size
    assert size(0, 1) == size(5, -1) == 0 and size(100, 7) > size(100, 0) > 0 and size(101, 0) > size(100, 0)
    for ws, n in ((None, 1 << 20), (0x400000, 16), (0x400004, 1 << 20)):
        calls = page_calls(batch(), pool(), ws, n)
        assert [call() for _, call in calls[:2] + calls[3:]] == [WORKSPACE] * 3
    b, p, other = ctypes.byref(batch()), ctypes.byref(pool()), ctypes.byref(pool(8, ((0x100000, 64),)))
    assert lib.dllm_pages_copy(p, other, 1, 0x60000, 0x70000, None) == INVAL
    assert lib.dllm_pages_copy(p, p, -1, 0x60000, 0x70000, None) == INVAL
    assert lib.dllm_pages_copy(p, p, 1, None, 0x70000, None) == INVAL
    assert lib.dllm_pages_copy(None, p, 1, 0x60000, 0x70000, None) == INVAL
    assert lib.dllm_pages_grow(b, 0x50000, 1, 0x60000, -1, 0x80000, 0x400000, 1 << 20, None) == INVAL
    assert lib.dllm_pages_free(b, 1, None, None) == INVAL
    assert lib.dllm_pages_compact(b, p, None, 0x70000, 0x400000, 1 << 20, None) == INVAL
    # nothing to do
    assert lib.dllm_pages_copy(p, p, 0, None, None, None) == 0
    assert lib.dllm_pages_fork(b, p, 0x50000, 0, None, None, None, None, 0, None) == 0
    assert lib.dllm_pages_grow(b, None, 0, None, 1, None, None, 0, None) == 0
    assert lib.dllm_pages_free(b, 0, None, None) == 0


def quantize_args(**kw):
    base = dict(M=2, K=128, block_rows=1, x_rows=2, ldx=128, x=0x10000, codes=0x20000, scale=0x30000)
    base.update(kw)
    return dllm.Fp8QuantizeArgs(**base)


@pytest.mark.parametrize("kw,code", [({"M": -1}, INVAL), ({"K": 0}, INVAL), ({"x_rows": -1}, INVAL), ({"ldx": 120}, INVAL),
                                     ({"block_rows": 2}, INVAL), ({"x": None}, INVAL), ({"codes": None}, INVAL),
                                     ({"scale": None}, INVAL), ({"K": 120}, ALIGN), ({"ldx": 132}, ALIGN),
                                     ({"x": 0x10002}, ALIGN), ({"codes": 0x20004}, ALIGN),
                                     ({"K": (1 << 24) + 16, "ldx": 1 << 25}, UNSUPPORTED),
                                     ({"M": 65536 * 128}, UNSUPPORTED)])
def test_quantize_refusals(kw, code):
    assert dllm.load().dllm_fp8_quantize(ctypes.byref(quantize_args(**kw)), None) == code


def matmul_args(**kw):
    base = dict(M=2, N=10, K=128, lda=128, ldb=128, ldo=16, a=0x10000, a_scale=0x20000, b=0x30000, b_scale=0x40000, out=0x50000)
    base.update(kw)
    return dllm.Fp8MatmulArgs(**base)


@pytest.mark.parametrize("kw,code", [({"M": -1}, INVAL), ({"N": 0}, INVAL), ({"K": 0}, INVAL), ({"lda": 127}, INVAL),
                                     ({"ldb": 112}, INVAL), ({"ldo": 8}, INVAL), ({"a": None}, INVAL), ({"b": None}, INVAL),
                                     ({"a_scale": None}, INVAL), ({"b_scale": None}, INVAL), ({"out": None}, INVAL),
                                     ({"a": 0x10008}, ALIGN), ({"b": 0x30001}, ALIGN), ({"out": 0x50002}, ALIGN),
                                     ({"K": 120}, ALIGN), ({"lda": 136}, ALIGN), ({"ldo": 20}, ALIGN),
                                     ({"N": (1 << 28) + 1, "ldo": 1 << 29}, UNSUPPORTED)])
def test_matmul_refusals(kw, code):
    assert dllm.load().dllm_fp8_matmul(ctypes.byref(matmul_args(**kw)), None) == code


def test_null_arguments_empty_calls_and_sizes():
    lib = dllm.load()
    for fn in (lib.dllm_sample, lib.dllm_fp8_quantize, lib.dllm_fp8_matmul):
        assert fn(None, None) == INVAL
    assert lib.dllm_sample(ctypes.byref(sample_args(N=0, u=None)), None) == 0
    assert lib.dllm_fp8_quantize(ctypes.byref(quantize_args(M=0)), None) == 0
    assert lib.dllm_fp8_matmul(ctypes.byref(matmul_args(M=0)), None) == 0
    for which, cls in ((14, dllm.SampleArgs), (15, dllm.PagesPool), (16, dllm.PagesBatch), (17, dllm.Fp8QuantizeArgs),
                       (18, dllm.Fp8MatmulArgs)):
        assert lib.dllm_struct_size(which) == ctypes.sizeof(cls)


def test_product_kernel_has_the_registers_it_shares_out(tmp_path):
    """fp8_matmul_kernel shares out 96 registers per thread between its warps, and its launch refuses any other number."""
    src = os.path.join(_build.CSRC, "fp8.cu")
    run = subprocess.run([_build.nvcc_path(), *_build.ARCH_FLAGS, *_build.NVCC_FLAGS, "-Xptxas", "-v", "-c", src, "-o",
                          str(tmp_path / "fp8.o")], capture_output=True, text=True, check=True)
    found = re.findall(r"Compiling entry function '\S*?fp8_matmul_kernel\S*'.*?Used (\d+) registers", run.stdout + run.stderr,
                       re.S)
    assert found == ["96"]


# ---------------------------------------------------------------------------
# the references themselves
# ---------------------------------------------------------------------------
def test_sample_reference_by_hand():
    x = np.log(np.array([1.0, 4.0, 2.0, 1.0]))   # in order: tokens 1, 2, 0, 3 of mass 4, 2, 1, 1
    draw = lambda u, **kw: sample_reference.sample(x, u, **kw)[:2]  # noqa: E731
    for u, tok, p in ((0.0, 1, 0.5), (0.49, 1, 0.5), (0.51, 2, 0.25), (0.8, 0, 0.125), (0.99, 3, 0.125), (1.0, 3, 0.125)):
        t, q = draw(u)
        assert t == tok and abs(q - p) < 1e-12
    assert draw(0.99, top_k=2)[0] == 2 and abs(draw(0.99, top_k=2)[1] - 1 / 3) < 1e-12
    assert draw(0.99, top_p=0.6)[0] == 2 and draw(0.99, top_p=0.4)[0] == 1 and draw(0.99, top_p=0.0)[0] == 1
    assert draw(0.99, min_p=0.4)[0] == 2 and draw(0.99, min_p=0.2)[0] == 3
    assert draw(0.99, top_k=3, top_p=0.9)[0] == 0       # 0.9 of 7, not of 8
    assert draw(0.99, T=0.0) == (1, 1.0)
    assert abs(draw(0.0, T=0.5)[1] - 16 / 22) < 1e-12   # 16, 4, 1, 1
    for bad in ([np.nan, 1.0], [np.inf, 1.0], [-np.inf, -np.inf]):
        assert sample_reference.sample(bad, 0.5)[0] == -1
    assert sample_reference.sample([0.0, -0.0, 0.0], 0.5)[0] == 1


def test_pages_reference_by_hand():
    table, held, lens = np.zeros((3, 4), dtype=np.int64), np.zeros(3, dtype=np.int64), np.zeros(3, dtype=np.int64)
    refs = np.zeros(6, dtype=np.int64)
    x = np.arange(6)
    table[0, :2], held[0], lens[0], refs[[4, 1]] = [4, 1], 2, 5, 1
    assert pages_reference.fork([x], refs, table, held, lens, [0, 0], [1, 2], 4) == ([0, 2], False)
    assert table[1, :2].tolist() == [4, 0] and refs.tolist() == [1, 1, 1, 0, 3, 0] and x[[0, 2]].tolist() == [1, 1]
    assert pages_reference.grow(refs, table, held, lens, [2, 1], 4, 4) == ([1, 1], False)
    assert table[2, :3].tolist() == [4, 2, 3] and table[1, 2] == 5
    assert pages_reference.grow(refs, table, held, lens, [0], 8, 4) == ([-1], True)
    assert not pages_reference.release(refs, table, held, [1])
    assert refs.tolist() == [0, 1, 1, 1, 2, 0]
    U, new = pages_reference.compact([x], refs, table, held)
    assert U == 4 and new.tolist() == [-1, 1, 2, 3, 0, -1] and table[0, :2].tolist() == [0, 1] and refs.tolist() == [2, 1, 1, 1, 0, 0]
