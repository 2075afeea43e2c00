"""dllm_fp8_quantize and dllm_fp8_matmul on the GPU.

Codes and scales are compared for equality with the definition in 32-bit
arithmetic (both quotients are correctly rounded on both sides).  The product
against 64 bits: the output's rounding to bf16, 2^-8 of the value at most (half
a step is 2^-9 relative to the leading power, 2^-8 to the value), and sums in 32 bits: a group's 128 products of
8 significant bits, then K / 128 scaled sums, each step within 2^-24 of the sum
of magnitudes, and allowing the tensor cores' own sums four times that:
(4 * 128 + K / 128 + 2) 2^-24 sum |a b|."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def dev():
    import torch
    return torch.device("cuda", 0)


def quantised(x, block_rows):
    """Codes (as values) and scales of float32 x by the definition, on the CPU."""
    import torch
    n, K = x.shape
    R, C = -(-n // block_rows), -(-K // 128)
    g = torch.zeros(R * block_rows, C * 128)
    g[:n, :K] = x
    g = g.reshape(R, block_rows, C, 128)
    top = g.abs().amax((1, 3), keepdim=True)
    bad = ~torch.isfinite(top) | torch.isnan(g).any(3, keepdim=True).any(1, keepdim=True)
    scale = torch.maximum(top / torch.tensor(448.0), torch.tensor(2.0 ** -126))
    q = (g / scale).clamp(-448, 448)
    q = torch.where(bad, torch.zeros(()), q).to(torch.float8_e4m3fn).float()
    scale = torch.where(bad, torch.tensor(float("nan")), scale)
    return q.reshape(R * block_rows, C * 128)[:n, :K], scale[:, 0, :, 0]


def same(a, b):
    np.testing.assert_array_equal(a.float().cpu().numpy(), b.float().cpu().numpy())


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("n,K", [(1, 16), (3, 128), (5, 144), (128, 256), (129, 2000), (300, 1040), (1000, 4096)])
def test_quantize(dllm, n, K, block_rows):
    import torch
    gen = torch.Generator().manual_seed(n + K)
    x = (torch.randn(n, K, generator=gen) * torch.exp(2 * torch.randn(n, 1, generator=gen))).to(torch.bfloat16)
    x[0] *= 1e30
    x[n // 2] *= 1e-30
    if n > 2:
        x[2] = 0
        x[1, K // 2] = -3.3895313892515355e38
    codes, scale = dllm.fp8_quantize(x.to(dev()), block_rows=block_rows)
    want = quantised(x.float(), block_rows)
    same(codes, want[0])
    same(scale, want[1])
    wide = torch.zeros(n, K + 24, dtype=torch.bfloat16)
    wide[:, 8:K + 8] = x
    rows = torch.tensor([n - 1, 0, -1, n, 0, n // 2, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    codes, scale = dllm.fp8_quantize(wide.to(dev())[:, 8:K + 8], rows=rows.to(dev()), block_rows=block_rows)
    picked = torch.zeros(8, K)
    for i, r in enumerate(rows.tolist()):
        if 0 <= r < n:
            picked[i] = x[r].float()
    want = quantised(picked, block_rows)
    same(codes, want[0])
    same(scale, want[1])
    assert dllm.get_device_error(dev()) == 0


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_every_value(dllm, block_rows):
    """All finite bf16 patterns, and groups that hold none of them finite."""
    import torch
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    x = bits.view(torch.bfloat16).reshape(512, 128).clone()
    x = x[torch.isfinite(x).all(1)]
    codes, scale = dllm.fp8_quantize(x.to(dev()), block_rows=block_rows)
    want = quantised(x.float(), block_rows)
    same(codes, want[0])
    same(scale, want[1])
    x = torch.randn(256, 256).to(torch.bfloat16)
    x[3, 130], x[200, 5], x[201, 255] = float("inf"), float("nan"), float("-inf")
    codes, scale = dllm.fp8_quantize(x.to(dev()), block_rows=block_rows)
    want = quantised(x.float(), block_rows)
    same(codes, want[0])
    same(scale, want[1])


def test_quantize_one_row_of_any_stride(dllm):
    """A single row's stride says nothing; its address does."""
    import torch
    x = torch.randn(1, 131).to(torch.bfloat16)
    codes, scale = dllm.fp8_quantize(x.to(dev())[:, :128])
    want = quantised(x[:, :128].float(), 1)
    same(codes, want[0])
    same(scale, want[1])


def made(gen, M, N, K):
    import torch
    a = torch.randn(M, K, generator=gen) * torch.exp(torch.randn(1, K, generator=gen))
    b = torch.randn(N, K, generator=gen) * torch.exp(0.5 * torch.randn(N, 1, generator=gen))
    return quantised(a.to(torch.bfloat16).float(), 1), quantised(b.to(torch.bfloat16).float(), 128)


def check(dllm, a, sa, b, sb, out=None):
    import torch
    d = dev()
    e4m3 = torch.float8_e4m3fn
    got = dllm.fp8_matmul(a.to(e4m3).to(d), sa.to(d), b.to(e4m3).to(d), sb.to(d), out=out)
    assert dllm.get_device_error(d) == 0
    (M, K), N = a.shape, b.shape[0]
    wide = lambda q, s, r: (q.double() * s.double().repeat_interleave(r, 0)[:q.shape[0]]  # noqa: E731
                            .repeat_interleave(128, 1)[:, :K]).to(d)
    A, B = wide(a, sa, 1), wide(b, sb, 128)
    want, size = A @ B.T, A.abs() @ B.abs().T
    y = got[:, :N].double()
    off = (y - want).abs()
    assert bool((off <= 2.0 ** -8 * want.abs() + (4 * 128 + K / 128 + 2) * 2.0 ** -24 * size).all()), float(
        (off / (2.0 ** -8 * want.abs() + 1e-30)).max())
    edge = -(-N // 8) * 8
    assert not got[:, N:edge].any()
    return got


@pytest.mark.parametrize("M,N,K", [(1, 1, 16), (1, 8, 128), (3, 130, 144), (128, 128, 256), (129, 257, 384), (256, 256, 1024),
                                   (257, 512, 128), (20, 1000, 2000), (300, 3003, 1040), (700, 777, 4096), (2, 50000, 512),
                                   (1100, 40001, 256)])
def test_product(dllm, M, N, K):
    """Tiles that are filled, cut on either side, and more of them than the grid holds; K that ends inside a group."""
    import torch
    gen = torch.Generator().manual_seed(M + N + K)
    (a, sa), (b, sb) = made(gen, M, N, K)
    check(dllm, a, sa, b, sb)


def test_product_exact_sums(dllm):
    """Small whole numbers: every product and sum is exact, so the result is; also rows of a larger output stay as they
    were behind the columns."""
    import torch
    gen = torch.Generator().manual_seed(1)
    M, N, K = 150, 300, 640
    a = torch.randint(-2, 3, (M, K), generator=gen).float()
    b = torch.randint(-2, 3, (N, K), generator=gen).float()
    sa = torch.exp2(torch.randint(-2, 3, (M, 5), generator=gen).float())
    sb = torch.exp2(torch.randint(-2, 3, (3, 5), generator=gen).float())
    out = torch.full((M, 400), 7.0, dtype=torch.bfloat16, device=dev())
    got = check(dllm, a, sa, b, sb, out=out)
    wide = lambda q, s, r: q * s.repeat_interleave(r, 0)[:q.shape[0]].repeat_interleave(128, 1)[:, :K]  # noqa: E731
    want = (wide(a, sa, 1) @ wide(b, sb, 128).T).to(torch.bfloat16)
    same(got[:, :N], want)
    assert bool((got[:, 304:] == 7).all())


def test_product_of_one_element(dllm):
    """Every row and column of a tile lands where it belongs: products of unit rows."""
    import torch
    M, N, K = 256, 256, 256
    for shift in (0, 77):
        a = torch.zeros(M, K)
        a[torch.arange(M), torch.arange(M)] = 1
        b = torch.zeros(N, K)
        b[torch.arange(N), (torch.arange(N) + shift) % K] = 2
        sa, sb = torch.ones(M, 2), torch.ones(2, 2)
        got = check(dllm, a, sa, b, sb)
        same(got, (a @ b.T).to(torch.bfloat16))


def test_product_of_all_codes(dllm):
    """Every finite code meets every other, in rows of their own."""
    import torch
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8)
    v = codes.view(torch.float8_e4m3fn).float()
    v = v[torch.isfinite(v)]
    a = torch.zeros(len(v), 16)
    a[:, 3] = v
    one = torch.ones(1, 1)
    got = check(dllm, a, one.repeat(len(v), 1), a, one.repeat(2, 1))
    same(got[:, :len(v)], (v[:, None] * v[None]).to(torch.bfloat16))


def test_nan_stays_in_its_rows(dllm):
    """A NaN scale makes its row of a, or its 128 rows of b, NaN and nothing else; a NaN code its row."""
    import torch
    gen = torch.Generator().manual_seed(2)
    (a, sa), (b, sb) = made(gen, 300, 500, 384)
    d, e4m3 = dev(), torch.float8_e4m3fn
    sa[7, 1], sb[2, 2] = float("nan"), float("nan")
    ca, cb = a.to(e4m3).to(d), b.to(e4m3).to(d)
    got = dllm.fp8_matmul(ca, sa.to(d), cb, sb.to(d))
    want = torch.zeros(300, 504, dtype=torch.bool)
    want[7, :500] = True
    want[:, 256:384] = True
    assert torch.equal(torch.isnan(got).cpu(), want)
    ca.view(torch.uint8)[100, 200] = 0x7F
    got = dllm.fp8_matmul(ca, sa.to(d), cb, sb.to(d))
    want[100, :500] = True
    assert torch.equal(torch.isnan(got).cpu(), want)


def test_equal_calls_graphs_and_streams(dllm):
    import torch
    gen = torch.Generator().manual_seed(3)
    (a, sa), (b, sb) = made(gen, 130, 3000, 512)
    d, e4m3 = dev(), torch.float8_e4m3fn
    t = a.to(e4m3).to(d), sa.to(d), b.to(e4m3).to(d), sb.to(d)
    want = dllm.fp8_matmul(*t)
    one = dllm.fp8_matmul(t[0][77:78], t[1][77:78], *t[2:])
    assert torch.equal(one[0], want[77])           # a row does not depend on its batch
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    x = torch.randn(40, 512, device=d).to(torch.bfloat16)
    with torch.cuda.graph(g):
        q, s = dllm.fp8_quantize(x)
        out = dllm.fp8_matmul(q, s, *t[2:])
    for _ in range(3):
        x.copy_(torch.randn(40, 512, device=d))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, dllm.fp8_matmul(*dllm.fp8_quantize(x), *t[2:]))
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = []
    torch.cuda.synchronize()
    for st in streams:
        with torch.cuda.stream(st):
            outs.append([dllm.fp8_matmul(*t) for _ in range(5)])
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for row in outs for o in row)
    assert dllm.get_device_error(d) == 0


def test_refusals(dllm):
    import torch
    d, e4m3 = dev(), torch.float8_e4m3fn
    a, sa = torch.zeros(4, 256, device=d).to(e4m3), torch.ones(4, 2, device=d)
    b, sb = torch.zeros(9, 256, device=d).to(e4m3), torch.ones(1, 2, device=d)
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device=d)
    assert dllm.fp8_matmul(a, sa, b, sb).shape == (4, 16)
    assert dllm.fp8_matmul(a[:0], sa[:0], b, sb).shape == (0, 16)
    assert dllm.fp8_quantize(x[:0])[0].shape == (0, 256)
    for bad in ((a.float(), sa, b, sb), (a, sa[:, :1].contiguous(), b, sb), (a, sa, b[:, :128].contiguous(), sb),
                (a, sa, b, sb.repeat(2, 1)), (a, sa.half(), b, sb)):
        with pytest.raises(TypeError):
            dllm.fp8_matmul(*bad)
    with pytest.raises(ValueError):
        dllm.fp8_matmul(a, sa, b.cpu(), sb)
    with pytest.raises(ValueError):
        dllm.fp8_matmul(a, sa, b.t().contiguous().t(), sb)
    with pytest.raises(dllm.DllmError):
        dllm.fp8_matmul(a, sa, b, sb, out=torch.zeros(4, 8, dtype=torch.bfloat16, device=d))
    with pytest.raises(dllm.DllmError):
        dllm.fp8_matmul(a[:, :24].contiguous(), sa[:, :1].contiguous(), b[:, :24].contiguous(), sb[:, :1].contiguous())
    with pytest.raises(TypeError):
        dllm.fp8_quantize(x.float())
    with pytest.raises(ValueError):
        dllm.fp8_quantize(x, block_rows=64)
    with pytest.raises(ValueError):
        dllm.fp8_quantize(x.t())
    with pytest.raises(dllm.DllmError):
        dllm.fp8_quantize(x[:, 1:17])
    assert dllm.get_device_error(d) == 0
