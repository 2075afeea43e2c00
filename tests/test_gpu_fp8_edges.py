"""dllm_fp8_matmul where the two scales' product leaves the range of 32 bits.

The tolerance is the product tests' own: the output's rounding to bf16 (half a step, 2^-8 of the value) and sums in 32
bits, (4 * 128 + K / 128 + 2) 2^-24 of the sum of magnitudes; and what is smaller than bf16 holds, half of its least
step, 2^-134.  With a scale of 2^-126 (`floor`) the scales' product is subnormal, off by half of 2^-149, which the group's
sum of codes multiplies: 2^-150 of the sum of the codes' magnitudes."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def check(dllm, a, sa, b, sb, floor=False):
    import torch
    d, e4m3 = torch.device("cuda", 0), torch.float8_e4m3fn
    got = dllm.fp8_matmul(a.to(e4m3).to(d), sa.to(d), b.to(e4m3).to(d), sb.to(d)).double().cpu()
    assert dllm.get_device_error(d) == 0
    (M, K), N = a.shape, b.shape[0]
    wide = lambda q, s, r: q.double() * s.double().repeat_interleave(r, 0)[:q.shape[0]].repeat_interleave(128, 1)[:, :K]  # noqa: E731
    A, B = wide(a, sa, 1), wide(b, sb, 128)
    want, size = A @ B.T, A.abs() @ B.abs().T
    held = size < 2.0 ** 127              # beyond it, partial sums of 32 bits may pass their range
    off = (got[:, :N] - want).abs()[held]
    bound = (2.0 ** -8 * want.abs() + (4 * 128 + K / 128 + 2) * 2.0 ** -24 * size + 2.0 ** -134)[held]
    if floor:
        bound = bound + (2.0 ** -150 * (a.double().abs() @ b.double().abs().T))[held]
    assert held.any() and bool((off <= bound).all()), float((off / bound).max())
    return got[:, :N]


def codes(gen, n, K):
    import torch
    return (torch.randn(n, K, generator=gen) * 100).clamp(-448, 448).to(torch.float8_e4m3fn).float()


@pytest.mark.parametrize("ea,eb", [(70, 70), (120, 20), (20, 120)])
def test_large_scales(dllm, ea, eb):
    """Scales whose product is 2^140: over codes of zero the result is zero, over the least codes it is finite."""
    import torch
    gen = torch.Generator().manual_seed(ea)
    M, N, K = 140, 300, 256
    a, b = torch.zeros(M, K), codes(gen, N, K)
    sa, sb = torch.full((M, 2), 2.0 ** ea), torch.full((3, 2), 2.0 ** eb)
    assert not check(dllm, a, sa, b, sb).any()
    # codes of 2^-9 in one place of each row: 2^-18 times the scales where the places meet
    a[torch.arange(M), torch.arange(M)] = 2.0 ** -9
    b = torch.zeros(N, K)
    b[torch.arange(N), torch.arange(N) % K] = 2.0 ** -9
    sa[::2] *= 1.5
    sa[3] = 1.0
    got = check(dllm, a, sa, b, sb)
    assert got.abs().max() == 1.5 * 2.0 ** 122


@pytest.mark.parametrize("ea,eb", [(-80, -60), (-90, -58), (-126, -10), (-10, -126), (-126, -126), (-149, 10), (-100, -30)])
def test_small_scales(dllm, ea, eb):
    """Scales whose product is below 2^-126, with large codes: the result is a normal number, good to its last bit."""
    import torch
    gen = torch.Generator().manual_seed(-ea)
    M, N, K = 140, 300, 400
    a, b = codes(gen, M, K), codes(gen, N, K)
    sa = (torch.rand(M, 4, generator=gen) + 1) * 2.0 ** ea
    sb = (torch.rand(3, 4, generator=gen) + 1) * 2.0 ** eb
    check(dllm, a, sa, b, sb)
    sa[::3], sb[:, 2] = 1.0, 0.5          # among ordinary rows and groups
    check(dllm, a, sa, b, sb)


def test_scales_of_zero(dllm):
    """A scale of 0 makes its part 0, whatever finite scale it meets."""
    import torch
    gen = torch.Generator().manual_seed(12)
    M, N, K = 140, 300, 256
    a, b = codes(gen, M, K), codes(gen, N, K)
    sa, sb = torch.rand(M, 2, generator=gen) + 0.5, torch.full((3, 2), 2.0 ** 110)
    sa[::3], sb[1] = 0, 0
    sa[1] = 2.0 ** -100
    got = check(dllm, a, sa * 2.0 ** -10, b, sb)
    assert not got[::3].any() and not got[:, 128:256].any() and got[1, :128].any()
    sa[:], sb[:] = 2.0 ** 120, 0
    assert not check(dllm, a, sa, b, sb).any()


def test_least_scale(dllm):
    """Rows at the quantiser's least scale, beside ordinary ones: zeros stay zeros, others are good to what is promised."""
    import torch
    gen = torch.Generator().manual_seed(11)
    M, N, K = 140, 300, 400
    a, b = codes(gen, M, K), codes(gen, N, K)
    a[::4] = 0
    sa, sb = torch.rand(M, 4, generator=gen) + 0.5, (torch.rand(3, 4, generator=gen) + 1) * 2.0 ** -10
    sa[::2] = 2.0 ** -126
    sb[1] = 2.0 ** -126
    got = check(dllm, a, sa, b, sb, floor=True)
    assert not got[::4].any() and got[2::4].any()


def test_quantised_rows_of_any_size(dllm):
    """The quantiser's own scales, from rows of zeros and of the least bf16 values to the largest."""
    import torch
    d = torch.device("cuda", 0)
    gen = torch.Generator().manual_seed(5)
    x, w = torch.randn(60, 512, generator=gen), torch.randn(200, 512, generator=gen)
    x *= torch.exp2(torch.linspace(-130, 120, 60).round()[:, None])
    x[7], x[8, :128] = 0, 0
    for power in (-100, -20, -8, 100):
        y = (w * 2.0 ** power).to(torch.bfloat16)
        qa, sa = dllm.fp8_quantize(x.to(torch.bfloat16).to(d))
        qb, sb = dllm.fp8_quantize(y.to(d), block_rows=128)
        got = check(dllm, qa.float().cpu(), sa.cpu(), qb.float().cpu(), sb.cpu())
        assert not got[7].any()


@pytest.mark.parametrize("M,N,K", [(3, 20, 144), (300, 513, 512)])
def test_rows_that_lie_apart(dllm, M, N, K):
    """Strides of both operands above K and of the output above N: the same bits as of packed ones, what lies between left
    as it was and never read (codes of NaN)."""
    import ctypes
    import torch
    d = torch.device("cuda", 0)
    gen = torch.Generator().manual_seed(M)
    e4m3 = torch.float8_e4m3fn
    blocks = -(-K // 128)
    a, b = codes(gen, M, K).to(e4m3), codes(gen, N, K).to(e4m3)
    sa, sb = torch.rand(M, blocks, generator=gen).to(d), torch.rand(-(-N // 128), blocks, generator=gen).to(d)
    want = dllm.fp8_matmul(a.to(d), sa, b.to(d), sb)

    def apart(x, pad):
        wide = torch.full((x.shape[0] + 1, K + pad), 0x7F, dtype=torch.uint8)
        wide[:-1, :K] = x.view(torch.uint8)
        return wide.to(d)
    wa, wb = apart(a, 48), apart(b, 16)
    ldo = -(-N // 8) * 8 + 24
    out = torch.full((M, ldo), 7.0, dtype=torch.bfloat16, device=d)
    args = dllm.Fp8MatmulArgs(M, N, K, 0, K + 48, K + 16, ldo, wa.data_ptr(), sa.data_ptr(), wb.data_ptr(), sb.data_ptr(),
                              out.data_ptr())
    assert dllm.load().dllm_fp8_matmul(ctypes.byref(args), torch.cuda.current_stream().cuda_stream) == 0
    assert dllm.get_device_error(d) == 0
    edge = want.shape[1]
    assert torch.equal(out[:, :edge], want) and bool((out[:, edge:] == 7).all())
