"""Scales of the e4m3 product at the ends of fp32: a group's two scales are multiplied first,
in fp32, so c is right as long as that product is in range, and what follows from it beyond."""

import pytest
import torch

from chunked_gated_delta_bwd_amd import binding as B
import layer_ref as R

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

F8 = torch.float8_e4m3fn
# few rows, small tiles, a split contraction, medium tiles (fp32) or the largest (bf16); medium tiles of both
SIZES = [(5, 40, 300), (40, 300, 301), (64, 200, 2048), (2560, 3340, 512), (2600, 3500, 650)]


def whole(M, N, K):
    gen = torch.Generator().manual_seed(M + K)
    return [torch.randint(-8, 9, s, generator=gen).float().to(F8) for s in ((M, K), (N, K))]


def product(M, N, K, block, dtype, a, sa, b, sb):
    c = torch.full((M, N), float("nan"), dtype=dtype, device="cuda")
    prob = B.GemmProblem(M, N, K, B.GDR_BF16 if dtype is torch.bfloat16 else B.GDR_F32, block=block)
    B.gdr_gemm(prob, a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), c, B.alloc_gemm_workspace(prob))
    torch.cuda.synchronize()
    return c.cpu()


def scales(M, N, K, block, x, y):
    G = -(-K // 128)
    return torch.full((M, G), x), torch.full((-(-N // block), G), y)


def scaled(M, N, K, block, dtype, a, b, x, y):
    sa, sb = scales(M, N, K, block, x, y)
    return product(M, N, K, block, dtype, a, sa, b, sb)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_scales_whose_product_is_in_range(M, N, K, block, dtype):
    """Whole numbers up to 8 in groups of 128 and powers of two, the product of two between 2^-126 and
    2^114: c is the exact sum, rounded to its type."""
    a, b = whole(M, N, K)
    sums = a.double() @ b.double().t()
    for x, y in ((2.0 ** 100, 2.0 ** -126), (2.0 ** -149, 2.0 ** 120), (2.0 ** 57, 2.0 ** 55), (2.0 ** -126, 1.0), (2.0 ** -60, 2.0 ** -66)):
        c = scaled(M, N, K, block, dtype, a, b, x, y)
        want = (sums * (x * y)).float().to(dtype)                     # exact in fp32
        assert torch.equal(c, want), (x, y)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_scales_whose_product_is_not(M, N, K, block, dtype):
    """A subnormal product has a subnormal's bits, and c those of the sums times it; an infinite one makes
    c infinite or NaN; one that is zero leaves nothing."""
    a, b = whole(M, N, K)
    x, y = 1.2345 * 2.0 ** -70, 1.3579 * 2.0 ** -66
    sa, sb = scales(M, N, K, block, x, y)
    f = float(sa[0, 0] * sb[0, 0])                                    # in fp32
    assert 0 < f < 2.0 ** -126 and abs(f / (float(sa[0, 0]) * float(sb[0, 0])) - 1) > 2.0 ** -20
    sums = a.double() @ b.double().t()
    # each group's sum times f is rounded once, by half of fp32's least step there
    err = (sa.shape[1] + 4) * (R.U * f * (a.double().abs() @ b.double().abs().t()) + 2.0 ** -150)
    c = product(M, N, K, block, dtype, a, sa, b, sb)
    off = (c.double() - sums * f).abs()
    assert (off <= err + R.HALF[dtype] * (sums * f).abs() + 2.0 ** -134).all()
    c = scaled(M, N, K, block, dtype, a, b, 2.0 ** 64, 2.0 ** 64)
    assert not torch.isfinite(c).any()
    c = scaled(M, N, K, block, dtype, a, b, 2.0 ** -100, 2.0 ** -100)
    assert not c.any()
