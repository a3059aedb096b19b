"""The e4m3 product with bf16 results, of whole numbers: exact sums, bit for bit."""

import pytest
import torch

from chunked_gated_delta_bwd_amd import binding as B
import lin_ref as L

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

F8 = torch.float8_e4m3fn


@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("M,N,K", [
    (1, 40, 640), (5, 300, 129), (32, 50, 2050),                          # few rows
    (40, 260, 640), (300, 260, 652), (200, 300, 650), (64, 200, 2100),    # small tiles, the last in two runs
    (200, 300, 4098),                                                     # in runs, rows through registers
    (3000, 3100, 384), (3000, 3100, 390),                                 # medium tiles, copied and through registers
    (2560, 3340, 512), (2500, 3500, 652), (2817, 2817, 1040),             # the largest
])
def test_whole_numbers(M, N, K, block):
    """Whole numbers up to 8: products are 1 to 64, so none of their bits lies 2^-13 below another
    product, and of a sum below 2^13 none is lost either (here below 2^11).  Scales are powers of two
    from 1/2 to 2: every sum is a whole number of quarters below 2^22, exact in fp32, and c is that
    sum rounded once."""
    gen = torch.Generator().manual_seed(M + N + K)
    a, b = (torch.randint(-8, 9, s, generator=gen).float() for s in ((M, K), (N, K)))
    G = -(-K // 128)
    sa = torch.exp2(torch.randint(-1, 2, (M, G), generator=gen).float())
    sb = torch.exp2(torch.randint(-1, 2, (-(-N // block), G), generator=gen).float())
    a, b = a.to(F8), b.to(F8)
    prob = B.GemmProblem(M, N, K, B.GDR_BF16, block=block)
    c, ws = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda"), B.alloc_gemm_workspace(prob)
    B.gdr_gemm(prob, a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), c, ws)
    torch.cuda.synchronize()
    want = L.product(a, sa, b, sb, block)[0]
    assert torch.equal(want.float().double(), want)
    assert torch.equal(c.cpu(), want.float().to(torch.bfloat16))
