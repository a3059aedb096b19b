"""The e4m3 product with scales for each 128 of the contraction (gdr_gemm) and the
quantisation that makes its operands (gdr_quant) through the C ABI: bytes and scales bit
for bit, sums within the bounds of lin_ref."""

import pytest
import torch

from chunked_gated_delta_bwd_amd import binding as B
import layer_ref as R
import lin_ref as L

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

F8 = torch.float8_e4m3fn
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
CODE = {"bf16": B.GDR_BF16, "f32": B.GDR_F32}


def rand8(gen, *shape):
    """Every finite byte."""
    b = torch.randint(0, 254, shape, generator=gen, dtype=torch.int32)
    return (b + (b >= 127).int()).to(torch.uint8).view(F8)


def make(seed, M, N, K, block):
    gen = torch.Generator().manual_seed(seed)
    G = -(-K // 128)
    sa = torch.exp2(4 * torch.rand(M, G, generator=gen) - 10)
    sb = torch.exp2(4 * torch.rand(-(-N // block), G, generator=gen) - 10)
    return rand8(gen, M, K), sa, rand8(gen, N, K), sb


def gemm(prob, a, sa, b, sb, dtype, ws=None):
    c = torch.full((prob.shape.M, prob.shape.N), float("nan"), dtype=DT[dtype], device="cuda")
    if ws is None:
        ws = B.alloc_gemm_workspace(prob)
        if ws is not None:
            ws.fill_(255)
    B.gdr_gemm(prob, a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), c, ws)
    torch.cuda.synchronize()
    return c


SIZES = [(1, 1, 1), (1, 16, 128), (1, 4096, 2048), (3, 17, 129), (16, 130, 300), (17, 33, 1000), (33, 48, 16),
         (64, 257, 1024), (65, 65, 128), (65, 129, 15), (128, 128, 4096), (129, 130, 1037), (200, 300, 2000),
         (256, 256, 256), (257, 511, 272), (1000, 2050, 1028), (66, 1, 130), (100, 4100, 144)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_product(M, N, K, block, dtype):
    a, sa, b, sb = make(M + N + K, M, N, K, block)
    c = gemm(B.GemmProblem(M, N, K, CODE[dtype], block=block), a, sa, b, sb, dtype)
    want, err = L.product(a, sa, b, sb, block, DT[dtype])
    R.check("c", c, want, err)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("M,N,K", [(3584, 3600, 272), (4096, 3328, 256), (2500, 3500, 652), (2560, 3340, 512), (2817, 2817, 1040)])
def test_large_tiles(M, N, K, block, dtype):
    """Enough rows and columns for the larger tiles and, from K = 512 on with a bf16 result, the largest,
    whole and cut; last groups of 16 and of 12."""
    a, sa, b, sb = make(M, M, N, K, block)
    c = gemm(B.GemmProblem(M, N, K, CODE[dtype], block=block), a, sa, b, sb, dtype)
    want, err = L.product(a, sa, b, sb, block, DT[dtype])
    R.check("c", c, want, err)


@pytest.mark.parametrize("M,N,K,block", [(5, 40, 640, 128), (300, 260, 640, 128), (300, 260, 650, 1), (3584, 3584, 384, 1)])
def test_small_numbers_are_exact(M, N, K, block):
    """Whole numbers up to 8 and scales that are powers of two: every sum fits fp32."""
    gen = torch.Generator().manual_seed(1)
    a, b = (torch.randint(-8, 9, s, generator=gen).float() for s in ((M, K), (N, K)))
    G = -(-K // 128)
    sa = torch.exp2(torch.randint(-1, 2, (M, G), generator=gen).float())
    sb = torch.exp2(torch.randint(-1, 2, (-(-N // block), G), generator=gen).float())
    c = gemm(B.GemmProblem(M, N, K, B.GDR_F32, block=block), a.to(F8), sa, b.to(F8), sb, "f32")
    assert torch.equal(c.cpu().double(), L.product(a.to(F8), sa, b.to(F8), sb, block)[0])


@pytest.mark.parametrize("M,N,K", [(20, 50, 300), (200, 150, 300), (3584, 3584, 256), (2600, 3500, 650), (2600, 3500, 656)])
def test_nan_stays_in_its_row_and_column(M, N, K):
    """A NaN byte or scale of a reaches its row of c, of b its column (a block's scale: its 128)."""
    a, sa, b, sb = make(2, M, N, K, 128)
    prob = B.GemmProblem(M, N, K, B.GDR_BF16)
    clean = gemm(prob, a, sa, b, sb, "bf16")
    a.view(torch.uint8)[7, K - 1], b.view(torch.uint8)[9, 0] = 0x7f, 0xff
    sa[11, 0], sb[(N - 1) // 128, 1] = float("nan"), float("inf")
    got = gemm(prob, a, sa, b, sb, "bf16")
    rows, cols = torch.ones(M, dtype=torch.bool), torch.ones(N, dtype=torch.bool)
    rows[[7, 11]] = False
    cols[9] = False
    cols[(N - 1) // 128 * 128:] = False
    keep = rows[:, None] & cols[None, :]
    assert torch.equal(got.cpu()[keep], clean.cpu()[keep])
    assert got[7].isnan().all() and got[11].isnan().all() and got[:, 9].isnan().all()
    assert not got[:, (N - 1) // 128 * 128:].isfinite().any()


def test_no_rows_or_columns():
    for M, N in ((0, 5), (5, 0), (0, 0)):
        a, b = torch.empty(M, 200, dtype=F8, device="cuda"), torch.empty(N, 200, dtype=F8, device="cuda")
        c = torch.empty(M, N, device="cuda")
        B.gdr_gemm(B.GemmProblem(M, N, 200, B.GDR_F32, block=1), a, torch.empty(M, 2, device="cuda"), b,
                   torch.empty(N, 2, device="cuda"), c)
        x = torch.empty(M, N, device="cuda")
        p = B.QuantProblem(M, N, B.GDR_F32)
        B.gdr_quant(p, x, torch.empty(p.q_shape, dtype=F8, device="cuda"), torch.empty(p.scales_shape, device="cuda"))
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 4096), (7, 130), (128, 128), (129, 127), (300, 1000), (64, 2050), (1025, 8),
                                       (255, 257)])
def test_quant(rows, cols, block, transpose, dtype):
    gen = torch.Generator().manual_seed(rows + cols)
    x = (R.rand(gen, rows, cols) * torch.exp(3 * R.rand(gen, rows, 1))).to(DT[dtype])
    if rows > 2:
        x[1] = 0
    p = B.QuantProblem(rows, cols, CODE[dtype], block=block, transpose=transpose)
    q = torch.full(p.q_shape, 255, dtype=torch.uint8, device="cuda").view(F8)
    scales = torch.full(p.scales_shape, float("nan"), device="cuda")
    B.gdr_quant(p, x.cuda(), q, scales)
    torch.cuda.synchronize()
    want, s = L.quantised(x.t() if transpose else x, block)
    assert torch.equal(scales.cpu(), s)
    assert torch.equal(q.cpu().view(torch.uint8), want.view(torch.uint8))


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("block", [1, 128])
def test_quant_nonfinite_and_tiny(block, transpose):
    """A NaN makes its group NaN; beside an infinity everything is zero but its own place, a NaN;
    numbers below the least scale."""
    x = torch.randn(256, 384, generator=torch.Generator().manual_seed(4))
    x[3, 5], x[200, 300], x[140, 20] = float("nan"), float("inf"), float("-inf")
    x[128:, 128:256] = 1e-40
    y = x.t() if transpose else x
    p = B.QuantProblem(256, 384, B.GDR_F32, block=block, transpose=transpose)
    q, s = torch.zeros(p.q_shape, dtype=F8, device="cuda"), torch.zeros(p.scales_shape, device="cuda")
    B.gdr_quant(p, x.cuda(), q, s)
    torch.cuda.synchronize()
    g = y.reshape(-1, block, y.shape[1] // 128, 128)
    top = g.abs().amax((1, 3))                        # NaN where one is, else the largest
    want = (top / torch.full_like(top, 448.0)).clamp(min=2.0 ** -126)
    z = (g / want[:, None, :, None]).reshape(y.shape).to(F8)
    assert torch.equal(s.cpu().nan_to_num(-1, posinf=1e39), want.nan_to_num(-1, posinf=1e39))
    a, b = q.cpu().float(), z.float()
    assert torch.equal(a.isnan(), b.isnan()) and torch.equal(a[~a.isnan()], b[~b.isnan()])


def test_streams_graphs_and_two_calls_at_once():
    gen = torch.Generator().manual_seed(6)
    M, N, K = 200, 300, 2100
    x, w = R.rand(gen, M, K).float().cuda(), R.rand(gen, N, K).float().cuda()
    px, pw = B.QuantProblem(M, K, B.GDR_F32), B.QuantProblem(N, K, B.GDR_F32, block=128)
    prob = B.GemmProblem(M, N, K, B.GDR_BF16)
    assert B.gdr_gemm_workspace_bytes(prob) > 0

    def new():
        f = lambda p: [torch.empty(p.q_shape, dtype=F8, device="cuda"), torch.empty(p.scales_shape, device="cuda")]  # noqa: E731
        return f(px) + f(pw) + [torch.empty(M, N, dtype=torch.bfloat16, device="cuda"), B.alloc_gemm_workspace(prob)]

    def go(b):
        B.gdr_quant(px, x, b[0], b[1])
        B.gdr_quant(pw, w, b[2], b[3])
        B.gdr_gemm(prob, *b[:4], b[4], b[5])

    ref, one, two, cap = new(), new(), new(), new()
    go(ref)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for s, b in ((s1, one), (s2, two)):
        with torch.cuda.stream(s):
            go(b)
    torch.cuda.synchronize()
    assert torch.equal(ref[4], one[4]) and torch.equal(ref[4], two[4])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(cap)
    for _ in range(4):
        x.copy_(x.flip(0))
        go(ref)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(ref[4], cap[4])
