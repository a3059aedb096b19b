"""The row norm (gdr_norm_fwd, gdr_norm_quant, gdr_norm_bwd) through the C ABI against
its formula in 64 bits, element by element within the bounds of layer_ref."""

import pytest
import torch

from chunked_gated_delta_bwd_amd import binding as B
import layer_ref as R

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
CODE = {"bf16": B.GDR_BF16, "f32": B.GDR_F32}
EPS = 1e-6

# every number of threads and vectors a row can take, their borders, and odd widths
WIDTHS = [1, 7, 8, 13, 16, 24, 64, 100, 128, 136, 200, 256, 260, 512, 520, 1000, 1024, 1028, 2040, 2048, 2056, 4096, 4100, 8192, 8200, 16384,
          16392, 32767, 32768]


def make(seed, rows, width, dtype, res=True, weight=True):
    gen = torch.Generator().manual_seed(seed)
    dt = DT[dtype]
    x = R.rand(gen, rows, width).to(dt)
    r = R.rand(gen, rows, width, std=4.0).to(dt) if res else None
    w = (1 + R.rand(gen, width, std=0.2)).float() if weight else None
    dy = R.rand(gen, rows, width).to(dt)
    dres = R.rand(gen, rows, width).to(dt) if res else None
    return x, r, w, dy, dres


def cu(*ts):
    return [None if t is None else t.cuda() for t in ts]


def nan_like(t, dtype=None):
    return torch.full_like(t, float("nan"), dtype=dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("width", WIDTHS)
def test_forward_and_backward(width, dtype):
    rows = 5 if width > 4096 else 33
    res, weight = width % 3 != 1, width % 5 != 0
    x, r0, w, dy, dres = make(width, rows, width, dtype, res, weight)
    r, rstd, y_ref, rel = R.norm(x, r0, w, EPS)
    xd, rd, wd, dyd, dresd = cu(x, r0, w, dy, dres)
    prob = B.NormProblem(rows, width, CODE[dtype], EPS)
    y, res_out = nan_like(xd), nan_like(xd) if res else None
    B.gdr_norm_fwd(prob, xd, wd, y, res=rd, res_out=res_out)
    torch.cuda.synchronize()
    R.check("y", y, y_ref, rel * y_ref.abs())
    if res:
        R.check("res_out", res_out, r, U1(r))
    rin = res_out if res else xd
    dx_ref, dx_err, dw_ref, dw_err = R.norm_bwd(rin.cpu(), w, dy, dres, EPS)
    dx, dw = nan_like(xd), torch.full((width,), float("nan"), device="cuda")
    ws = B.alloc_norm_workspace(prob)
    ws.fill_(255)
    B.gdr_norm_bwd(prob, rin, wd, dyd, dx, dw, ws, dres=dresd)
    torch.cuda.synchronize()
    R.check("dx", dx, dx_ref, dx_err)
    R.check("dw", dw, dw_ref, dw_err)


def U1(r):
    return R.U * r.abs()


@pytest.mark.parametrize("rows,width", [(1, 128), (4099, 128), (70001, 16), (2050, 2048), (1500, 40)])
def test_many_rows(rows, width):
    """Several rows a workgroup, a last workgroup that is not full, more rows than the
    backward has workgroups."""
    x, _, w, dy, _ = make(rows, rows, width, "bf16", res=False)
    xd, wd, dyd = cu(x, w, dy)
    prob = B.NormProblem(rows, width, B.GDR_BF16, EPS)
    y, dx, dw = nan_like(xd), nan_like(xd), nan_like(wd)
    B.gdr_norm_fwd(prob, xd, wd, y)
    B.gdr_norm_bwd(prob, xd, wd, dyd, dx, dw, B.alloc_norm_workspace(prob))
    torch.cuda.synchronize()
    _, _, y_ref, rel = R.norm(x, None, w, EPS)
    dx_ref, dx_err, dw_ref, dw_err = R.norm_bwd(x, w, dy, None, EPS)
    R.check("y", y, y_ref, rel * y_ref.abs())
    R.check("dx", dx, dx_ref, dx_err)
    R.check("dw", dw, dw_ref, dw_err)


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("width", WIDTHS)
def test_e4m3(width, dtype, group):
    rows = 3 if width > 4096 else 19
    res = width % 3 != 1
    x, r0, w, _, _ = make(width + 1, rows, width, dtype, res)
    x[1] = 0
    if res:
        r0[1] = 0
    xd, rd, wd = cu(x, r0, w)
    prob = B.NormProblem(rows, width, CODE[dtype], EPS, group=group)
    n = -(-width // group) if group else 1
    q = torch.full((rows, width), 255, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    scales, res_out = torch.full((rows, n), float("nan"), device="cuda"), nan_like(xd) if res else None
    B.gdr_norm_quant(prob, xd, wd, q, scales, res=rd, res_out=res_out)
    torch.cuda.synchronize()
    r, _, y_ref, rel = R.norm(x, r0, w, EPS)
    s_ref, z = R.e4m3_ref(y_ref, group)
    R.check("scales", scales, s_ref, (rel + 2 * R.U) * s_ref)
    # half a step of e4m3: 2^-4 of a normal value, 2^-10 below 2^-6; y / scale carries both errors
    off = (q.cpu().float().double() - z).abs()
    tol = (2.0 ** -4 + 2 * rel + 4 * R.U) * z.abs() + 2.0 ** -10
    assert (off <= tol).all(), float((off / tol).max())
    assert (q[1].float() == 0).all() and (scales[1] == 2.0 ** -126).all()
    if res:
        R.check("res_out", res_out, r, U1(r))


def test_e4m3_rounds_to_even_and_keeps_the_sign():
    """y = n w with n = +-1 exactly: the bytes are those of torch's conversion."""
    width = 512
    x = torch.ones(2, width)
    x[1, ::2] = -1
    w = torch.linspace(-448, 448, width)
    prob = B.NormProblem(2, width, B.GDR_F32, 0.0)
    q = torch.empty(2, width, dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty(2, 1, device="cuda")
    B.gdr_norm_quant(prob, x.cuda(), w.cuda(), q, scales)
    torch.cuda.synchronize()
    assert torch.equal(scales.cpu(), torch.ones(2, 1))
    assert torch.equal(q.cpu().view(torch.uint8), (x * w).to(torch.float8_e4m3fn).view(torch.uint8))


@pytest.mark.parametrize("group", [0, 128])
def test_nan_and_infinity_stay_in_their_row(group):
    for width in (256, 300):
        x, r0, w, _, _ = make(3, 6, width, "bf16")
        clean = [t.clone() for t in (x, r0)]
        x[2, 5], x[4, 200] = float("nan"), float("inf")
        prob = B.NormProblem(6, width, B.GDR_BF16, EPS, group=group)
        n = -(-width // group) if group else 1

        def go(a, b):
            q = torch.empty(6, width, dtype=torch.float8_e4m3fn, device="cuda")
            s, ro, y = torch.empty(6, n, device="cuda"), torch.empty(6, width, dtype=torch.bfloat16, device="cuda"), None
            B.gdr_norm_quant(prob, a.cuda(), w.cuda(), q, s, res=b.cuda(), res_out=ro)
            y = torch.empty_like(ro)
            B.gdr_norm_fwd(prob, a.cuda(), w.cuda(), y, res=b.cuda(), res_out=ro)
            torch.cuda.synchronize()
            return q.float(), s, y

        (q, s, y), (q0, s0, y0) = go(x, r0), go(*clean)
        keep = [0, 1, 3, 5]
        assert torch.equal(q[keep], q0[keep]) and torch.equal(s[keep], s0[keep]) and torch.equal(y[keep], y0[keep])
        assert y[2].isnan().all() and s[2].isnan().all() and q[2].isnan().all()
        # an infinity: 1 / rms is zero, so its own place is NaN (0 * inf) and the others zero
        g = 200 // group if group else 0
        assert y[4, 200].isnan() and s[4, g].isnan()
        others = torch.ones(width, dtype=torch.bool)
        others[200] = False
        assert (y[4].cpu()[others] == 0).all()


def test_in_place_and_no_rows():
    """res_out over res, y over x, dx over dy; no rows: nothing but dw = 0."""
    x, r0, w, dy, dres = make(9, 40, 1024, "bf16")
    prob = B.NormProblem(40, 1024, B.GDR_BF16, EPS)
    xd, rd, wd, dyd, dresd = cu(x, r0, w, dy, dres)
    y, ro = torch.empty_like(xd), torch.empty_like(xd)
    B.gdr_norm_fwd(prob, xd, wd, y, res=rd, res_out=ro)
    dx, dw, ws = torch.empty_like(xd), torch.empty_like(wd), B.alloc_norm_workspace(prob)
    B.gdr_norm_bwd(prob, ro, wd, dyd, dx, dw, ws, dres=dresd)
    x2, r2, d2 = xd.clone(), rd.clone(), dyd.clone()
    B.gdr_norm_fwd(prob, x2, wd, x2, res=r2, res_out=r2)
    dw2 = torch.empty_like(wd)
    B.gdr_norm_bwd(prob, r2, wd, d2, d2, dw2, ws, dres=dresd)
    torch.cuda.synchronize()
    assert torch.equal(x2, y) and torch.equal(r2, ro) and torch.equal(d2, dx) and torch.equal(dw2, dw)
    d3 = torch.empty_like(xd)
    B.gdr_norm_bwd(prob, ro, wd, dyd, d3, None, None, dres=dresd)   # dw not returned: no workspace
    torch.cuda.synchronize()
    assert torch.equal(d3, dx)
    none = B.NormProblem(0, 1024, B.GDR_BF16, EPS)
    e = torch.empty(0, 1024, dtype=torch.bfloat16, device="cuda")
    dw.fill_(1)
    B.gdr_norm_fwd(none, e, wd, e)
    B.gdr_norm_bwd(none, e, wd, e, e, dw, B.alloc_norm_workspace(none))
    torch.cuda.synchronize()
    assert not dw.any()


def test_differences():
    rows, width = 6, 72
    x, r0, w, dy, dres = make(13, rows, width, "f32")
    prob = B.NormProblem(rows, width, B.GDR_F32, EPS)
    xd, rd, wd, dyd, dresd = cu(x, r0, w, dy, dres)

    def loss(a, b, c):
        y, ro = torch.empty_like(a), torch.empty_like(a)
        B.gdr_norm_fwd(prob, a, c, y, res=b, res_out=ro)
        return float((y.double() * dyd.double()).sum() + (ro.double() * dresd.double()).sum()), ro

    _, ro = loss(xd, rd, wd)
    dx, dw = torch.empty_like(xd), torch.empty_like(wd)
    B.gdr_norm_bwd(prob, ro, wd, dyd, dx, dw, B.alloc_norm_workspace(prob), dres=dresd)
    gen = torch.Generator().manual_seed(1)
    v, u = torch.randn(rows, width, generator=gen).cuda(), torch.randn(width, generator=gen).cuda()
    h = 1e-2
    for num, ana, size in (
            ((loss(xd + h * v, rd, wd)[0] - loss(xd - h * v, rd, wd)[0]) / (2 * h), dx * v, (dx * v).abs().sum()),
            ((loss(xd, rd + h * v, wd)[0] - loss(xd, rd - h * v, wd)[0]) / (2 * h), dx * v, (dx * v).abs().sum()),
            ((loss(xd, rd, wd + h * u)[0] - loss(xd, rd, wd - h * u)[0]) / (2 * h), dw * u, (dw * u).abs().sum())):
        # 432 terms of size ~4 with ~1e-7 each over 2 h: below 1e-3; the third difference ~ h^2
        assert abs(num - float(ana.double().sum())) <= 1e-3 * float(size) + 1e-3


def test_streams_and_graph():
    x, r0, w, dy, dres = make(17, 300, 520, "bf16")
    xd, rd, wd, dyd, dresd = cu(x, r0, w, dy, dres)
    prob, quant = B.NormProblem(300, 520, B.GDR_BF16, EPS), B.NormProblem(300, 520, B.GDR_BF16, EPS, group=128)
    ws = B.alloc_norm_workspace(prob)

    def buffers():
        return [torch.empty_like(xd), torch.empty_like(xd), torch.empty_like(xd), torch.empty_like(wd),
                torch.empty(300, 520, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(300, 5, device="cuda")]

    def go(b, work):
        B.gdr_norm_fwd(prob, xd, wd, b[0], res=rd, res_out=b[1])
        B.gdr_norm_bwd(prob, b[1], wd, dyd, b[2], b[3], work, dres=dresd)
        B.gdr_norm_quant(quant, xd, wd, b[4], b[5], res=rd, res_out=b[1])

    same = lambda a, b: all(torch.equal(u.view(torch.uint8), v.view(torch.uint8)) for u, v in zip(a, b))  # noqa: E731
    ref, got = buffers(), buffers()
    go(ref, ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        go(got, ws)
    s.synchronize()
    assert same(ref, got)
    cap, ws2 = buffers(), B.alloc_norm_workspace(prob)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(cap, ws2)
    for _ in range(4):
        xd.copy_(xd.flip(0))
        go(ref, ws)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert same(ref, cap)
