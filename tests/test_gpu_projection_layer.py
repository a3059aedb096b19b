"""The operators of an attention layer together: norm to e4m3, the projections, linear
attention with a decay for each head, the quantisation between, and their gradients, each
stage against 64 bits from what the stage before gave; a prompt and the tokens after it; the
whole as one graph.  Packs of many sequences, and offsets beyond 32 bits (mostly zeros, the
last rows checked)."""

import pytest
import torch

from chunked_gated_delta_bwd_amd import binding as B
import layer_ref as R
import lin_ref as L

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

BF, F8, F32 = torch.bfloat16, torch.float8_e4m3fn, torch.float32


def dev(*s, dtype=F32):
    return torch.full(s, float("nan"), device="cuda").to(dtype)


def quant(x, block=1, transpose=False):
    p = B.QuantProblem(*x.shape, B.GDR_BF16 if x.dtype is BF else B.GDR_F32, block=block, transpose=transpose)
    q, s = torch.empty(p.q_shape, dtype=F8, device="cuda"), torch.empty(p.scales_shape, device="cuda")
    B.gdr_quant(p, x, q, s)
    return q, s


def gemm(a, b, dtype=BF, block=128):
    p = B.GemmProblem(a[0].shape[0], b[0].shape[0], a[0].shape[1], B.GDR_BF16 if dtype is BF else B.GDR_F32, block=block)
    c = dev(a[0].shape[0], b[0].shape[0], dtype=dtype)
    B.gdr_gemm(p, *a, *b, c, B.alloc_gemm_workspace(p))
    return c


class Layer:
    """y = W_o lin(W_q n, W_k n, W_v n), n = norm(x): every weight [out, in], e4m3 by blocks
    of 128 x 128, transposed once for the backward."""

    def __init__(self, gen, W, H, Hk, D):
        self.W, self.H, self.Hk, self.D = W, H, Hk, D
        self.norm = (1 + 0.2 * R.rand(gen, W)).float().cuda()
        self.decay = (-torch.exp2(-1.0 - 6.0 * torch.rand(H, generator=gen))).cuda()
        shapes = {"q": (Hk * D, W), "k": (Hk * D, W), "v": (H * D, W), "o": (W, H * D)}
        w = {n: R.rand(gen, *s, std=s[1] ** -0.5).to(BF).cuda() for n, s in shapes.items()}
        self.w = {n: quant(x, 128) for n, x in w.items()}
        self.wt = {n: quant(x, 128, True) for n, x in w.items()}

    def project(self, x):
        rows = x.shape[0]
        n = torch.empty(rows, self.W, dtype=F8, device="cuda"), dev(rows, self.W // 128)
        B.gdr_norm_quant(B.NormProblem(rows, self.W, B.GDR_BF16, 1e-6, group=128), x, self.norm, *n)
        t = {m: gemm(n, self.w[m]).view(rows, -1, self.D) for m in "qkv"}
        return n, {**t, "log_decay": self.decay}

    def problem(self, lengths):
        cu = [0]
        for n in lengths:
            cu.append(cu[-1] + n)
        return B.LinProblem(1, cu[-1], self.H, self.D, len(lengths), B.GDR_BF16, 1.0, cu_seqlens=cu, Hk=self.Hk)

    def forward(self, x, lengths):
        r = {"x": x}
        r["n"], t = self.project(x)
        prob = self.problem(lengths)
        r["t"], r["ws"] = {**t, "h0": None}, B.alloc_lin_workspace(prob, backward=True)
        r["o"], r["ht"] = dev(*t["v"].shape, dtype=BF), dev(len(lengths), self.H, self.D, self.D)
        B.gdr_lin_fwd(prob, r["t"], r["ws"], r["o"], ht=r["ht"])
        r["o8"] = quant(r["o"].view(len(x), -1))
        r["y"] = gemm(r["o8"], self.w["o"])
        return r

    def backward(self, r, dy, lengths):
        T, g = len(dy), {}
        g["dy8"] = quant(dy)
        g["dO"] = gemm(g["dy8"], self.wt["o"]).view(T, self.H, self.D)
        g["dyt"], g["ot"] = quant(dy, transpose=True), quant(r["o"].view(T, -1), transpose=True)
        g["dWo"] = gemm(g["dyt"], g["ot"], F32, block=1)
        g.update({"d" + m: dev(*r["t"][m].shape, dtype=BF) for m in "qkv"})
        B.gdr_lin_bwd(self.problem(lengths), r["t"], g["dO"], None, r["ws"], g)
        n = dev(T, self.W, dtype=BF)
        B.gdr_norm_fwd(B.NormProblem(T, self.W, B.GDR_BF16, 1e-6), r["x"], self.norm, n)
        g["nt"] = quant(n, transpose=True)
        dn = torch.zeros(T, self.W, device="cuda")
        for m in "qkv":
            d = g["d" + m].view(T, -1)
            g[m + "8"], g[m + "t"] = quant(d), quant(d, transpose=True)
            g["dn" + m] = gemm(g[m + "8"], self.wt[m])
            dn += g["dn" + m]
            g["dW" + m] = gemm(g[m + "t"], g["nt"], F32, block=1)
        g["dn"] = dn.to(BF)
        prob = B.NormProblem(T, self.W, B.GDR_BF16, 1e-6)
        g["dx"], g["dw"] = dev(T, self.W, dtype=BF), dev(self.W)
        B.gdr_norm_bwd(prob, r["x"], self.norm, g["dn"], g["dx"], g["dw"], B.alloc_norm_workspace(prob))
        return g


def cpu(pair):
    return pair[0].cpu(), pair[1].cpu()


def same_bytes(name, got, x, block=1):
    q, s = L.quantised(x, block)
    assert torch.equal(got[1].cpu(), s), name
    assert torch.equal(got[0].cpu().view(torch.uint8), q.view(torch.uint8)), name


def product(name, got, a, b, block=128):
    c, err = L.product(*cpu(a), *cpu(b), block, got.dtype)
    R.check(name, got.reshape(c.shape), c, err)


SHAPES = [(256, 4, 2, 64, [70, 0, 129, 1]), (384, 2, 2, 128, [300]), (128, 2, 1, 128, [33, 64])]


@pytest.mark.parametrize("W,H,Hk,D,lengths", SHAPES)
def test_layer(W, H, Hk, D, lengths):
    gen = torch.Generator().manual_seed(W)
    T, layer = sum(lengths), Layer(gen, W, H, Hk, D)
    x, dy = R.rand(gen, T, W).to(BF).cuda(), R.rand(gen, T, W).to(BF).cuda()
    r = layer.forward(x, lengths)
    g = layer.backward(r, dy, lengths)
    torch.cuda.synchronize()
    # the norm's bytes as its scales and quotients allow
    want, rel = R.norm(x.cpu(), None, layer.norm.cpu(), 1e-6)[2:]
    s, z = R.e4m3_ref(want, 128)
    R.check("norm scales", r["n"][1], s, (rel + 2 * R.U) * s)
    assert ((r["n"][0].cpu().float().double() - z).abs() <= (2.0 ** -4 + 4 * rel) * z.abs() + 2.0 ** -10).all()
    for m in "qkv":
        product(m, r["t"][m].view(T, -1), r["n"], layer.w[m])
    t = {n: None if v is None else v.cpu() for n, v in r["t"].items()}
    ref = L.lin(t["q"], t["k"], t["v"], t["log_decay"], None, lengths, 1.0, g["dO"].cpu())
    for m in ("o", "ht"):
        R.check(m, r[m], *ref[m])
    same_bytes("o8", r["o8"], r["o"].view(T, -1).cpu())
    product("y", r["y"], r["o8"], layer.w["o"])
    same_bytes("dy8", g["dy8"], dy.cpu())
    product("dO", g["dO"].view(T, -1), g["dy8"], layer.wt["o"])
    same_bytes("dyt", g["dyt"], dy.t().cpu())
    product("dWo", g["dWo"], g["dyt"], g["ot"], 1)
    for m in "qkv":
        R.check("d" + m, g["d" + m], *ref["d" + m])
        same_bytes(m + "t", g[m + "t"], g["d" + m].view(T, -1).t().cpu())
        product("dn" + m, g["dn" + m], g[m + "8"], layer.wt[m])
        product("dW" + m, g["dW" + m], g[m + "t"], g["nt"], 1)
    dx, dx_err, dw, dw_err = R.norm_bwd(x.cpu(), layer.norm.cpu(), g["dn"].cpu(), None, 1e-6)
    R.check("dx", g["dx"], dx, dx_err)
    R.check("dw", g["dw"], dw, dw_err)


def test_prompt_then_tokens_through_the_layer():
    W, H, Hk, D, lengths = 256, 4, 2, 64, [70, 5, 130]
    gen = torch.Generator().manual_seed(3)
    layer = Layer(gen, W, H, Hk, D)
    r = layer.forward(R.rand(gen, sum(lengths), W).to(BF).cuda(), lengths)
    pool = torch.zeros(7, H, D, D, device="cuda")
    slots = torch.tensor([4, 0, 6], dtype=torch.int32, device="cuda")
    pool[slots.long()] = r["ht"]
    state, prob = r["ht"].cpu(), B.LinProblem(3, 1, H, D, 3, B.GDR_BF16, 1.0, Hk=Hk)
    for i in range(4):
        n, t = layer.project(R.rand(gen, 3, W).to(BF).cuda())
        o = dev(3, H, D, dtype=BF)
        B.gdr_lin_step(prob, t, pool, o, slots=slots)
        o8 = quant(o.view(3, -1))
        y = gemm(o8, layer.w["o"])
        torch.cuda.synchronize()
        c = {m: v.cpu() for m, v in t.items()}
        ref = L.lin(c["q"], c["k"], c["v"], c["log_decay"], state, [1, 1, 1], 1.0)
        R.check(f"o {i}", o, *ref["o"])
        R.check(f"state {i}", pool[slots.long()], *ref["ht"])
        for m in "qkv":
            product(f"{m} {i}", t[m].view(3, -1), n, layer.w[m])
        product(f"y {i}", y, o8, layer.w["o"])
        state = pool[slots.long()].cpu()
    assert not pool[[1, 2, 3, 5]].any()


def test_layer_as_one_graph():
    W, H, Hk, D, lengths = 256, 4, 2, 64, [700, 0, 29, 300]
    gen = torch.Generator().manual_seed(4)
    T, layer = sum(lengths), Layer(gen, W, H, Hk, D)
    x, dy = R.rand(gen, T, W).to(BF).cuda(), R.rand(gen, T, W).to(BF).cuda()

    def go():
        r = layer.forward(x, lengths)
        return r, layer.backward(r, dy, lengths)

    go()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap, cap_g = go()
    for _ in range(4):
        x.copy_(x.flip(0))
        dy.copy_(dy.roll(1, 0))
        r, g = go()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(r["y"], cap["y"]) and torch.equal(r["ht"], cap["ht"])
        for m in ("dx", "dw", "dWq", "dWk", "dWv", "dWo"):
            assert torch.equal(g[m], cap_g[m]), m
        assert torch.isfinite(g["dx"]).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_many_sequences(dtype):
    """More sequences than one launch of the table takes, some empty, some of several
    segments, each as it comes alone."""
    gen = torch.Generator().manual_seed(5)
    H, D = 2, 64
    lengths = [int(n) for n in torch.randint(0, 9, (400,), generator=gen)]
    lengths[7], lengths[130], lengths[399] = 900, 600, 0
    T, N, code = sum(lengths), 400, B.GDR_BF16 if dtype is BF else B.GDR_F32
    t = {m: R.rand(gen, T, H, D, std=D ** -0.5).to(dtype).cuda() for m in "qkv"}
    t["log_decay"], t["h0"] = torch.tensor([-0.02, -0.3]).cuda(), R.rand(gen, N, H, D, D).float().cuda()
    dO, dht = R.rand(gen, T, H, D).to(dtype).cuda(), R.rand(gen, N, H, D, D).float().cuda()

    def run(prob, t, dO, dht):
        ws = B.alloc_lin_workspace(prob, backward=True)
        ws.fill_(255)
        out = {m: torch.full_like(t["v"], float("nan")) for m in ("o", "dq", "dk", "dv")}
        out["ht"], out["dh0"] = torch.full_like(t["h0"], float("nan")), torch.full_like(t["h0"], float("nan"))
        B.gdr_lin_fwd(prob, t, ws, out["o"], ht=out["ht"])
        B.gdr_lin_bwd(prob, t, dO, dht, ws, out)
        return {m: v.cpu() for m, v in out.items()}

    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    got = run(B.LinProblem(1, T, H, D, N, code, 0.5, cu_seqlens=cu), t, dO, dht)
    for n in (0, 6, 7, 8, 119, 120, 121, 130, 239, 240, 398, 399):
        at = slice(cu[n], cu[n + 1])
        part = {m: t[m][at].contiguous() for m in "qkv"}
        c = {m: v.cpu() for m, v in part.items()}
        ref = L.lin(c["q"], c["k"], c["v"], t["log_decay"].cpu(), t["h0"][n:n + 1].cpu(), [lengths[n]], 0.5, dO[at].cpu(), dht[n:n + 1].cpu())
        for m, (value, err) in ref.items():
            R.check(f"{n} {m}", got[m][n:n + 1] if m in ("ht", "dh0") else got[m][at], value, err)
    assert all(torch.isfinite(v).all() for v in got.values())


# ---- offsets beyond 32 bits ----

def test_attention_beyond_32_bits():
    """4.4e9 elements a tensor: the last tokens of the last heads, zeros elsewhere."""
    T, H, D, tail, heads = 134470, 256, 128, 70, 2                   # the tail starts a block
    gen = torch.Generator().manual_seed(1)
    small = {m: R.rand(gen, tail, heads, D, std=D ** -0.5).to(BF) for m in "qkv"}
    g = R.rand(gen, tail, heads, D).to(BF)
    decay = -torch.exp2(-1.0 - 6.0 * torch.rand(H, generator=gen))
    ref = L.lin(small["q"], small["k"], small["v"], decay[-heads:], None, [tail], 1.0, g)

    def big(x):
        y = torch.zeros(T, H, D, dtype=BF, device="cuda")
        y[-tail:, -heads:] = x.cuda()
        return y

    t = {**{m: big(x) for m, x in small.items()}, "log_decay": decay.cuda()}
    assert T % 64 == 6 and t["q"].numel() > 1 << 32
    prob = B.LinProblem(1, T, H, D, 1, B.GDR_BF16, 1.0)
    ws, o, ht = B.alloc_lin_workspace(prob, backward=True), torch.empty_like(t["q"]), dev(1, H, D, D)
    B.gdr_lin_fwd(prob, t, ws, o, ht=ht)
    R.check("o", o[-tail:, -heads:], *ref["o"])
    R.check("ht", ht[:, -heads:], *ref["ht"])
    assert not o[:-tail].any() and not o[:, :-heads].any() and not ht[:, :-heads].any()
    dO, out = big(g), {"dq": o, "dk": torch.empty_like(o), "dv": torch.empty_like(o)}
    B.gdr_lin_bwd(prob, t, dO, None, ws, out)
    for m, x in out.items():
        R.check(m, x[-tail:, -heads:], *ref[m])
        assert not x[:-tail].any() and not x[:, :-heads].any(), m


@pytest.mark.parametrize("T,dtype,Hk", [(65, BF, 1 << 16), (65, BF, 1 << 15), (33, F32, 1 << 16)])
def test_the_most_heads(T, dtype, Hk):
    """2^16 heads: a block's rows reach 2^31 bytes from its first (dq and dk of grouped heads, and
    fp32 tensors).  The last heads' tokens, zeros elsewhere."""
    H, D, heads = 1 << 16, 128, 2
    G, gen = H // Hk, torch.Generator().manual_seed(6)
    hk = heads // G
    small = {m: R.rand(gen, T, heads if m == "v" else hk, D, std=D ** -0.5).to(dtype) for m in "qkv"}
    g, decay = R.rand(gen, T, heads, D).to(dtype), -torch.rand(H, generator=gen)
    ref = L.lin(small["q"], small["k"], small["v"], decay[-heads:], None, [T], 1.0, g)

    def big(x, n):
        y = torch.zeros(T, n, D, dtype=dtype, device="cuda")
        y[:, -x.shape[1]:] = x.cuda()
        return y

    t = {**{m: big(x, H if m == "v" else Hk) for m, x in small.items()}, "log_decay": decay.cuda()}
    prob = B.LinProblem(1, T, H, D, 1, B.GDR_BF16 if dtype is BF else B.GDR_F32, 1.0, Hk=Hk)
    ws, o, dO = B.alloc_lin_workspace(prob, backward=True), torch.full_like(t["v"], float("nan")), big(g, H)
    B.gdr_lin_fwd(prob, t, ws, o)
    out = {m: torch.full_like(t[m[1]], float("nan")) for m in ("dq", "dk", "dv")}
    B.gdr_lin_bwd(prob, t, dO, None, ws, out)
    for m, x in (("o", o), *out.items()):
        n = heads if m in ("o", "dv") else hk
        R.check(m, x[:, -n:], *ref[m])
        assert not x[:, :-n].any(), m


def test_pool_beyond_32_bits():
    N, H, D, P = 3, 16, 128, 16500
    gen = torch.Generator().manual_seed(2)
    t = {m: R.rand(gen, N, H, D).to(BF) for m in "qkv"}
    t["log_decay"], states, slots = -torch.rand(H, generator=gen), R.rand(gen, N, H, D, D).float(), [P - 1, 0, P - 5]
    pool = torch.zeros(P, H, D, D, device="cuda")
    assert pool.numel() > 1 << 32
    for n in range(N):
        pool[slots[n]] = states[n].cuda()
    o = dev(N, H, D, dtype=BF)
    B.gdr_lin_step(B.LinProblem(N, 1, H, D, N, B.GDR_BF16, 0.3), {m: x.cuda() for m, x in t.items()}, pool, o,
                   slots=torch.tensor(slots, dtype=torch.int32, device="cuda"))
    ref = L.lin(t["q"], t["k"], t["v"], t["log_decay"], states, [1] * N, 0.3)
    R.check("o", o, *ref["o"])
    R.check("state", pool[torch.tensor(slots)], *ref["ht"])
    assert not pool[1:P - 5].any() and not pool[P - 4:P - 1].any()


def e4m3_rows(gen, rows, K, last):
    """[rows, K] zeros but for the last rows, and scales for each 128."""
    x = torch.zeros(rows, K, dtype=torch.uint8, device="cuda")
    x[-last:] = R.rand(gen, last, K).to(F8).view(torch.uint8).cuda()
    return x.view(F8), torch.rand(rows, -(-K // 128), generator=gen).cuda()


@pytest.mark.parametrize("M,N,K,dtype", [
    (1050000, 256, 4112, BF),      # rows of 16 bytes
    (1050000, 200, 4111, F32),     # rows through registers
    (4200000, 1040, 128, BF),      # c
    (4200000, 1040, 516, BF),      # c, the largest tiles
    (4200000, 1030, 130, F32),
])
def test_product_beyond_32_bits(M, N, K, dtype):
    gen = torch.Generator().manual_seed(3)
    last = 150
    a, sa = e4m3_rows(gen, M, K, last)
    b, sb = R.rand(gen, N, K).to(F8), torch.rand(-(-N // 128), -(-K // 128), generator=gen)
    assert max(M * N, M * K) > 1 << 32
    c = torch.empty(M, N, dtype=dtype, device="cuda")
    prob = B.GemmProblem(M, N, K, B.GDR_BF16 if dtype is BF else B.GDR_F32)
    B.gdr_gemm(prob, a, sa, b.cuda(), sb.cuda(), c, B.alloc_gemm_workspace(prob))
    R.check("c", c[-last:], *L.product(a[-last:].cpu(), sa[-last:].cpu(), b, sb, 128, dtype))
    assert not c[:-last].any()


@pytest.mark.parametrize("M,N,K", [(130, 20, 1 << 22), (130, 20, (1 << 22) + 4), (40, 300, 1 << 22), (5, 20, (1 << 24) + 1)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_long_contractions(M, N, K, dtype):
    """The longest whose rows go to LDS directly, and longer ones: zeros but for the first and last
    200 of the contraction."""
    gen = torch.Generator().manual_seed(7)
    G, at = -(-K // 128), K % 128 or 128                              # at: of the last group

    def sparse(rows):
        x = torch.zeros(rows, K, dtype=torch.uint8, device="cuda")
        first, last = (R.rand(gen, rows, 200).to(F8) for _ in range(2))
        x[:, :200], x[:, -200:] = first.view(torch.uint8).cuda(), last.view(torch.uint8).cuda()
        s = torch.rand(rows if rows == M else -(-rows // 128), G, generator=gen)
        # the same product over the groups at both ends alone
        y = torch.cat([x[:, :256], x[:, K - at - 256:]], 1).cpu().view(F8)
        return (x.view(F8), s.cuda()), (y, torch.cat([s[:, :2], s[:, -3:]], 1))

    (a, sa), short_a = sparse(M)
    (b, sb), short_b = sparse(N)
    c = dev(M, N, dtype=dtype)
    prob = B.GemmProblem(M, N, K, B.GDR_BF16 if dtype is BF else B.GDR_F32)
    B.gdr_gemm(prob, a, sa, b, sb, c, B.alloc_gemm_workspace(prob))
    R.check("c", c, *L.product(*short_a, *short_b, 128, dtype))


@pytest.mark.parametrize("M,K", [(3, 4112), (32, 4111)])
def test_few_rows_beyond_32_bits(M, K):
    gen = torch.Generator().manual_seed(4)
    N, last = 1050000, 150
    b, sb = e4m3_rows(gen, N, K, last)
    a, sa = R.rand(gen, M, K).to(F8), torch.rand(M, -(-K // 128), generator=gen)
    assert N * K > 1 << 32
    c = dev(M, N, dtype=BF)
    B.gdr_gemm(B.GemmProblem(M, N, K, B.GDR_BF16, block=1), a.cuda(), sa.cuda(), b, sb, c)
    R.check("c", c[:, -last:], *L.product(a, sa, b[-last:].cpu(), sb[-last:].cpu(), 1, BF))
    assert not c[:, :-last].any()


@pytest.mark.parametrize("block,transpose", [(1, False), (1, True), (128, False), (128, True)])
def test_quant_beyond_32_bits(block, transpose):
    gen = torch.Generator().manual_seed(5)
    rows, cols, last = 2100096, 2056, 128                                # the last rows are a tile's
    x = torch.zeros(rows, cols, dtype=BF, device="cuda")
    tail = R.rand(gen, last, cols).to(BF)
    x[-last:] = tail.cuda()
    assert x.numel() > 1 << 32 and rows % 128 == 0
    p = B.QuantProblem(rows, cols, B.GDR_BF16, block=block, transpose=transpose)
    q, s = torch.empty(p.q_shape, dtype=F8, device="cuda"), dev(*p.scales_shape)
    B.gdr_quant(p, x, q, s)
    if transpose:
        same_bytes("tail", (q[:, -last:], s[:, -1:]), tail.t(), block)
        assert not q[:, :-last].view(torch.uint8).any()
    else:
        same_bytes("tail", (q[-last:], s[-last // block:]), tail, block)
        assert not q[:-last].view(torch.uint8).any()
