"""Linear attention with a decay for each head (gdr_lin_fwd, gdr_lin_bwd, gdr_lin_step)
through the C ABI against its formulas in 64 bits, element by element within the bounds
of lin_ref."""

import pytest
import torch

from chunked_gated_delta_bwd_amd import binding as B
import layer_ref as R
import lin_ref as L

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
CODE = {"bf16": B.GDR_BF16, "f32": B.GDR_F32}


def make(seed, lengths, H, Hk, D, dtype, h0=True, lam=None):
    gen = torch.Generator().manual_seed(seed)
    dt, T, N = DT[dtype], sum(lengths), len(lengths)
    t = {"q": R.rand(gen, T, Hk, D, std=D ** -0.5).to(dt), "k": R.rand(gen, T, Hk, D, std=D ** -0.5).to(dt),
         "v": R.rand(gen, T, H, D).to(dt),
         "log_decay": -torch.exp2(-1.0 - 9.0 * torch.rand(H, generator=gen)) if lam is None else torch.tensor(lam),
         "h0": R.rand(gen, N, H, D, D, std=0.3).float() if h0 else None}
    return t, R.rand(gen, T, H, D).to(dt), R.rand(gen, N, H, D, D, std=0.3).float()


def problem(lengths, H, Hk, D, dtype, scale, packed=True):
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    if packed:
        return B.LinProblem(1, cu[-1], H, D, len(lengths), CODE[dtype], scale, cu_seqlens=cu, Hk=Hk)
    return B.LinProblem(len(lengths), lengths[0], H, D, len(lengths), CODE[dtype], scale, Hk=Hk)


def nan_like(t):
    return torch.full_like(t, float("nan"), device="cuda")


def buffers(t, dht=True):
    v = t["v"]
    N, (T, H, D) = (t["h0"].shape[0] if t["h0"] is not None else None), v.shape
    return {"o": nan_like(v), "dq": nan_like(t["q"]), "dk": nan_like(t["k"]), "dv": nan_like(v)}


def cuda(t):
    return {n: None if x is None else x.cuda() for n, x in t.items()}


def go(prob, t, dO, dht, out, ws=None):
    """Forward and backward; every byte of the workspace is set before."""
    if ws is None:
        ws = B.alloc_lin_workspace(prob, backward=True)
        ws.fill_(255)
    B.gdr_lin_fwd(prob, t, ws, out["o"], ht=out["ht"])
    B.gdr_lin_bwd(prob, t, dO, dht, ws, out)
    return ws


CASES = [
    # lengths, H, Hk, D, h0, dht, packed
    ([1], 1, 1, 64, True, True, False),
    ([2], 2, 1, 128, False, False, True),
    ([63], 3, 3, 128, True, False, False),
    ([64], 1, 1, 128, True, True, True),
    ([65], 2, 2, 64, False, True, False),
    ([130, 130, 130], 4, 2, 128, True, True, False),
    ([0, 63, 0, 129, 1, 64, 0], 2, 2, 128, True, True, True),
    ([300, 5], 6, 2, 64, True, True, True),
    ([700], 1, 1, 128, True, True, True),
    ([1030, 257, 256], 2, 1, 128, False, True, True),
    ([577, 577], 3, 1, 64, True, True, False),
    ([321], 5, 5, 128, False, False, False),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lengths,H,Hk,D,h0,dht,packed", CASES)
def test_forward_and_backward(lengths, H, Hk, D, h0, dht, packed, dtype):
    t, dO, dS = make(sum(lengths) + H, lengths, H, Hk, D, dtype, h0)
    dS = dS if dht else None
    scale = D ** -0.5 * 3
    ref = L.lin(t["q"], t["k"], t["v"], t["log_decay"], t["h0"], lengths, scale, dO, dS)
    d, out = cuda(t), buffers(t)
    out["ht"] = torch.full((len(lengths), H, D, D), float("nan"), device="cuda")
    out["dh0"] = torch.full_like(out["ht"], float("nan"))
    go(problem(lengths, H, Hk, D, dtype, scale, packed), d, dO.cuda(), None if dS is None else dS.cuda(), out)
    torch.cuda.synchronize()
    for name, (value, err) in ref.items():
        R.check(name, out[name], value, err)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lam", [0.0, -1e-6, -20.0, -1e4, float("-inf"), 0.02])
def test_decays(lam, dtype):
    """No decay, one that rounds away in a token, ones that leave nothing of the state, and growth."""
    lengths, H, D = [400, 70], 2, 64
    t, dO, dht = make(3, lengths, H, H, D, dtype, lam=[lam, -0.01])
    ref = L.lin(t["q"], t["k"], t["v"], t["log_decay"], t["h0"], lengths, 1.0, dO, dht)
    d, out = cuda(t), buffers(t)
    out["ht"], out["dh0"] = nan_like(t["h0"]), nan_like(t["h0"])
    go(problem(lengths, H, H, D, dtype, 1.0), d, dO.cuda(), dht.cuda(), out)
    torch.cuda.synchronize()
    for name, (value, err) in ref.items():
        R.check(name, out[name], value, err)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("packed", [False, True])
def test_what_a_strong_decay_leaves_of_a_state(packed, dtype):
    """Tokens that add nothing: the states alone, decayed to as little as e^-60, to fp32's precision."""
    H, D, scale = 6, 64, 1.0
    lam = [-0.3, -0.8, -6.0, -16.0, -30.0, -60.0]
    lengths = [1, 1, 1] if not packed else [1, 2, 0, 1]
    t, dO, dht = make(19, lengths, H, H, D, dtype, lam=lam)
    t["v"], dO = torch.zeros_like(t["v"]), torch.zeros_like(dO)
    ref = L.lin(t["q"], t["k"], t["v"], t["log_decay"], t["h0"], lengths, scale, dO, dht)
    d, out = cuda(t), buffers(t)
    out["ht"], out["dh0"] = nan_like(t["h0"]), nan_like(t["h0"])
    go(problem(lengths, H, H, D, dtype, scale, packed), d, dO.cuda(), dht.cuda(), out)
    torch.cuda.synchronize()
    for name, (value, err) in ref.items():
        R.check(name, out[name], value, err)


def test_gradients_against_autograd_and_differences():
    lengths, H, Hk, D = [70, 0, 33], 4, 2, 64
    t, dO, dht = make(5, lengths, H, Hk, D, "f32")
    p = {n: x.double().requires_grad_(n != "log_decay") for n, x in t.items()}
    o, ht = L.tokens(p["q"], p["k"], p["v"], p["log_decay"], p["h0"], lengths, 0.7)
    ((o * dO.double()).sum() + (ht * dht.double()).sum()).backward()
    d, out, prob = cuda(t), buffers(t), problem(lengths, H, Hk, D, "f32", 0.7)
    out["ht"], out["dh0"] = nan_like(t["h0"]), nan_like(t["h0"])
    ws = go(prob, d, dO.cuda(), dht.cuda(), out)
    torch.cuda.synchronize()
    ref = L.lin(t["q"], t["k"], t["v"], t["log_decay"], t["h0"], lengths, 0.7, dO, dht)
    for name, g in (("o", o), ("ht", ht), ("dq", p["q"].grad), ("dk", p["k"].grad), ("dv", p["v"].grad), ("dh0", p["h0"].grad)):
        assert (ref[name][0] - g).abs().max() <= 1e-11 * g.abs().max(), name      # the two definitions
        R.check(name, out[name], g.detach(), ref[name][1])
    # central differences of the loss along a direction; the loss is quadratic in v and h0
    # (linear, so exact) and bilinear in q and k: differences of one tensor are exact but
    # for rounding, 1e-7 of the sum of the magnitudes over 2 h
    gen = torch.Generator().manual_seed(9)

    def loss(x):
        y, s = torch.empty_like(out["o"]), torch.empty_like(out["ht"])
        B.gdr_lin_fwd(prob, x, ws, y, ht=s)
        return float((y.double() * dO.cuda().double()).sum() + (s.double() * dht.cuda().double()).sum())

    size = float(((o * dO.double()).abs().sum() + (ht * dht.double()).abs().sum()).detach())
    for name in ("q", "k", "v", "h0"):
        u, h = torch.randn(t[name].shape, generator=gen), 0.5
        up, down = dict(d), dict(d)
        up[name], down[name] = (t[name] + h * u).cuda(), (t[name] - h * u).cuda()
        num = (loss(up) - loss(down)) / (2 * h)
        ana = float((out["d" + name].double().cpu() * u.double()).sum())
        assert abs(num - ana) <= 4e-5 * size, name


@pytest.mark.parametrize("dtype,D,H,Hk", [("bf16", 128, 4, 2), ("f32", 64, 3, 3), ("bf16", 64, 2, 1), ("f32", 128, 2, 2)])
def test_step(dtype, D, H, Hk):
    """Slots in any order, padding rows on both sides of the pool, rows that share a slot."""
    P, N = 9, 12
    slots = torch.tensor([3, -1, 0, 3, 8, 9, 2, 3, 2000000000, 8, 5, -7], dtype=torch.int32)
    t, _, _ = make(7, [N], H, Hk, D, dtype, h0=False)
    gen = torch.Generator().manual_seed(8)
    pool = R.rand(gen, P, H, D, D).float()
    d = cuda(t)
    o, state = torch.full((N, H, D), 7.0, dtype=DT[dtype], device="cuda"), pool.cuda()
    B.gdr_lin_step(B.LinProblem(N, 1, H, D, N, CODE[dtype], 0.5, Hk=Hk), d, state, o, slots=slots.cuda())
    torch.cuda.synchronize()
    S, err = pool.double(), torch.zeros(P, H, D, D, dtype=torch.float64)
    want, want_err = torch.full((N, H, D), 7.0, dtype=torch.float64), torch.zeros(N, H, D, dtype=torch.float64)
    q, k = (t[x].double().repeat_interleave(H // Hk, 1) for x in ("q", "k"))
    a = t["log_decay"].double().exp()[:, None, None]
    for n, s in enumerate(slots.tolist()):
        if not 0 <= s < P:
            continue
        add = t["v"][n].double()[:, :, None] * k[n][:, None, :]
        err[s] = a * err[s] + 8 * R.U * (a * S[s].abs() + add.abs())
        S[s] = a * S[s] + add
        want[n] = 0.5 * (S[s] * q[n][:, None, :]).sum(-1)
        want_err[n] = 0.5 * ((err[s] + D * R.U * S[s].abs()) * q[n].abs()[:, None, :]).sum(-1)
    R.check("state", state, S, err)
    R.check("o", o, want, want_err)
    off = [n for n, s in enumerate(slots.tolist()) if not 0 <= s < P]
    assert (o[off] == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_then_tokens(dtype):
    """A prompt's final states as the pool, then single tokens: as the whole sequence."""
    H, Hk, D, prompt, more = 4, 2, 64, [70, 1, 130], 5
    lengths = [p + more for p in prompt]
    t, _, _ = make(11, lengths, H, Hk, D, dtype)
    ref = L.lin(t["q"], t["k"], t["v"], t["log_decay"], t["h0"], lengths, 1.0)
    start = [sum(lengths[:n]) for n in range(3)]
    idx = torch.cat([torch.arange(s, s + p) for s, p in zip(start, prompt)])
    d = cuda({n: x if n in ("log_decay", "h0") else x[idx].contiguous() for n, x in t.items()})
    o, pool = nan_like(t["v"][idx]), nan_like(t["h0"])
    prob = problem(prompt, H, Hk, D, dtype, 1.0)
    B.gdr_lin_fwd(prob, d, B.alloc_lin_workspace(prob), o, ht=pool)
    torch.cuda.synchronize()
    R.check("prompt o", o, ref["o"][0][idx], ref["o"][1][idx])
    step = B.LinProblem(3, 1, H, D, 3, CODE[dtype], 1.0, Hk=Hk)
    for i in range(more):
        at = torch.tensor([s + p + i for s, p in zip(start, prompt)])
        d = cuda({n: x[at].contiguous() for n, x in t.items() if n in "qkv"})
        d["log_decay"] = t["log_decay"].cuda()
        y = nan_like(t["v"][at])
        B.gdr_lin_step(step, d, pool, y)
        torch.cuda.synchronize()
        R.check(f"token {i}", y, ref["o"][0][at], ref["o"][1][at])
    R.check("states", pool, ref["ht"][0], ref["ht"][1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("name", ["q", "k", "v", "dO"])
def test_infinities_and_nan_stay_behind_their_token(name, bad, dtype):
    """Other heads, other sequences and the tokens on the other side keep their bits."""
    lengths, H, D, at = [300, 200, 64], 2, 128, 300 + 70
    t, dO, dht = make(13, lengths, H, H, D, dtype)
    prob = problem(lengths, H, H, D, dtype, 1.0)

    def run(x, g):
        out = buffers(t)
        out["ht"], out["dh0"] = nan_like(t["h0"]), nan_like(t["h0"])
        go(prob, cuda(x), g.cuda(), dht.cuda(), out)
        torch.cuda.synchronize()
        return {n: v.cpu() for n, v in out.items()}

    clean = run(t, dO)
    x, g = {n: v.clone() for n, v in t.items()}, dO.clone()
    (g if name == "dO" else x[name])[at, 1, 5] = bad
    got = run(x, g)
    T, seq = sum(lengths), torch.zeros(sum(lengths), dtype=torch.bool)
    seq[300:500] = True
    i = torch.arange(T)
    # tokens that the changed one may reach: itself, later ones of its sequence, or earlier ones
    here, later, earlier = i == at, seq & (i >= at), seq & (i <= at)
    reach = {"q": {"o": here, "dq": None, "dk": earlier, "dv": earlier}, "k": {"o": later, "dq": later, "dk": None, "dv": here},
             "v": {"o": later, "dq": later, "dk": here, "dv": None}, "dO": {"o": None, "dq": here, "dk": earlier, "dv": earlier}}
    for out, rows in reach[name].items():
        keep = torch.ones(T, H, dtype=torch.bool)
        if rows is not None:
            keep[rows, 1] = False
        assert torch.equal(got[out][keep], clean[out][keep]), (name, out)
        if rows is not None:
            assert not torch.isfinite(got[out][rows, 1]).all(-1).any(), (name, out)
    for out, touched in (("ht", name in "kv"), ("dh0", name in ("q", "dO"))):
        keep = torch.ones(3, H, dtype=torch.bool)
        keep[1, 1] = not touched
        assert torch.equal(got[out][keep], clean[out][keep]), (name, out)
        assert torch.isfinite(got[out][1, 1]).all() != touched


def test_streams_graphs_and_two_calls_at_once():
    lengths, H, Hk, D = [900, 30, 300], 4, 2, 128
    t, dO, dht = make(17, lengths, H, Hk, D, "bf16")
    prob, d, dO, dht = problem(lengths, H, Hk, D, "bf16", 1.0), cuda(t), dO.cuda(), dht.cuda()

    def new():
        out = buffers(t)
        out["ht"], out["dh0"] = nan_like(t["h0"]), nan_like(t["h0"])
        return out

    same = lambda a, b: all(torch.equal(a[n], b[n]) for n in a)  # noqa: E731
    ref = new()
    go(prob, d, dO, dht, ref)
    s1, s2, a, b = torch.cuda.Stream(), torch.cuda.Stream(), new(), new()
    w1, w2 = B.alloc_lin_workspace(prob, backward=True), B.alloc_lin_workspace(prob, backward=True)
    torch.cuda.synchronize()
    for s, out, ws in ((s1, a, w1), (s2, b, w2)):
        with torch.cuda.stream(s):
            go(prob, d, dO, dht, out, ws)
    torch.cuda.synchronize()
    assert same(ref, a) and same(ref, b)
    cap, pool, step_o = new(), d["h0"].clone(), nan_like(d["v"][:3])
    step = B.LinProblem(3, 1, H, D, 3, B.GDR_BF16, 1.0, Hk=Hk)
    first = {"q": d["q"][:3], "k": d["k"][:3], "v": d["v"][:3], "log_decay": d["log_decay"]}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(prob, d, dO, dht, cap, w1)
        B.gdr_lin_step(step, first, pool, step_o)
    for _ in range(4):
        d["v"].copy_(d["v"].flip(0))
        go(prob, d, dO, dht, ref, w2)
        want = pool.clone()
        y = torch.empty_like(step_o)
        B.gdr_lin_step(step, first, want, y)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert same(ref, cap) and torch.equal(pool, want) and torch.equal(step_o, y)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_states_not_asked_for_and_a_second_backward(dtype):
    """Without ht and dh0 everything is within the same bounds (fp32: the same bits); a second
    backward on the same workspace gives the same bits."""
    lengths, H, Hk, D = [700, 64, 3], 4, 2, 128
    t, dO, dht = make(23, lengths, H, Hk, D, dtype)
    ref = L.lin(t["q"], t["k"], t["v"], t["log_decay"], t["h0"], lengths, 1.0, dO, dht)
    prob, d, dO, dht = problem(lengths, H, Hk, D, dtype, 1.0), cuda(t), dO.cuda(), dht.cuda()
    full, bare, again = buffers(t), buffers(t), buffers(t)
    full["ht"], full["dh0"] = nan_like(t["h0"]), nan_like(t["h0"])
    ws = go(prob, d, dO, dht, full)
    again["dh0"] = nan_like(t["h0"])
    B.gdr_lin_bwd(prob, d, dO, dht, ws, again)
    ws.fill_(255)
    B.gdr_lin_fwd(prob, d, ws, bare["o"])
    B.gdr_lin_bwd(prob, d, dO, dht, ws, bare)
    torch.cuda.synchronize()
    for m in ("dq", "dk", "dv", "dh0"):
        assert torch.equal(full[m], again[m]), m
    for m, x in bare.items():
        R.check(m, x, *ref[m])
        assert dtype == "bf16" or torch.equal(full[m], x), m


def test_no_tokens():
    t, _, dht = make(1, [0, 0], 2, 2, 64, "f32")
    for packed in (True, False):
        prob, d = problem([0, 0], 2, 2, 64, "f32", 1.0, packed), cuda(t)
        out = buffers(t)
        out["ht"], out["dh0"] = nan_like(t["h0"]), nan_like(t["h0"])
        go(prob, d, out["o"], dht.cuda(), out)
        torch.cuda.synchronize()
        assert torch.equal(out["ht"].cpu(), t["h0"]) and torch.equal(out["dh0"].cpu(), dht)
    none = B.LinProblem(1, 0, 2, 64, 1, B.GDR_F32, 1.0)
    e = torch.empty(0, 2, 64, device="cuda")
    ht = torch.ones(1, 2, 64, 64, device="cuda")
    B.gdr_lin_fwd(none, {"q": e, "k": e, "v": e, "log_decay": d["log_decay"]}, B.alloc_lin_workspace(none), e, ht=ht)
    torch.cuda.synchronize()
    assert not ht.any()
