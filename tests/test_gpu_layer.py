"""The operators together, as a layer uses them: residual norm, gated linear recurrence,
norm of the delta rule's output per head, forward and backward, against 64-bit autograd
through the same formulas; and in serving, prompt and then single tokens."""

import pytest
import torch

import oracle
from chunked_gated_delta_bwd_amd import binding as B
from chunked_gated_delta_bwd_amd import synth
import layer_ref as R

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

EPS, GS = 1e-6, -2.0


def rel(a, b):
    return float((a.cpu().double() - b).norm() / b.norm())


def test_residual_norm_then_recurrence_forward_and_backward():
    """r = x + res; y = rmsnorm(r) w; s = scan(y, g); loss = <ds, s> + <dres, r>, in fp32:
    every gradient against autograd in 64 bits."""
    lengths, H, D = [90, 0, 41], 3, 64
    T, C = sum(lengths), H * D
    gen = torch.Generator().manual_seed(1)
    x, res, w = R.rand(gen, T, C).float(), R.rand(gen, T, C).float(), (1 + 0.2 * R.rand(gen, C)).float()
    g, A, bias = R.gate_inputs(gen, 1, T, H, D, torch.float32)
    h0, ds, dres, dht = (R.rand(gen, *sh).float() for sh in ((3, H, D), (T, C), (T, C), (3, H, D)))
    # 64 bits, by autograd
    p = {k: v.double().requires_grad_() for k, v in dict(x=x, res=res, w=w, g=g, A=A, bias=bias, h0=h0).items()}
    r = p["x"] + p["res"]
    y = r / (r.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * p["w"]
    lam = -p["A"].exp()[:, None] * torch.nn.functional.softplus(p["g"] + p["bias"], threshold=1e3)
    a, u = lam.exp(), -torch.expm1(lam) * y.view(T, H, D)
    rows, at, loss = [], 0, (r * dres.double()).sum()
    for n, L in enumerate(lengths):
        s = p["h0"][n]
        for t in range(at, at + L):
            s = a[t] * s + u[t]
            rows.append(s)
        loss = loss + (s * dht[n].double()).sum()
        at += L
    s64 = torch.stack(rows).view(T, C)
    loss = loss + (s64 * ds.double()).sum()
    loss.backward()
    # the library
    c = lambda t: t.cuda()  # noqa: E731
    np_, sp = B.NormProblem(T, C, B.GDR_F32, EPS), B.ScanProblem(1, T, H, D, 3, 1, B.GDR_F32, [0, 90, 90, 131], convex=True)
    yd, rd, s, ht = torch.empty(T, C, device="cuda"), torch.empty(T, C, device="cuda"), torch.empty(T, C, device="cuda"), None
    wd, nws, sws = c(w), B.alloc_norm_workspace(np_), B.alloc_scan_workspace(sp)
    B.gdr_norm_fwd(np_, c(x), wd, yd, res=c(res), res_out=rd)
    t = {"x": yd, "g": c(g), "A_log": c(A), "dt_bias": c(bias), "h0": c(h0)}
    B.gdr_scan_fwd(sp, t, sws, s, ht=ht)
    out = {"dx": torch.empty_like(yd), "dg": torch.empty_like(t["g"]), "dh0": torch.empty_like(t["h0"]),
           "dA_log": torch.empty_like(t["A_log"]), "ddt_bias": torch.empty_like(t["dt_bias"])}
    B.gdr_scan_bwd(sp, t, c(ds), c(dht), sws, out)
    dx, dw = torch.empty_like(yd), torch.empty_like(wd)
    B.gdr_norm_bwd(np_, rd, wd, out["dx"], dx, dw, nws, dres=c(dres))
    torch.cuda.synchronize()
    # fp32 throughout: a relative error of some 1e-6 in the norm
    for name, got, want in (("s", s, s64.detach()), ("dx", dx, p["x"].grad), ("dres", dx, p["res"].grad),
                            ("dw", dw, p["w"].grad), ("dg", out["dg"], p["g"].grad), ("dA_log", out["dA_log"], p["A"].grad),
                            ("ddt_bias", out["ddt_bias"], p["bias"].grad), ("dh0", out["dh0"], p["h0"].grad)):
        assert rel(got.view(want.shape), want) <= 2e-5, (name, rel(got.view(want.shape), want))


def test_delta_rule_then_head_norm_forward_and_backward():
    """o = gdr_fwd; y = rmsnorm over each head's channels; its backward's dx is the dO of
    gdr_bwd: the delta rule's gradients then equal the oracle's for that dO."""
    H, D = 3, 64
    inp = synth.generate(synth.Spec("ln", 0, "f32", H=H, K=D, V=D, lengths=[100, 37], h0_std=0.2, seed=3))
    T = inp["T"]
    prob, d = B.Problem.from_inputs(inp), B.to_device(inp)
    ws, o, out = B.alloc_workspace(prob), torch.empty_like(d["v"]), B.alloc_outputs(inp, d)
    B.gdr_fwd(prob, d, ws, o)
    gen = torch.Generator().manual_seed(2)
    w, dy = (1 + 0.2 * R.rand(gen, D)).float(), R.rand(gen, T * H, D).float()
    nprob = B.NormProblem(T * H, D, B.GDR_F32, EPS)
    y, dO, dw = torch.empty_like(o), torch.empty_like(o), torch.empty(D, device="cuda")
    B.gdr_norm_fwd(nprob, o, w.cuda(), y)
    B.gdr_norm_bwd(nprob, o, w.cuda(), dy.cuda(), dO, dw, B.alloc_norm_workspace(nprob))
    B.gdr_bwd(prob, d, dO, None, ws, out)
    torch.cuda.synchronize()
    o64 = o.cpu().double().view(T * H, D)
    _, _, y64, _ = R.norm(o64, None, w, EPS)
    dx64, _, dw64, _ = R.norm_bwd(o64, w, dy, None, EPS)
    assert rel(y.view(T * H, D), y64) <= 1e-6 and rel(dO.view(T * H, D), dx64) <= 1e-6 and rel(dw, dw64) <= 1e-6
    ref = oracle.run({**inp, "dO": dO.cpu()})
    for k in ("dq", "dk", "dv", "dg", "db"):
        assert rel(out[k], torch.from_numpy(ref[k])) <= 2e-2, k


def test_serving_a_prompt_and_then_tokens():
    """Two requests on scattered slots of both pools: prompts through the forwards, then
    three tokens through norm, recurrence step and delta step, with a padding row, equal
    the same tokens appended to the prompts."""
    H, D, P, more, lengths = 2, 64, 5, 3, [70, 33]
    slots, C = [4, 1], 128
    gen = torch.Generator().manual_seed(4)
    full = [L + more for L in lengths]
    x, w = [R.rand(gen, L, C).float() for L in full], (1 + 0.2 * R.rand(gen, C)).float()
    lg = [(-0.1 * torch.rand(L, H, generator=gen)) for L in full]
    rest = [{k: R.rand(gen, L, H, D).float() for k in ("q", "k")} | {"b": R.rand(gen, L, H).float()} for L in full]

    def forward(seqs, upto):
        """norm -> recurrence -> delta rule with v = the recurrence's output."""
        lens = [u for u in upto]
        T, cu = sum(lens), [0, lens[0], sum(lens)]
        cat = lambda f: torch.cat([f(i)[:lens[i]] for i in range(2)]).contiguous().cuda()  # noqa: E731
        y, s = torch.empty(T, C, device="cuda"), torch.empty(T, C, device="cuda")
        B.gdr_norm_fwd(B.NormProblem(T, C, B.GDR_F32, EPS), cat(lambda i: x[i]), w.cuda(), y)
        sp = B.ScanProblem(1, T, H, D, 2, 0, B.GDR_F32, cu, convex=True)
        ht = torch.empty(2, H, D, device="cuda")
        g = cat(lambda i: lg[i])
        B.gdr_scan_fwd(sp, {"x": y, "g": g}, B.alloc_scan_workspace(sp), s, ht=ht)
        dp = B.Problem(1, T, H, D, 2, 0, B.GDR_F32, 0.125, cu_seqlens=cu)
        o, St = torch.empty(T, H, D, device="cuda"), torch.empty(2, H, D, D, device="cuda")
        t = {"q": cat(lambda i: rest[i]["q"]), "k": cat(lambda i: rest[i]["k"]), "v": s, "g": g, "b": cat(lambda i: rest[i]["b"])}
        B.gdr_fwd(dp, t, B.alloc_workspace(dp), o, ht=St)
        torch.cuda.synchronize()
        return s, ht, o, St

    s_all, ht_all, o_all, St_all = forward(x, full)
    _, ht, _, St = forward(x, lengths)
    pool, Pool = torch.zeros(P, H, D, device="cuda"), torch.zeros(P, H, D, D, device="cuda")
    at = torch.tensor(slots, device="cuda")
    pool[at], Pool[at] = ht, St
    rows = torch.tensor(slots + [-1], dtype=torch.int32, device="cuda")
    ends = [full[0], full[0] + full[1]]
    for j in range(more):
        tok = lambda f: torch.cat([f(i)[lengths[i] + j][None] for i in range(2)] + [f(0)[:1]]).contiguous().cuda()  # noqa: E731
        y, s = torch.empty(3, C, device="cuda"), torch.zeros(3, C, device="cuda")
        B.gdr_norm_fwd(B.NormProblem(3, C, B.GDR_F32, EPS), tok(lambda i: x[i]), w.cuda(), y)
        g = tok(lambda i: lg[i])
        B.gdr_scan_step(B.ScanProblem(3, 1, H, D, 3, 0, B.GDR_F32, convex=True), {"x": y, "g": g}, pool, s, slots=rows)
        o = torch.zeros(3, H, D, device="cuda")
        t = {"q": tok(lambda i: rest[i]["q"]), "k": tok(lambda i: rest[i]["k"]), "v": s, "g": g, "b": tok(lambda i: rest[i]["b"])}
        B.gdr_step(B.Problem(3, 1, H, D, 3, 0, B.GDR_F32, 0.125), t, Pool, o, slots=rows)
        torch.cuda.synchronize()
        for i in range(2):
            k = ends[i] - more + j
            assert rel(s[i], s_all[k].cpu().double()) <= 1e-5
            # the chunked forward multiplies in bf16 (the bar its own tests hold it to); the step is fp32
            assert rel(o[i], o_all[k].cpu().double()) <= 2e-2
        assert not s[2].any() and not o[2].any()
    assert rel(pool[at], ht_all.cpu().double()) <= 1e-5 and rel(Pool[at], St_all.cpu().double()) <= 2e-2
    idle = [p for p in range(P) if p not in slots]
    assert not pool[idle].any() and not Pool[idle].any()
