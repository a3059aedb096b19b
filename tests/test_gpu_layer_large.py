"""The operators around the delta rule where element offsets pass 32 bits, and two calls
at once on streams and workspaces of their own.  Mostly zeros; a few rows or channels
far out are checked against 64 bits."""

import pytest
import torch

from chunked_gated_delta_bwd_amd import binding as B
import layer_ref as R

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

BF = torch.bfloat16


def test_norm_beyond_32_bits():
    rows, width, last = 66000, 32768, 3          # 2.16e9 elements
    gen = torch.Generator().manual_seed(1)
    tail, dy_tail, w = R.rand(gen, last, width).to(BF), R.rand(gen, last, width).to(BF), (1 + 0.2 * R.rand(gen, width)).float()
    x, dy = torch.zeros(rows, width, dtype=BF, device="cuda"), torch.zeros(rows, width, dtype=BF, device="cuda")
    x[-last:], dy[-last:] = tail.cuda(), dy_tail.cuda()
    prob = B.NormProblem(rows, width, B.GDR_BF16, 1e-6)
    y = torch.empty_like(x)
    B.gdr_norm_fwd(prob, x, w.cuda(), y)
    _, _, want, rel = R.norm(tail, None, w, 1e-6)
    R.check("y", y[-last:], want, rel * want.abs())
    assert not y[:-last].any()
    dw = torch.empty(width, device="cuda")
    B.gdr_norm_bwd(prob, x, w.cuda(), dy, y, dw, B.alloc_norm_workspace(prob))
    dx, dx_err, dw_ref, dw_err = R.norm_bwd(tail, w, dy_tail, None, 1e-6)
    R.check("dx", y[-last:], dx, dx_err)
    R.check("dw", dw, dw_ref, dw_err)
    del y
    q, s = torch.empty(rows, width, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(rows, 256, device="cuda")
    B.gdr_norm_quant(B.NormProblem(rows, width, B.GDR_BF16, 1e-6, group=128), x, w.cuda(), q, s)
    s_ref, z = R.e4m3_ref(want, 128)
    R.check("scales", s[-last:], s_ref, (rel + 2 * R.U) * s_ref)
    assert ((q[-last:].cpu().float().double() - z).abs() <= (2.0 ** -4 + 4 * rel) * z.abs() + 2.0 ** -10).all()


@pytest.mark.parametrize("T,H,D", [(1030, 1 << 21, 1), (67000, 256, 128)])
def test_scan_beyond_32_bits(T, H, D):
    """2.2e9 elements: the most channels there may be, and a long sequence."""
    C, keep = H * D, 8
    gen = torch.Generator().manual_seed(2)
    tail = min(T, 300)
    xs, gs = R.rand(gen, tail, keep).to(BF), (-0.1 * torch.rand(tail, keep // min(D, keep), generator=gen)).to(BF)
    dys = R.rand(gen, tail, keep).to(BF)
    x, dy = torch.zeros(T, C, dtype=BF, device="cuda"), torch.zeros(T, C, dtype=BF, device="cuda")
    g = torch.zeros(T, H, dtype=BF, device="cuda")
    x[-tail:, -keep:], dy[-tail:, -keep:] = xs.cuda(), dys.cuda()
    g[-tail:, -gs.shape[1]:] = gs.cuda()
    prob = B.ScanProblem(1, T, H, D, 1, 0, B.GDR_BF16)
    ws, y, ht = B.alloc_scan_workspace(prob), torch.empty_like(x), torch.empty(H, D, device="cuda")
    B.gdr_scan_fwd(prob, {"x": x, "g": g}, ws, y, ht=ht)
    # the last channels: heads of one channel, or the last head's last ones
    heads, d = (keep, 1) if D == 1 else (1, keep)
    ref = R.scan(0, xs.view(tail, heads, d), gs, None, None, None, [tail], 0.0, False, dys.view(tail, heads, d))
    R.check("y", y[-tail:, -keep:].reshape(tail, heads, d), *ref["y"])
    R.check("ht", ht.view(-1)[-keep:].view(1, heads, d), *ref["ht"])
    assert not y[:, :-keep].any()
    out = {"dx": y, "dg": torch.empty_like(g)}
    B.gdr_scan_bwd(prob, {"x": x, "g": g}, dy, None, ws, out)
    R.check("dx", y[-tail:, -keep:].reshape(tail, heads, d), *ref["dx"])
    R.check("dg", out["dg"][-tail:, -heads:], *ref["dg"])


def test_pools_beyond_32_bits():
    """Slots at the end of pools of more than 2^31 elements."""
    N, H, D, P = 3, 16, 128, 8300
    gen = torch.Generator().manual_seed(3)
    g, _, _ = R.gate_inputs(gen, 0, N, H, D, torch.float32)
    t = {"q": R.rand(gen, N, H, D).float(), "k": R.rand(gen, N, H, D).float(), "v": R.rand(gen, N, H, D).float(), "g": g,
         "b": R.rand(gen, N, H).float()}
    states, slots = R.rand(gen, N, H, D, D, std=0.5).float(), [P - 1, 0, P - 5]
    pool = torch.zeros(P, H, D, D, device="cuda")
    assert pool.numel() > 1 << 31
    for n in range(N):
        pool[slots[n]] = states[n].cuda()
    o = torch.empty(N, H, D, device="cuda")
    prob = B.Problem(N, 1, H, D, N, 0, B.GDR_F32, 0.1)
    B.gdr_step(prob, {k: v.cuda() for k, v in t.items()}, pool, o, slots=torch.tensor(slots, dtype=torch.int32, device="cuda"))
    want, err, _, S, S_err = R.step_delta(0, t["q"], t["k"], t["v"], t["g"], t["b"], None, None, states, list(range(N)), 0.1)
    R.check("o", o, want, err)
    R.check("state", pool[torch.tensor(slots)], S, S_err)
    assert not pool[1:P - 5].any()
    del pool
    C, P = 1 << 19, 4200
    pool = torch.zeros(P, C, 1, device="cuda")
    assert pool.numel() > 1 << 31
    x = torch.zeros(2, C, 1, dtype=BF, device="cuda")
    x[:, -8:] = 1.5
    y = torch.empty_like(x)
    sp = B.ScanProblem(2, 1, C, 1, 2, 0, B.GDR_BF16)
    B.gdr_scan_step(sp, {"x": x, "g": torch.zeros(2, C, dtype=BF, device="cuda")}, pool, y,
                    slots=torch.tensor([P - 1, 1], dtype=torch.int32, device="cuda"))
    assert torch.equal(y, x) and (pool[P - 1, -8:] == 1.5).all() and (pool[1, -8:] == 1.5).all()
    assert not pool[2:P - 1].any()


def test_two_calls_at_once():
    """Two recurrences on two streams, each with its workspace, running together, give what
    each gives alone."""
    T, H, D = 20000, 4, 128
    prob = B.ScanProblem(1, T, H, D, 1, 1, B.GDR_BF16, convex=True)
    sets = []
    for seed in (1, 2):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
        sets.append(({"x": r(T, H, D).to(BF), "g": r(T, H, D).to(BF), "A_log": r(H) - 5, "dt_bias": r(H, D), "h0": r(1, H, D)},
                     r(T, H, D).to(BF), B.alloc_scan_workspace(prob)))

    def outputs(t):
        return {"y": torch.empty_like(t["x"]), "dx": torch.empty_like(t["x"]), "dg": torch.empty_like(t["g"]),
                "dh0": torch.empty_like(t["h0"]), "dA_log": torch.empty_like(t["A_log"]), "ddt_bias": torch.empty_like(t["dt_bias"])}

    def go(s, o):
        t, dy, ws = s
        B.gdr_scan_fwd(prob, t, ws, o["y"])
        B.gdr_scan_bwd(prob, t, dy, None, ws, o)

    alone = [outputs(s[0]) for s in sets]
    for s, o in zip(sets, alone):
        go(s, o)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        together = [outputs(s[0]) for s in sets]
        torch.cuda.synchronize()
        for stream, s, o in zip(streams, sets, together):
            with torch.cuda.stream(stream):
                go(s, o)
        torch.cuda.synchronize()
        for a, b in zip(alone, together):
            for k in a:
                assert torch.equal(a[k], b[k]), k
