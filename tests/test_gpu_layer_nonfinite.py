"""Infinities and NaN in the operators around the delta rule: they go where the
formulas take them, token by token, and nowhere else."""

import pytest
import torch

import layer_ref as R
import test_gpu_scan as S

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("kind,dtype", [(1, "f32"), (2, "f32"), (1, "bf16")])
def test_parameter_sums_of_a_ragged_end_take_no_state_after_it(kind, dtype, bad):
    """The last token's input reaches y and ht alone: with a length that ends inside a tile,
    every gradient, those of the gate's parameters among them, is finite."""
    lengths, H, D = [70, 64, 3], 2, 8
    t, dy, dht = S.make(5, kind, dtype, lengths, H, D)
    t["x"][69, 0, 2] = t["x"][136, 1, 3] = bad
    ref = R.scan(kind, t["x"], t["g"], t["A_log"], t["dt_bias"], t["h0"], lengths, S.GS, False, dy, dht)
    got = S.run(S.problem(kind, dtype, lengths, H, D, False, False), S.dev(t), dy.cuda(), dht.cuda(), kind, 3, H, D)
    torch.cuda.synchronize()
    for k in ("dx", "dg", "dh0", "dA_log", "ddt_bias"):
        R.check(k, got[k], *ref[k])
    for k, at in (("y", ((69, 0, 2), (136, 1, 3))), ("ht", ((0, 0, 2), (2, 1, 3)))):
        want = ref[k][0].isnan() if bad != bad else ref[k][0].isinf()
        assert want.sum() == len(at) and all(want[i] for i in at)
        g = got[k].cpu().double()
        assert torch.equal(g.isnan() if bad != bad else g == bad, want)
        R.check(k, torch.where(want, 0.0, g), torch.where(want, 0.0, ref[k][0]), torch.where(want, 0.0, ref[k][1]), got[k].dtype)


# kind, dtype, H, D, convex: a decay per channel, per head, softplus and sigmoid gates
RUNS = [(0, "f32", 5, 1, False), (0, "bf16", 2, 8, False), (0, "f32", 2, 16, True), (1, "bf16", 2, 8, False),
        (2, "f32", 2, 8, True)]


@pytest.mark.parametrize("kind,dtype,H,D,convex", RUNS)
@pytest.mark.parametrize("T", [60, 700, 64 * 40 + 7])
def test_an_infinity_lasts_through_decays_whose_product_underflows(kind, dtype, H, D, convex, T):
    """Strong decays, none of them zero in fp32 (e^-20 a token; the product of six is below
    2^-149): an infinite state stays what it is token by token, within a thread's tokens, a
    tile's groups, a group of tiles and beyond; so does an infinite gradient, backwards."""
    def strong(t):
        if kind == 0:
            t["g"][:] = -20.0
        elif kind == 1:      # softplus(4.5) e^1.5 = 20.2
            t["A_log"][:], t["dt_bias"][:], t["g"][:] = 1.5, 0.0, 4.5
        else:                # 20 sigmoid(6) = 19.95
            t["A_log"][:], t["dt_bias"][:], t["g"][:] = 0.0, 0.0, 6.0
        return t
    gs = -20.0 if kind == 2 else S.GS
    t, dy, dht = S.make(6 + kind, kind, dtype, [T], H, D)
    strong(t)
    prob = S.B.ScanProblem(1, T, H, D, 1, kind, S.CODE[dtype], gate_scale=gs, convex=convex)
    inf = float("inf")

    def go(name, at, value):
        """One infinity in one input; every output against the reference."""
        u = {**t, "dy": dy, "dht": dht}
        u[name] = u[name].clone()
        u[name][at] = value
        ref = R.scan(kind, u["x"], u["g"], u["A_log"], u["dt_bias"], u["h0"], [T], gs, convex, u["dy"], u["dht"])
        d = S.dev(u)
        got = S.run(prob, d, d["dy"], d["dht"], kind, 1, H, D)
        torch.cuda.synchronize()
        for k in ("y", "ht") if name in ("x", "h0") else ("dx", "dg", "dh0"):
            g, (want, err) = got[k].cpu().double(), ref[k]
            assert torch.equal(g.isnan(), want.isnan()), (name, k, int(g.isnan().sum()), int(want.isnan().sum()))
            odd = ~want.isfinite()
            assert torch.equal(g[odd & ~want.isnan()], want[odd & ~want.isnan()]), (name, k)
            z = torch.zeros(())
            R.check(k, torch.where(odd, z.double(), g), torch.where(odd, z.double(), want),
                    torch.where(odd, z.double(), err), got[k].dtype)
        return ref

    ref = go("x", (3, 0, 0), inf)
    assert ref["y"][0][3:, 0, 0].isinf().all()
    go("x", (T - 5, H - 1, D - 1), -inf)
    ref = go("h0", (0, 1, 0), -inf)
    assert ref["ht"][0].isinf().sum() == 1
    ref = go("dy", (T - 7, 0, 0), inf)
    assert ref["dx"][0][:T - 6, 0, 0].isinf().all()
    ref = go("dht", (0, 1, D - 1), -inf)
    assert ref["dh0"][0].isinf().sum() == 1


def test_a_shut_gate_still_cuts():
    """A decay of exactly zero among those that underflow: nothing before it is felt, and an
    infinity before it is 0 * inf = NaN from there on, as token by token."""
    T, H = 900, 3
    t, dy, dht = S.make(9, 0, "f32", [T], H, 1)
    t["g"][:] = -20.0
    t["g"][400] = float("-inf")
    t["x"][2, 1] = float("inf")
    ref = R.scan(0, t["x"], t["g"], None, None, t["h0"], [T], S.GS, False, dy, dht)
    got = S.run(S.problem(0, "f32", [T], H, 1, False, True), S.dev(t), dy.cuda(), dht.cuda(), 0, 1, H, 1)
    torch.cuda.synchronize()
    y = got["y"].cpu()
    assert y[400:, 1].isnan().all() and (y[2:400, 1] == float("inf")).all()
    keep = [0, 2]
    for k in ("y", "dx", "dg"):
        R.check(k, got[k][:, keep], ref[k][0][:, keep], ref[k][1][:, keep])
    assert torch.equal(y[400, keep], t["x"][400, keep])


@pytest.mark.parametrize("kind,dtype", [(0, "f32"), (0, "bf16")])
def test_a_decay_below_the_normal_numbers_is_a_reset(kind, dtype):
    """e^-88 < 2^-126: nothing is left of a state of 1e37, by token, by tile or by step; and
    e^-87 > 2^-126 leaves its share."""
    T, H, B = 300, 2, S.B
    t, dy, dht = S.make(4, kind, dtype, [T], H, 1)
    for lam, left in ((-88.0, False), (-87.0, True)):
        t["g"][:], t["x"][:], t["h0"][:] = 0.0, 0.0, 1e37
        t["g"][0] = lam
        want = torch.tensor(1e37, dtype=torch.float64) * torch.tensor(lam, dtype=torch.float64).exp() if left else 0.0
        got = S.run(S.problem(kind, dtype, [T], H, 1, False, True), S.dev(t), dy.cuda(), dht.cuda(), kind, 1, H, 1)
        state, y = t["h0"].cuda(), torch.full((1, H, 1), float("nan"), dtype=S.DT[dtype], device="cuda")
        one = B.ScanProblem(1, 1, H, 1, 1, kind, S.CODE[dtype])
        B.gdr_scan_step(one, {"x": t["x"][:1].cuda(), "g": t["g"][:1].cuda()}, state, y)
        torch.cuda.synchronize()
        for name, v in (("ht", got["ht"]), ("y", got["y"]), ("state", state)):
            # e^-87: lambda's 87 carries U relative, 8 |lambda| U in the exponential
            ref = torch.full(v.shape, float(want), dtype=torch.float64)
            R.check(name, v, ref, (16 + 8 * 87) * R.U * ref.abs())


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("convex", [False, True])
def test_the_types_lowest_value_masks_as_an_infinity_does(kind, dtype, convex):
    """A gate of the type's lowest or highest value, as masks are written, shuts or opens it
    like -inf or inf does: the same bits in every output."""
    T, H, D = 260, 2, 16
    t, dy, dht = S.make(21, kind, dtype, [T], H, D)
    at = (5, 63, 64, 130, T - 1)
    big = torch.finfo(S.DT[dtype]).max
    outs = []
    for v in (big, float("inf")):
        u = dict(t, g=t["g"].clone())
        for i, r in enumerate(at):
            if kind == 0:
                u["g"][r, i % H] = -v
            else:
                u["g"][r, i % H, 2 * i] = -v if i % 2 else v
        outs.append(S.run(S.problem(kind, dtype, [T], H, D, convex, True), S.dev(u), dy.cuda(), dht.cuda(), kind, 1, H, D))
    torch.cuda.synchronize()
    for k in outs[0]:
        assert torch.isfinite(outs[0][k]).all(), k
        assert torch.equal(outs[0][k], outs[1][k]), k


def test_a_step_with_shut_and_open_gates_of_the_lowest_value():
    """The same for the single-token steps; a beta logit of the lowest value writes nothing."""
    B = S.B
    N, H, D = 4, 2, 64
    gen = torch.Generator().manual_seed(3)
    big = torch.finfo(torch.bfloat16).max
    bf = torch.bfloat16
    for kind in (0, 1, 2):
        g, A, bias = R.gate_inputs(gen, kind, N, H, D, bf)
        t = {"q": R.rand(gen, N, H, D).to(bf), "k": R.rand(gen, N, H, D).to(bf), "v": R.rand(gen, N, H, D).to(bf),
             "x": R.rand(gen, N, H, D).to(bf), "b": R.rand(gen, N, H).to(bf), "A_log": A, "dt_bias": bias}
        states, state = R.rand(gen, N, H, D, D).float(), R.rand(gen, N, H, D).float()
        outs = []
        for v in (big, float("inf")):
            u = {k: None if w is None else w.clone().cuda() for k, w in dict(t, g=g).items()}
            u["g"][1, 0] = -v
            if kind:
                u["g"][2, 1, :8] = v
            u["b"][3, 0] = -v
            o, y = torch.empty(N, H, D, dtype=bf, device="cuda"), torch.empty(N, H, D, dtype=bf, device="cuda")
            St, st = states.cuda(), state.cuda()
            B.gdr_step(B.Problem(N, 1, H, D, N, kind, B.GDR_BF16, 0.125, gate_scale=S.GS if kind == 2 else 0.0), u, St, o)
            B.gdr_scan_step(B.ScanProblem(N, 1, H, D, N, kind, B.GDR_BF16, gate_scale=S.GS, convex=True), u, st, y)
            outs.append((o, y, St, st))
        torch.cuda.synchronize()
        for a, b in zip(*outs):
            assert torch.isfinite(a).all() and torch.equal(a, b)
        # beta = 0: the state only decays, one product
        lam, _, _, rel = (v.expand(1, H, D)[0, 0] for v in R.gate(kind, g[3:], A, bias, S.GS))
        want = states[3, 0].double() * lam.exp()
        R.check("state", outs[0][2][3, 0], want, (rel + 2 * R.U) * want.abs())
