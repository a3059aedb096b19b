"""The gated linear recurrence (gdr_scan_fwd, gdr_scan_bwd, gdr_scan_step) through the
C ABI against the token-by-token recurrence in 64 bits, element by element within
the running error bound of layer_ref."""

import pytest
import torch

from chunked_gated_delta_bwd_amd import binding as B
import layer_ref as R

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
CODE = {"bf16": B.GDR_BF16, "f32": B.GDR_F32}
GS = -2.0


def make(seed, kind, dtype, lengths, H, D, h0=True, dense=None):
    gen = torch.Generator().manual_seed(seed)
    dt, tokens, N = DT[dtype], sum(lengths), len(lengths)
    g, A, bias = R.gate_inputs(gen, kind, tokens, H, D, dt)
    t = {"x": R.rand(gen, tokens, H, D).to(dt), "g": g, "A_log": A, "dt_bias": bias,
         "h0": R.rand(gen, N, H, D).float() if h0 else None}
    dy = R.rand(gen, tokens, H, D).to(dt)
    dht = R.rand(gen, N, H, D).float() if h0 else None
    return t, dy, dht


def dev(t):
    return {k: None if v is None else v.cuda() for k, v in t.items()}


def problem(kind, dtype, lengths, H, D, convex, dense):
    N = len(lengths)
    if dense:
        assert len(set(lengths)) == 1
        return B.ScanProblem(N, lengths[0], H, D, N, kind, CODE[dtype], gate_scale=GS, convex=convex)
    cu = [0]
    for L in lengths:
        cu.append(cu[-1] + L)
    return B.ScanProblem(1, cu[-1], H, D, N, kind, CODE[dtype], cu_seqlens=cu, gate_scale=GS, convex=convex)


def outputs(d, kind, N, H, D, dh0=True):
    nan = float("nan")
    full = lambda ref: torch.full_like(ref, nan)  # noqa: E731
    out = {"dx": full(d["x"]), "dg": full(d["g"]),
           "dh0": torch.full((N, H, D), nan, device="cuda") if dh0 else None}
    if kind:
        out["dA_log"], out["ddt_bias"] = full(d["A_log"]), full(d["dt_bias"])
    return out


def run(prob, d, dy, dht, kind, N, H, D, ws=None, stream=None):
    ws = B.alloc_scan_workspace(prob) if ws is None else ws
    y = torch.full_like(d["x"], float("nan"))
    ht = torch.full((N, H, D), float("nan"), device="cuda")
    out = outputs(d, kind, N, H, D)
    B.gdr_scan_fwd(prob, d, ws, y, ht=ht, stream=stream)
    B.gdr_scan_bwd(prob, d, dy, dht, ws, out, stream=stream)
    return {"y": y, "ht": ht, **{k: v for k, v in out.items() if v is not None}}


def compare(got, ref):
    assert set(got) == set(ref)
    for k in ref:
        R.check(k, got[k], *ref[k])


# tile 128 tokens; 128-channel tiles of 16-byte vectors; heads that fill a tile,
# share one, straddle none; odd channel counts take the one-channel lanes
CASES = [
    # kind, dtype, lengths, H, D, convex, dense, h0
    (1, "bf16", [300], 2, 128, False, True, True),
    (1, "f32", [300], 2, 128, True, True, True),
    (2, "bf16", [129, 129], 3, 64, True, True, True),
    (2, "f32", [127, 127], 1, 64, False, True, False),
    (0, "bf16", [257], 2, 128, True, True, True),
    (0, "f32", [257], 2, 128, False, True, True),
    (0, "bf16", [1, 127, 128, 129, 0, 400], 3, 64, True, False, True),
    (1, "bf16", [1, 127, 128, 129, 0, 400], 3, 64, False, False, True),
    (2, "f32", [0, 5, 0, 0, 260, 1, 0], 2, 8, True, False, True),
    (0, "bf16", [200, 60], 5, 1, False, False, True),     # odd channel count: one channel a lane
    (0, "f32", [130], 7, 1, True, True, False),
    (1, "bf16", [140], 67, 1, True, True, True),
    (2, "f32", [140], 67, 1, False, True, True),
    (0, "bf16", [150], 264, 1, True, True, True),         # per-channel decays, three tiles, the last ragged
    (0, "bf16", [200], 7, 40, True, True, True),           # three heads a tile, lanes left over
    (0, "f32", [200], 5, 24, False, True, True),
    (0, "bf16", [140], 2, 256, True, True, True),          # one head wider than 128 channels
    (0, "f32", [140], 2, 200, True, True, True),
    (1, "bf16", [140], 3, 200, True, True, True),
    (0, "bf16", [1], 1, 1, False, True, False),
    (0, "f32", [1, 1], 1, 8, True, True, True),
    (1, "f32", [3], 1, 1, False, True, True),
]


@pytest.mark.parametrize("case", CASES, ids=[f"{i}-gate{c[0]}-{c[1]}-{len(c[2])}x{max(c[2])}-h{c[3]}d{c[4]}"
                                              for i, c in enumerate(CASES)])
def test_scan_against_the_recurrence(case):
    kind, dtype, lengths, H, D, convex, dense, h0 = case
    t, dy, dht = make(100 + len(lengths) + D, kind, dtype, lengths, H, D, h0)
    ref = R.scan(kind, t["x"], t["g"], t["A_log"], t["dt_bias"], t["h0"], lengths, GS, convex, dy, dht)
    d = dev(t)
    got = run(problem(kind, dtype, lengths, H, D, convex, dense), d, dy.cuda(), None if dht is None else dht.cuda(),
              kind, len(lengths), H, D)
    torch.cuda.synchronize()
    compare(got, ref)


def test_many_tiles_and_sequences():
    """More sequences than one table launch holds, and one sequence of many tiles."""
    lengths = [(7 * i) % 23 for i in range(150)] + [3000] + [1] * 100
    t, dy, dht = make(7, 0, "f32", lengths, 2, 8)
    ref = R.scan(0, t["x"], t["g"], None, None, t["h0"], lengths, GS, True, dy, dht)
    got = run(problem(0, "f32", lengths, 2, 8, True, False), dev(t), dy.cuda(), dht.cuda(), 0, len(lengths), 2, 8)
    torch.cuda.synchronize()
    compare(got, ref)


@pytest.mark.parametrize("kind,dtype,H,D,convex", [(0, "f32", 3, 1, False), (1, "bf16", 1, 8, True),
                                                   (0, "bf16", 1, 16, False)])
def test_lengths_at_the_borders_of_groups(kind, dtype, H, D, convex):
    """Tiles of 64, 128 and 256 tokens, six to a group: sequences of a group of tiles,
    a token more or less, a tile more, and of more than six groups."""
    lengths = [384, 385, 383, 448, 449, 768, 769, 0, 896, 897, 1, 1536, 1537, 1793, 64 * 37 + 1, 128 * 37]
    t, dy, dht = make(61 + kind, kind, dtype, lengths, H, D)
    ref = R.scan(kind, t["x"], t["g"], t["A_log"], t["dt_bias"], t["h0"], lengths, GS, convex, dy, dht)
    d = dev(t)
    got = run(problem(kind, dtype, lengths, H, D, convex, False), d, dy.cuda(), dht.cuda(), kind, len(lengths), H, D)
    torch.cuda.synchronize()
    compare(got, ref)


@pytest.mark.parametrize("dense", [True, False])
def test_no_tokens(dense):
    """T = 0: the states pass through, the parameter gradients are zero."""
    lengths = [0, 0]
    t, dy, dht = make(3, 1, "bf16", lengths, 2, 64)
    d = dev(t)
    got = run(problem(1, "bf16", lengths, 2, 64, False, dense), d, dy.cuda(), dht.cuda(), 1, 2, 2, 64)
    torch.cuda.synchronize()
    assert torch.equal(got["ht"].cpu(), t["h0"]) and torch.equal(got["dh0"].cpu(), dht)
    assert not got["dA_log"].any() and not got["ddt_bias"].any()


def test_resets_and_shut_gates():
    """A log decay of -inf forgets everything before it; a raw gate of +-inf is a gate
    open or shut for good.  No NaN comes of either, and the gradients behind a reset
    are exactly zero."""
    T, H, D = 300, 2, 64
    t, dy, dht = make(11, 0, "f32", [T], H, D)
    t["g"][130, 0] = float("-inf")
    d = dev(t)
    got = run(problem(0, "f32", [T], H, D, False, True), d, dy.cuda(), dht.cuda(), 0, 1, H, D)
    torch.cuda.synchronize()
    assert torch.equal(got["y"][130, 0].cpu(), t["x"][130, 0])
    assert (got["dg"][130, 0] == 0).all()
    two = {k: v for k, v in t.items()}
    two["x"], two["g"] = t["x"][130:], t["g"][130:].clone()
    two["g"][0, 0] = 0
    two["h0"] = torch.zeros_like(t["h0"])
    ref = R.scan(0, two["x"][:, :1], two["g"][:, :1], None, None, two["h0"][:, :1], [T - 130], GS, False,
                 dy[130:, :1], dht[:, :1])
    R.check("y", got["y"][130:, :1], *ref["y"])
    R.check("dx", got["dx"][130:, :1], *ref["dx"])
    for kind in (1, 2):
        t, dy, dht = make(12, kind, "bf16", [T], H, D)
        t["g"][5, 0, 0], t["g"][6, 0, 1], t["g"][200, 1, 3] = float("inf"), float("-inf"), float("inf")
        for convex in (False, True):
            got = run(problem(kind, "bf16", [T], H, D, convex, True), dev(t), dy.cuda(), dht.cuda(), kind, 1, H, D)
            torch.cuda.synchronize()
            for k, v in got.items():
                assert torch.isfinite(v).all(), (kind, convex, k)


def test_optional_outputs_and_stale_workspace():
    """ht, dh0, h0 and dht may be absent; a workspace of NaN bytes serves as well, and a
    second backward on the same workspace gives the same bits."""
    lengths, H, D = [150, 70], 2, 64
    t, dy, _ = make(21, 1, "bf16", lengths, H, D, h0=False)
    prob, d, dy = problem(1, "bf16", lengths, H, D, True, False), dev(t), dy.cuda()
    ws = torch.full((B.gdr_scan_workspace_bytes(prob),), 255, dtype=torch.uint8, device="cuda")
    ref = run(prob, d, dy, None, 1, 2, H, D)
    y, out, again = torch.empty_like(d["x"]), outputs(d, 1, 2, H, D, dh0=False), outputs(d, 1, 2, H, D)
    B.gdr_scan_fwd(prob, d, ws, y)
    B.gdr_scan_bwd(prob, d, dy, None, ws, out)
    B.gdr_scan_bwd(prob, d, dy, None, ws, again)
    torch.cuda.synchronize()
    assert torch.equal(y, ref["y"])
    for k in ("dx", "dg", "dA_log", "ddt_bias"):
        assert torch.equal(out[k], ref[k]) and torch.equal(again[k], ref[k]), k
    assert torch.equal(again["dh0"], ref["dh0"])


def test_differences():
    """The gradients against central differences of the loss through the forward (fp32,
    64 bits for the loss's sum)."""
    lengths, H, D = [40, 13], 2, 8
    for kind, convex in ((0, True), (1, False), (2, True)):
        t, dy, dht = make(31, kind, "f32", lengths, H, D)
        prob, d = problem(kind, "f32", lengths, H, D, convex, False), dev(t)
        ws = B.alloc_scan_workspace(prob)
        dyc, dhtc = dy.cuda(), dht.cuda()
        got = run(prob, d, dyc, dhtc, kind, 2, H, D)

        def loss(dd):
            y, ht = torch.empty_like(d["x"]), torch.empty(2, H, D, device="cuda")
            B.gdr_scan_fwd(prob, dd, ws, y, ht=ht)
            return float((y.double() * dyc.double()).sum() + (ht.double() * dhtc.double()).sum())

        names = {"x": "dx", "g": "dg", "h0": "dh0"}
        if kind:
            names.update(A_log="dA_log", dt_bias="ddt_bias")
        gen = torch.Generator().manual_seed(5)
        for name, grad in names.items():
            v = torch.randn(d[name].shape, generator=gen).cuda()
            h = 1e-2
            f = [loss({**d, name: d[name] + c * h * v}) for c in (-1, 1)]
            num, ana = (f[1] - f[0]) / (2 * h), float((got[grad].double() * v.double()).sum())
            # fp32 forward: each of the ~850 terms of the loss carries ~1e-7 of its size (<= ~10): 1e-6 in all,
            # 1e-4 after / 2h; the third difference h^2 / 6 times a third derivative below ~100: 2e-3
            size = float((got[grad].double() * v.double()).abs().sum())
            assert abs(num - ana) <= 2e-3 * size + 5e-3, (kind, name, num, ana)


def test_streams_and_graph():
    """A call on another stream, and forward with backward captured into a graph and
    replayed on new inputs, give the eager call's bits."""
    lengths, H, D, kind = [700], 4, 64, 1
    prob = problem(kind, "bf16", lengths, H, D, True, True)
    t, dy, dht = make(41, kind, "bf16", lengths, H, D)
    d, dy, dht = dev(t), dy.cuda(), dht.cuda()
    ref = run(prob, d, dy, dht, kind, 1, H, D)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = run(prob, d, dy, dht, kind, 1, H, D)
    s.synchronize()
    for k in ref:
        assert torch.equal(got[k], ref[k]), k
    ws = B.alloc_scan_workspace(prob)
    y, ht, out = torch.empty_like(d["x"]), torch.empty(1, H, D, device="cuda"), outputs(d, kind, 1, H, D)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.gdr_scan_fwd(prob, d, ws, y, ht=ht)
        B.gdr_scan_bwd(prob, d, dy, dht, ws, out)
    for rep in range(4):
        d["x"].copy_(d["x"].flip(0))
        ref = run(prob, d, dy, dht, kind, 1, H, D)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k, v in {"y": y, "ht": ht, **out}.items():
            assert torch.equal(v, ref[k]), (rep, k)


@pytest.mark.parametrize("kind,dtype,H,D,convex", [(0, "bf16", 3, 64, True), (1, "bf16", 2, 128, False),
                                                   (2, "f32", 2, 64, True), (0, "f32", 5, 1, False),
                                                   (1, "f32", 3, 200, True), (0, "bf16", 2056, 1, True)])
def test_step_on_a_pool(kind, dtype, H, D, convex):
    """Rows on scattered slots, padding rows (their outputs and every other state stay as
    they were) and a slot named three times, taken in the order of the rows."""
    N, P = 9, 7
    t, _, _ = make(51, kind, dtype, [N], H, D, h0=False)
    gen = torch.Generator().manual_seed(9)
    state = R.rand(gen, P, H, D).float()
    slots = [3, -1, 0, 3, 6, 7, 1, 3, 1 << 30]
    prob = B.ScanProblem(N, 1, H, D, N, kind, CODE[dtype], gate_scale=GS, convex=convex)
    d, st, y = dev(t), state.cuda(), torch.full((N, H, D), 7.0, dtype=DT[dtype], device="cuda")
    B.gdr_scan_step(prob, d, st, y, slots=torch.tensor(slots, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    for p in range(P):
        rows = [n for n in range(N) if slots[n] == p]
        if not rows:
            assert torch.equal(st[p].cpu(), state[p])
            continue
        ref = R.scan(kind, t["x"][rows], t["g"][rows], t["A_log"], t["dt_bias"], state[p:p + 1], [len(rows)], GS, convex)
        R.check("y", y[rows], *ref["y"])
        R.check("state", st[p:p + 1], *ref["ht"])
    for n in range(N):
        if not 0 <= slots[n] < P:
            assert (y[n] == 7.0).all()
    # without slots: row n on state n
    st2, y2 = torch.zeros(N + 1, H, D, device="cuda"), torch.empty_like(y)
    B.gdr_scan_step(prob, d, st2, y2)
    ref = R.scan(kind, t["x"], t["g"], t["A_log"], t["dt_bias"], None, [1] * N, GS, convex)
    R.check("y", y2, *ref["y"])
    assert not st2[N].any()


def test_steps_continue_the_forward():
    """The forward's final state and then single steps equal the recurrence over the whole
    sequence."""
    T, more, H, D, kind = 200, 5, 2, 64, 2
    t, _, _ = make(61, kind, "f32", [T + more], H, D)
    ref = R.scan(kind, t["x"], t["g"], t["A_log"], t["dt_bias"], t["h0"], [T + more], GS, False)
    d = dev(t)
    head = {**d, "x": d["x"][:T].contiguous(), "g": d["g"][:T].contiguous()}
    prob = problem(kind, "f32", [T], H, D, False, True)
    y, state = torch.empty_like(head["x"]), torch.empty(1, H, D, device="cuda")
    B.gdr_scan_fwd(prob, head, B.alloc_scan_workspace(prob), y, ht=state)
    one = B.ScanProblem(1, 1, H, D, 1, kind, B.GDR_F32, gate_scale=GS)
    for i in range(T, T + more):
        yi = torch.empty(1, H, D, device="cuda")
        B.gdr_scan_step(one, {**d, "x": d["x"][i].contiguous(), "g": d["g"][i].contiguous(), "h0": None}, state, yi)
        R.check(f"y[{i}]", yi[0], ref["y"][0][i], ref["y"][1][i])
    R.check("state", state, *ref["ht"])


@pytest.mark.parametrize("kind,dtype,H,D,convex", [(0, "bf16", 4, 64, True), (0, "f32", 200, 1, False),
                                                   (1, "bf16", 3, 128, False), (2, "bf16", 2, 128, True)])
def test_slow_decays_give_the_same_bits_every_time(kind, dtype, H, D, convex):
    """Decays so slow that every tile's state reaches far: how far a tile looked back over
    its predecessors, which is a matter of timing, must not show in the result."""
    lengths = [9000, 1, 3000]
    t, dy, dht = make(71, kind, dtype, lengths, H, D)
    if kind == 0:
        t["g"] = (t["g"].double() * 1e-3).to(DT[dtype])
    elif kind == 1:
        t["A_log"] = t["A_log"] - 7
    else:
        t["dt_bias"] = t["dt_bias"] - 8
    prob, d = problem(kind, dtype, lengths, H, D, convex, False), dev(t)
    dyc, dhtc = dy.cuda(), dht.cuda()
    first = run(prob, d, dyc, dhtc, kind, 3, H, D)
    for _ in range(10):
        again = run(prob, d, dyc, dhtc, kind, 3, H, D)
        for k in first:
            assert torch.equal(first[k], again[k]), k
    # few channels against the recurrence
    part = {k: v if v is None or k == "A_log" else v[..., :1, :] if v.dim() == 3 and k != "dt_bias" else v
            for k, v in t.items()}
    part["g"], part["A_log"] = t["g"][:, :1], None if t["A_log"] is None else t["A_log"][:1]
    part["dt_bias"] = None if t["dt_bias"] is None else t["dt_bias"][:1]
    ref = R.scan(kind, part["x"], part["g"], part["A_log"], part["dt_bias"], part["h0"], lengths, GS, convex,
                 dy[:, :1], dht[:, :1])
    for k in ("y", "ht", "dx", "dg", "dh0"):
        R.check(k, first[k][:, :1], *ref[k])
