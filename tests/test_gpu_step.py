"""The delta rule's single-token step (gdr_step) through the C ABI against the rule in
64 bits, element by element within the bounds of layer_ref; and after gdr_fwd, whose
final state it continues."""

import pytest
import torch

import oracle
from chunked_gated_delta_bwd_amd import binding as B
from chunked_gated_delta_bwd_amd import synth
import layer_ref as R

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
CODE = {"bf16": B.GDR_BF16, "f32": B.GDR_F32}
GS = -2.0


def make(seed, kind, dtype, N, H, Hk, D):
    gen = torch.Generator().manual_seed(seed)
    dt = DT[dtype]
    g, A, bias = R.gate_inputs(gen, kind, N, H, D, dt)
    return {"q": R.rand(gen, N, Hk, D).to(dt), "k": R.rand(gen, N, Hk, D).to(dt), "v": R.rand(gen, N, H, D).to(dt),
            "g": g, "b": R.rand(gen, N, H).to(dt), "A_log": A, "dt_bias": bias}, gen


def dev(t):
    return {k: None if v is None else v.cuda() for k, v in t.items()}


def reference(kind, t, state, slots, scale):
    return R.step_delta(kind, t["q"], t["k"], t["v"], t["g"], t["b"], t["A_log"], t["dt_bias"], state, slots, scale, GS)


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,H,Hk,D", [(1, 1, 1, 64), (1, 16, 16, 128), (5, 6, 3, 128), (7, 4, 1, 64), (130, 2, 2, 64)])
def test_step(kind, dtype, N, H, Hk, D):
    t, gen = make(N + D, kind, dtype, N, H, Hk, D)
    P = N + 2
    state = R.rand(gen, P, H, D, D, std=0.5).float()
    slots = torch.randperm(P, generator=gen)[:N].to(torch.int32)
    prob = B.Problem(N, 1, H, D, N, kind, CODE[dtype], D ** -0.5, gate_scale=GS, Hk=Hk)
    d, st, o = dev(t), state.cuda(), torch.full((N, H, D), float("nan"), dtype=DT[dtype], device="cuda")
    B.gdr_step(prob, d, st, o, slots=slots.cuda())
    torch.cuda.synchronize()
    o_ref, o_err, wrote, S, err = reference(kind, t, state, slots, D ** -0.5)
    assert wrote.all()
    R.check("o", o, o_ref, o_err)
    R.check("state", st, S, err)
    used = set(slots.tolist())
    for p in range(P):
        if p not in used:
            assert torch.equal(st[p].cpu(), state[p])


def test_padding_and_shared_slots():
    """Padding rows leave o and every state alone; rows that share a slot are successive
    tokens in the order of the rows."""
    N, H, D, P, kind = 9, 2, 64, 7, 1
    t, gen = make(5, kind, "bf16", N, H, H, D)
    state = R.rand(gen, P, H, D, D, std=0.5).float()
    slots = torch.tensor([3, -1, 0, 3, 6, 7, 1, 3, -(1 << 31)], dtype=torch.int32)
    prob = B.Problem(N, 1, H, D, N, kind, B.GDR_BF16, 0.125)
    st, o = state.cuda(), torch.full((N, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    B.gdr_step(prob, dev(t), st, o, slots=slots.cuda())
    torch.cuda.synchronize()
    o_ref, o_err, wrote, S, err = reference(kind, t, state, slots, 0.125)
    assert wrote.tolist() == [True, False, True, True, True, False, True, True, False]
    R.check("o", o[wrote.cuda()], o_ref[wrote], o_err[wrote])
    assert (o[~wrote.cuda()] == 7.0).all()
    R.check("state", st, S, err)
    for p in (2, 4, 5):
        assert torch.equal(st[p].cpu(), state[p])


def test_all_rows_padding_and_a_gate_shut():
    N, H, D = 3, 2, 128
    t, gen = make(6, 0, "f32", N, H, H, D)
    state = R.rand(gen, 2, H, D, D).float()
    prob = B.Problem(N, 1, H, D, N, 0, B.GDR_F32, 0.1)
    st, o = state.cuda(), torch.full((N, H, D), 7.0, device="cuda")
    B.gdr_step(prob, dev(t), st, o, slots=torch.full((N,), -1, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(st.cpu(), state) and (o == 7.0).all()
    # a log decay of -inf forgets the state: S = beta v k^T
    t["g"][0] = float("-inf")
    slots = torch.tensor([1, -1, -1], dtype=torch.int32)
    B.gdr_step(prob, dev(t), st, o, slots=slots.cuda())
    torch.cuda.synchronize()
    k = t["k"][0].double()
    k = k / (k.pow(2).sum(-1, keepdim=True) + 1e-6).sqrt()
    want = torch.sigmoid(t["b"][0].double())[:, None, None] * t["v"][0].double()[:, :, None] * k[:, None, :]
    R.check("state", st[1], want, 96 * R.U * want.abs())


@pytest.mark.parametrize("gate", [0, 1, 2])
def test_steps_continue_the_forward(gate):
    """gdr_fwd over a prompt, then gdr_step token by token on its final state: outputs and
    state are those of the 64-bit oracle over the whole sequence, within the bars the
    forward itself is held to."""
    T, more, H, D = 150, 6, 2, 128
    inp = synth.generate(synth.Spec("st", gate, "bf16", H=H, K=D, V=D, B=1, T=T + more, h0_std=0.3, seed=71))
    ref = oracle.run(inp, backward=False)
    head = dict(inp)
    for key in ("q", "k", "v", "g", "b", "dO"):
        head[key] = inp[key][:, :T].contiguous()
    head.update(T=T, lengths=[T])
    prob, d = B.Problem.from_inputs(head), B.to_device(head)
    o, state = torch.empty(1, T, H, D, dtype=torch.bfloat16, device="cuda"), torch.empty(1, H, D, D, device="cuda")
    B.gdr_fwd(prob, d, B.alloc_workspace(prob), o, ht=state)
    one = B.Problem(1, 1, H, D, 1, gate, B.GDR_BF16, inp["scale"], gate_scale=inp["gate_scale"])
    for i in range(T, T + more):
        tok = {key: inp[key][:, i].contiguous().cuda() for key in ("q", "k", "v", "g", "b")}
        tok.update(A_log=d["A_log"], dt_bias=d["dt_bias"])
        oi = torch.empty(1, 1, H, D, dtype=torch.bfloat16, device="cuda")
        B.gdr_step(one, tok, state, oi)
        want = torch.from_numpy(ref["o"][:, i:i + 1])
        assert float((oi.cpu().double() - want).norm() / want.norm()) <= 2e-2
    want = torch.from_numpy(ref["ht"])
    assert float((state.cpu().double() - want).norm() / want.norm()) <= 5e-3


def test_streams_and_graph():
    N, H, D, kind = 20, 4, 128, 1
    t, gen = make(8, kind, "bf16", N, H, 2, D)
    prob, d = B.Problem(N, 1, H, D, N, kind, B.GDR_BF16, 0.1, Hk=2), dev(t)
    state = R.rand(gen, N, H, D, D).float().cuda()
    slots = torch.randperm(N, generator=gen).to(torch.int32).cuda()
    o = [torch.empty(N, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    a, b, c = state.clone(), state.clone(), state.clone()
    B.gdr_step(prob, d, a, o[0], slots=slots)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        B.gdr_step(prob, d, b, o[1], slots=slots)
    s.synchronize()
    assert torch.equal(a, b) and torch.equal(o[0], o[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.gdr_step(prob, d, c, o[2], slots=slots)
    c.copy_(state)
    a.copy_(state)
    for _ in range(4):
        slots.copy_(slots.flip(0))
        B.gdr_step(prob, d, a, o[0], slots=slots)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, c) and torch.equal(o[0], o[2])
