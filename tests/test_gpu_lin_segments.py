"""Linear attention where a workgroup walks several blocks and a sequence has several
segments of them, as long sequences and many heads have it: a few heads against 64 bits."""

import pytest
import torch

from chunked_gated_delta_bwd_amd import binding as B
import layer_ref as R
import lin_ref as L

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

BF, F32 = torch.bfloat16, torch.float32
CODE = {BF: B.GDR_BF16, F32: B.GDR_F32}


def problem(lengths, H, Hk, D, dtype, packed, scale=1.0):
    cu = [sum(lengths[:n]) for n in range(len(lengths) + 1)]
    if packed:
        return B.LinProblem(1, cu[-1], H, D, len(lengths), CODE[dtype], scale, cu_seqlens=cu, Hk=Hk)
    return B.LinProblem(len(lengths), lengths[0], H, D, len(lengths), CODE[dtype], scale, Hk=Hk)


def segments(prob, H, D):
    """A split problem keeps a state for each segment; its table is smaller than one."""
    return B.gdr_lin_workspace_bytes(prob) // (H * D * D * 4)


def run(prob, t, dO, dht):
    ws = B.alloc_lin_workspace(prob, backward=True)
    ws.fill_(255)
    out = {n: torch.full_like(t[x], float("nan")) for n, x in (("o", "v"), ("ht", "h0"), ("dq", "q"), ("dk", "k"), ("dv", "v"), ("dh0", "h0"))}
    B.gdr_lin_fwd(prob, t, ws, out["o"], ht=out["ht"])
    B.gdr_lin_bwd(prob, t, dO, dht, ws, out)
    torch.cuda.synchronize()
    return {n: x.cpu() for n, x in out.items()}


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lengths,H,Hk,D,packed,least,most", [
    # least, most: blocks of 64 tokens a segment, 0 for sequences that are not cut
    ([2000], 64, 64, 128, False, 3, 16),
    ([1500, 1500], 32, 16, 128, False, 3, 12),
    ([1900, 300, 700], 32, 32, 128, True, 3, 15),
    ([2600, 90], 48, 24, 64, True, 3, 30),
    ([700], 256, 256, 128, False, 0, 0),
    ([650, 64, 333], 96, 32, 64, True, 0, 0),
])
def test_segments_of_several_blocks(lengths, H, Hk, D, packed, least, most, dtype):
    N, T, G = len(lengths), sum(lengths), H // Hk
    prob = problem(lengths, H, Hk, D, dtype, packed)
    n, blocks = segments(prob, H, D), sum(-(-x // 64) for x in lengths)
    if least:
        assert n > N and least <= blocks / n <= most
    else:
        assert n == 0 and blocks / N > 3
    gen = torch.Generator().manual_seed(T + H)
    t = {"q": R.rand(gen, T, Hk, D, std=D ** -0.5).to(dtype), "k": R.rand(gen, T, Hk, D, std=D ** -0.5).to(dtype),
         "v": R.rand(gen, T, H, D).to(dtype), "log_decay": -torch.exp2(-1.0 - 9.0 * torch.rand(H, generator=gen)),
         "h0": R.rand(gen, N, H, D, D, std=0.3).float()}
    t["log_decay"][0], t["log_decay"][-1] = -2.0 ** -11, -0.8            # one that reaches far, and one over a half
    dO, dht = R.rand(gen, T, H, D).to(dtype), R.rand(gen, N, H, D, D, std=0.3).float()
    got = run(prob, {m: x.cuda() for m, x in t.items()}, dO.cuda(), dht.cuda())
    keys = [0, Hk // 2, Hk - 1] if G == 1 else [0, Hk - 1]
    heads = [k * G + i for k in keys for i in range(G)]
    ref = L.lin(t["q"][:, keys], t["k"][:, keys], t["v"][:, heads], t["log_decay"][heads], t["h0"][:, heads], lengths, 1.0,
                dO[:, heads], dht[:, heads])
    for m, (value, err) in ref.items():
        R.check(m, got[m][:, keys if m in ("dq", "dk") else heads], value, err)
    assert all(torch.isfinite(x).all() for x in got.values())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_segments_among_many_sequences(dtype):
    """A table that several launches fill (120 sequences each) with several segments of the sequences
    on both sides of a launch's end, each sequence as its formulas have it."""
    H, D, N = 2, 64, 400
    gen = torch.Generator().manual_seed(5)
    lengths = [int(n) for n in torch.randint(0, 9, (N,), generator=gen)]
    lengths[7], lengths[119], lengths[120], lengths[239], lengths[360] = 700, 2000, 1500, 900, 1100
    lengths[121], lengths[399] = 0, 1
    prob = problem(lengths, H, H, D, dtype, True)
    assert segments(prob, H, D) > N + 5
    T = sum(lengths)
    t = {m: R.rand(gen, T, H, D, std=D ** -0.5).to(dtype) for m in "qkv"}
    t["log_decay"], t["h0"] = torch.tensor([-0.002, -0.3]), R.rand(gen, N, H, D, D).float()
    dO, dht = R.rand(gen, T, H, D).to(dtype), R.rand(gen, N, H, D, D).float()
    got = run(prob, {m: x.cuda() for m, x in t.items()}, dO.cuda(), dht.cuda())
    assert all(torch.isfinite(x).all() for x in got.values())
    for n in (0, 6, 7, 8, 118, 119, 120, 121, 122, 238, 239, 240, 359, 360, 361, 398, 399):
        at = slice(sum(lengths[:n]), sum(lengths[:n + 1]))
        ref = L.lin(t["q"][at], t["k"][at], t["v"][at], t["log_decay"], t["h0"][n:n + 1], lengths[n:n + 1], 1.0, dO[at], dht[n:n + 1])
        for m, (value, err) in ref.items():
            R.check(f"{n} {m}", got[m][n:n + 1] if m in ("ht", "dh0") else got[m][at], value, err)
