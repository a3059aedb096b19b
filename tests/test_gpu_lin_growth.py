"""Linear attention with log decays so far above zero that c^n leaves fp32 within a block of
tokens, though not within the sequences: places of a block that hold no token add nothing."""

import pytest
import torch

from chunked_gated_delta_bwd_amd import binding as B
import layer_ref as R
import lin_ref as L

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype,lam,lengths,H,Hk,D,packed", [
    (BF, [2.0, 1.9], [10], 2, 2, 64, False),
    (BF, [2.0, -0.1, 1.7, 2.1], [10, 1, 40, 0, 33], 4, 2, 128, True),     # e^84, and c^55 = e^115
    (BF, [1.45], [50, 50], 1, 1, 128, False),                            # e^72, e^91
    (F32, [4.0, 3.5], [10], 2, 2, 64, False),                            # blocks of 32 tokens: c^31 = e^124
    (F32, [4.0, 3.0, -1.0, 2.9], [10, 1, 20, 17], 4, 2, 128, True),
])
def test_growth_beyond_a_block(dtype, lam, lengths, H, Hk, D, packed):
    gen = torch.Generator().manual_seed(sum(lengths))
    T, N = sum(lengths), len(lengths)
    t = {"q": R.rand(gen, T, Hk, D, std=D ** -0.5).to(dtype), "k": R.rand(gen, T, Hk, D, std=D ** -0.5).to(dtype),
         "v": R.rand(gen, T, H, D).to(dtype), "log_decay": torch.tensor(lam), "h0": R.rand(gen, N, H, D, D, std=0.3).float()}
    dO, dht = R.rand(gen, T, H, D).to(dtype), R.rand(gen, N, H, D, D, std=0.3).float()
    ref = L.lin(t["q"], t["k"], t["v"], t["log_decay"], t["h0"], lengths, 1.0, dO, dht)
    cu = [sum(lengths[:n]) for n in range(N + 1)] if packed else None
    prob = B.LinProblem(1 if packed else N, T if packed else lengths[0], H, D, N, B.GDR_BF16 if dtype is BF else B.GDR_F32, 1.0,
                        cu_seqlens=cu, Hk=Hk)
    d = {n: x.cuda() for n, x in t.items()}
    out = {n: torch.full_like(d[x], float("nan")) for n, x in (("o", "v"), ("ht", "h0"), ("dq", "q"), ("dk", "k"), ("dv", "v"), ("dh0", "h0"))}
    ws = B.alloc_lin_workspace(prob, backward=True)
    ws.fill_(255)
    B.gdr_lin_fwd(prob, d, ws, out["o"], ht=out["ht"])
    B.gdr_lin_bwd(prob, d, dO.cuda(), dht.cuda(), ws, out)
    torch.cuda.synchronize()
    for name, (value, err) in ref.items():
        R.check(name, out[name], value, err)
