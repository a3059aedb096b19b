"""Decays so slow that e^lambda, rounded to fp32, is another decay: a single token's step
rounds the state, not the decay."""

import pytest
import torch

from chunked_gated_delta_bwd_amd import binding as B

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

U = 2.0 ** -24
LAM = [-1e-6, -2.0 ** -13, -2.0 ** -17, 0.0, 3e-6, -2.0 ** -8, -1.3e-5, -7e-4]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
def test_slow_decays(D, dtype):
    """Tokens that add nothing (v = 0).  A token's result is e^lambda S rounded once: within U of its
    size, and 2^-6 of that for e^lambda - 1, which is 2^-8 at most and itself right to a few U.  These
    roundings go either way, so the mean over a head's 2^14 elements and more stays far below N U.  A
    factor rounded to fp32 errs the same way every time, by 0.22 U a token at lambda = -1e-6 and 0.12 U
    at -2^-13; the tolerance is U / 32 a token."""
    H, rows, N = len(LAM), 4, 1000
    dt, code = (torch.bfloat16, B.GDR_BF16) if dtype == "bf16" else (torch.float32, B.GDR_F32)
    gen = torch.Generator().manual_seed(D)
    t = {n: torch.randn(rows, H, D, generator=gen).to(dt).cuda() for n in "qk"}
    t["v"], t["log_decay"] = torch.zeros(rows, H, D, dtype=dt, device="cuda"), torch.tensor(LAM).cuda()
    state = (1 + torch.rand(rows, H, D, D, generator=gen)) * (1 - 2 * torch.randint(0, 2, (rows, H, D, D), generator=gen))
    pool, o = state.cuda(), torch.empty_like(t["v"])
    lam = t["log_decay"].cpu().double()[:, None, None]
    prob = B.LinProblem(rows, 1, H, D, rows, code, 1.0)
    B.gdr_lin_step(prob, t, pool, o)
    torch.cuda.synchronize()
    want = state.double() * lam.exp()
    off = (pool.cpu().double() - want).abs() / (U * want.abs())
    print("  worst error of a token / U:", [round(float(x), 3) for x in off.amax((0, 2, 3))], flush=True)
    assert (off <= 1 + 2.0 ** -6).all()
    for _ in range(N - 1):
        B.gdr_lin_step(prob, t, pool, o)
    torch.cuda.synchronize()
    drift = ((pool.cpu().double() / state.double()).log() - N * lam) / U
    mean = drift.mean((0, 2, 3))
    print("  mean drift / (N U):", [round(float(x) / N, 4) for x in mean], flush=True)
    assert (drift.abs() <= N * (1 + 2.0 ** -6)).all()
    assert (mean.abs() <= N / 32).all()
