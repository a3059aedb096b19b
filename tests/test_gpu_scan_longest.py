"""The gated linear recurrence over the longest sequence that it takes, 2^31 - 128 tokens:
one head of eight channels with a decay of its own, as a batch and as a pack."""

import pytest
import torch

from chunked_gated_delta_bwd_amd import binding as B
import layer_ref as R

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU"),
              pytest.mark.skipif(torch.cuda.is_available() and torch.cuda.mem_get_info()[0] < 110 << 30,
                                 reason="needs 110 GiB of GPU memory")]

BF = torch.bfloat16


@pytest.mark.parametrize("packed", [False, True])
def test_the_longest_sequence(packed):
    """The first token's input lasts through tokens without decay to the last 300, which are
    random; backwards, their gradients reach the first token."""
    T, D, tail = (1 << 31) - 128, 8, 300
    gen = torch.Generator().manual_seed(5)
    xs, gs = R.rand(gen, tail, 1, D).to(BF), (-0.1 * torch.rand(tail, 1, generator=gen)).to(BF)
    x, g = torch.zeros(T, 1, D, dtype=BF, device="cuda"), torch.zeros(T, 1, dtype=BF, device="cuda")
    x[0], x[-tail:], g[-tail:] = 1.0, xs.cuda(), gs.cuda()
    prob = B.ScanProblem(1, T, 1, D, 1, 0, B.GDR_BF16, cu_seqlens=[0, T] if packed else None)
    ws, y, ht = B.alloc_scan_workspace(prob), torch.empty_like(x), torch.empty(1, 1, D, device="cuda")
    print("forward", flush=True)
    B.gdr_scan_fwd(prob, {"x": x, "g": g}, ws, y, ht=ht)
    torch.cuda.synchronize()
    # dy is x itself, so the last tokens' dy is xs
    ref = R.scan(0, xs, gs, None, None, torch.ones(1, 1, D), [tail], 0.0, False, xs)
    R.check("y", y[-tail:], *ref["y"])
    R.check("ht", ht, *ref["ht"])
    for t in (0, 1, 255, 256, 1 << 20, 1 << 30, T - (1 << 24), T - tail - 1):
        assert (y[t] == 1).all(), t
    print("backward", flush=True)
    out = {"dx": y, "dg": torch.empty_like(g), "dh0": torch.empty(1, 1, D, device="cuda")}
    B.gdr_scan_bwd(prob, {"x": x, "g": g}, x, None, ws, out)
    torch.cuda.synchronize()
    R.check("dx", y[-tail:], *ref["dx"])
    R.check("dg", out["dg"][-tail:], *ref["dg"])
    e, err = (v[0] for v in ref["dh0"])
    for t in (1, 255, 256, 1 << 20, 1 << 30, T - (1 << 24), T - tail - 1):
        R.check(f"dx[{t}]", y[t], e, err)
    # the first token's own dy is one; h0 = 0, so nothing but its state is in dh0
    R.check("dx[0]", y[0], e + 1, err + R.U * (e.abs() + 1))
    R.check("dh0", out["dh0"][0], e + 1, err + R.U * (e.abs() + 1))
