"""The bytes of gdr_norm_quant are those of e4m3(y / scale), the quotient rounded to fp32
once, for the y that gdr_norm_fwd returns in fp32."""

import pytest
import torch

from chunked_gated_delta_bwd_amd import binding as B

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("rows,width", [(32768, 4096), (200000, 136), (4097, 20000)])
def test_bytes_are_those_of_the_quotient(rows, width, group):
    """So many values that some quotients lie next to a border between two bytes."""
    gen = torch.Generator(device="cuda").manual_seed(rows + group)
    x = torch.randn(rows, width, device="cuda", generator=gen)
    x[1] = 0
    w = 1 + 0.2 * torch.randn(width, device="cuda", generator=gen)
    y, n = torch.empty_like(x), -(-width // group) if group else 1
    q, s = torch.empty(rows, width, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(rows, n, device="cuda")
    B.gdr_norm_fwd(B.NormProblem(rows, width, B.GDR_F32), x, w, y)
    B.gdr_norm_quant(B.NormProblem(rows, width, B.GDR_F32, group=group), x, w, q, s)
    # a tensor divided by a tensor: rounded once
    most, low = torch.full((), 448.0, device="cuda"), torch.full((), 2.0 ** -126, device="cuda")
    for i, part in enumerate(y.split(group or width, -1)):
        scale = torch.maximum(part.abs().amax(-1) / most.expand(rows), low)
        assert torch.equal(s[:, i], scale)
        want = (part / scale[:, None].expand_as(part)).clamp(-448, 448).to(torch.float8_e4m3fn)
        got = q[:, i * (group or width):i * (group or width) + part.shape[1]]
        assert torch.equal(got.contiguous().view(torch.uint8), want.view(torch.uint8)), i


def test_infinite_scales():
    """A weight of infinity: its channel's bytes are NaN, the others' y / inf = 0."""
    x, w = torch.ones(3, 256, device="cuda"), torch.ones(256, device="cuda")
    x[1, ::2] = -1
    w[5] = float("inf")
    q, s = torch.empty(3, 256, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(3, 2, device="cuda")
    B.gdr_norm_quant(B.NormProblem(3, 256, B.GDR_F32, group=128), x, w, q, s)
    torch.cuda.synchronize()
    assert (s[:, 0] == float("inf")).all() and s[:, 1].isfinite().all()
    f = q.float()
    assert f[:, 5].isnan().all() and (f[:, :5] == 0).all() and (f[:, 6:128] == 0).all()
    assert torch.equal(f[:, 128:].cpu(), torch.where(x[:, 128:] > 0, 448.0, -448.0).cpu())


@pytest.mark.parametrize("group", [0, 128])
def test_zeros_keep_their_signs(group):
    x, w = torch.zeros(2, 200, device="cuda"), torch.ones(200, device="cuda")
    x[1, 0] = 3.0
    w[::3] = -1
    q = torch.empty(2, 200, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty(2, 2 if group else 1, device="cuda")
    B.gdr_norm_quant(B.NormProblem(2, 200, B.GDR_F32, group=group), x, w, q, s)
    torch.cuda.synchronize()
    want = torch.where(w < 0, 0x80, 0).to(torch.uint8)
    assert torch.equal(q[0].view(torch.uint8), want) and torch.equal(q[1, 1:].view(torch.uint8), want[1:])
