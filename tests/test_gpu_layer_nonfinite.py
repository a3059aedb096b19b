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
