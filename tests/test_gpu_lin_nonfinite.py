"""Infinities and NaN in linear attention where workgroups walk several blocks, sequences have
several segments and value heads share q and k; infinite states at either end."""

import pytest
import torch

from chunked_gated_delta_bwd_amd import binding as B
import layer_ref as R
from test_gpu_lin_segments import BF, F32, problem, run, segments

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

# lengths, H, Hk, D, packed, cut into segments, sequence and token in it
CASES = [
    ([130, 190], 2, 2, 128, True, False, 1, 70),          # the second of three blocks (fp32: the third of six)
    ([130, 190], 4, 2, 64, True, False, 1, 70),
    ([2000], 64, 64, 128, False, True, 0, 1000),          # inside a segment of several blocks
    ([1500, 1500], 32, 16, 128, False, True, 1, 800),
    ([700, 200], 4, 1, 64, True, True, 0, 300),
]


def make(lengths, H, Hk, D, dtype):
    gen = torch.Generator().manual_seed(sum(lengths) + H)
    T, N = sum(lengths), len(lengths)
    t = {"q": R.rand(gen, T, Hk, D, std=D ** -0.5).to(dtype), "k": R.rand(gen, T, Hk, D, std=D ** -0.5).to(dtype),
         "v": R.rand(gen, T, H, D).to(dtype), "log_decay": -torch.exp2(-1.0 - 9.0 * torch.rand(H, generator=gen)),
         "h0": R.rand(gen, N, H, D, D, std=0.3).float()}
    return {n: x.cuda() for n, x in t.items()}, R.rand(gen, T, H, D).to(dtype).cuda(), R.rand(gen, N, H, D, D, std=0.3).float().cuda()


def plan(lengths, H, Hk, D, packed, cut, dtype):
    prob = problem(lengths, H, Hk, D, dtype, packed)
    assert (segments(prob, H, D) > len(lengths)) == cut
    return prob


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("name", ["q", "k", "v", "dO"])
@pytest.mark.parametrize("lengths,H,Hk,D,packed,cut,seq,token", CASES)
def test_tokens(lengths, H, Hk, D, packed, cut, seq, token, name, bad, dtype):
    """What a token's infinity or NaN reaches is not finite, in its own and in later (earlier) blocks and
    segments; everything else keeps its bits."""
    prob = plan(lengths, H, Hk, D, packed, cut, dtype)
    t, dO, dht = make(lengths, H, Hk, D, dtype)
    clean = run(prob, t, dO, dht)
    G, T, first = H // Hk, sum(lengths), sum(lengths[:seq])
    at, head = first + token, H - 1 if name in ("v", "dO") else Hk - 1
    x, g = dict(t), dO
    if name == "dO":
        g = dO.clone()
        g[at, head, 5] = bad
    else:
        x[name] = t[name].clone()
        x[name][at, head, 5] = bad
    got = run(prob, x, g, dht)
    # heads of o and dv, and of dq and dk, that it may reach
    own = [head] if name in ("v", "dO") else list(range(head * G, head * G + G))
    shared = [own[0] // G]
    i, inside = torch.arange(T), torch.zeros(T, dtype=torch.bool)
    inside[first:first + lengths[seq]] = True
    here, later, earlier = i == at, inside & (i >= at), inside & (i <= at)
    reach = {"q": {"o": here, "dq": None, "dk": earlier, "dv": earlier}, "k": {"o": later, "dq": later, "dk": None, "dv": here},
             "v": {"o": later, "dq": later, "dk": here, "dv": None}, "dO": {"o": None, "dq": here, "dk": earlier, "dv": earlier}}
    for out, rows in reach[name].items():
        heads = shared if out in ("dq", "dk") else own
        keep = torch.ones(got[out].shape[:2], dtype=torch.bool)
        for h in heads if rows is not None else []:
            keep[rows, h] = False
        assert torch.equal(got[out][keep], clean[out][keep]), (name, out)
        for h in heads if rows is not None else []:
            assert not torch.isfinite(got[out][rows, h]).all(-1).any(), (name, out, h)
    for out, touched in (("ht", name in "kv"), ("dh0", name in ("q", "dO"))):
        keep = torch.ones(len(lengths), H, dtype=torch.bool)
        keep[seq, own] = not touched
        assert torch.equal(got[out][keep], clean[out][keep]), (name, out)
        assert all(torch.isfinite(got[out][seq, h]).all() != touched for h in own), (name, out)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("name", ["h0", "dht"])
@pytest.mark.parametrize("lengths,H,Hk,D,packed,cut,seq,token", CASES)
def test_states(lengths, H, Hk, D, packed, cut, seq, token, name, bad, dtype):
    """An element [v][k] of a state that is not finite: channel v of o (dv) and channel k of dq (dk) at every
    token of its sequence, and its own element of the state at the other end."""
    prob = plan(lengths, H, Hk, D, packed, cut, dtype)
    t, dO, dht = make(lengths, H, Hk, D, dtype)
    clean = run(prob, t, dO, dht)
    h, v, k = H - 1, 37, 20
    x, g = dict(t), dht
    if name == "h0":
        x["h0"] = t["h0"].clone()
        x["h0"][seq, h, v, k] = bad
    else:
        g = dht.clone()
        g[seq, h, v, k] = bad
    got = run(prob, x, dO, g)
    first = sum(lengths[:seq])
    rows = slice(first, first + lengths[seq])
    reach = {"h0": {"o": (rows, h, v), "dq": (rows, h * Hk // H, k), "ht": (seq, h, v, k)},
             "dht": {"dv": (rows, h, v), "dk": (rows, h * Hk // H, k), "dh0": (seq, h, v, k)}}[name]
    for out, value in got.items():
        keep = torch.ones(value.shape, dtype=torch.bool)
        if out in reach:
            keep[reach[out]] = False
            assert not torch.isfinite(value[reach[out]]).any(), (name, out)
        assert torch.equal(value[keep], clean[out][keep]), (name, out)
