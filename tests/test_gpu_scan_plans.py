"""The gated linear recurrence where its work is cut up in more ways than one: channel
counts that are no multiple of a 16-byte vector over several channel tiles (which then
share the channels evenly and overlap in a vector), and batches of several sequences of
several groups of six tiles each.  Against the token-by-token recurrence in 64 bits."""

import pytest
import torch

import test_gpu_scan as S
import layer_ref as R

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


def against_the_recurrence(seed, kind, dtype, lengths, H, D, convex, dense):
    t, dy, dht = S.make(seed, kind, dtype, lengths, H, D)
    ref = R.scan(kind, t["x"], t["g"], t["A_log"], t["dt_bias"], t["h0"], lengths, S.GS, convex, dy, dht)
    got = S.run(S.problem(kind, dtype, lengths, H, D, convex, dense), S.dev(t), dy.cuda(), dht.cuda(), kind,
                len(lengths), H, D)
    torch.cuda.synchronize()
    S.compare(got, ref)


# 131: two tiles of 65 and 66; 261 and 263: three; 130 and 258 are odd vectors for bf16 alone
@pytest.mark.parametrize("channels,dtype", [(131, "bf16"), (130, "bf16"), (261, "bf16"), (258, "bf16"), (263, "f32"),
                                            (131, "f32"), (2050, "bf16")])
@pytest.mark.parametrize("kind,convex", [(0, False), (0, True), (1, False), (1, True), (2, False), (2, True)])
def test_channel_tiles_that_share_uneven_channels(kind, convex, channels, dtype):
    lengths = [137, 0, 1, 900] if channels < 1000 else [130, 60]
    against_the_recurrence(channels + kind, kind, dtype, lengths, channels, 1, convex, False)


@pytest.mark.parametrize("channels,dtype", [(131, "bf16"), (263, "f32")])
def test_uneven_channels_of_a_batch(channels, dtype):
    against_the_recurrence(3, 0, dtype, [1601, 1601], channels, 1, False, True)


# tiles of 64 to 256 tokens: a group is 384 to 1536, and these sequences are of one to thirteen
@pytest.mark.parametrize("T", [384, 385, 1536, 1537, 2500])
@pytest.mark.parametrize("kind,dtype,H,D,convex,N", [
    (0, "bf16", 2, 16, False, 3),     # a decay per head: tiles of 256 and 128 tokens
    (0, "f32", 2, 16, True, 2),
    (0, "bf16", 16, 1, False, 3),     # a decay per channel: 128, and 64 in the convex backward
    (0, "f32", 8, 1, True, 4),
    (1, "bf16", 2, 8, False, 3),      # gate functions: 128 and 64
    (2, "f32", 1, 8, True, 2),
    (0, "bf16", 1, 136, True, 2),     # a wide head
])
def test_batches_of_several_groups_of_tiles(kind, dtype, H, D, convex, N, T):
    against_the_recurrence(T + kind, kind, dtype, [T] * N, H, D, convex, True)


def test_a_batch_equals_the_pack_of_the_same_sequences():
    """The same sequences as [B, T] and packed: the same tiles, so the same bits."""
    N, T, H, D = 3, 1000, 3, 64
    t, dy, dht = S.make(8, 1, "bf16", [T] * N, H, D)
    d = S.dev(t)
    a, b = (S.run(S.problem(1, "bf16", [T] * N, H, D, True, dense), d, dy.cuda(), dht.cuda(), 1, N, H, D)
            for dense in (True, False))
    torch.cuda.synchronize()
    for k in a:
        assert torch.equal(a[k], b[k]), k


def test_a_pack_captured_into_a_graph():
    """The tile table of a pack is written by the captured calls themselves: replays on new
    inputs, between other calls on the same card, give the eager call's bits."""
    lengths, H, D, kind = [700, 0, 3, 450], 2, 64, 2
    prob = S.problem(kind, "bf16", lengths, H, D, True, False)
    t, dy, dht = S.make(17, kind, "bf16", lengths, H, D)
    d, dy, dht = S.dev(t), dy.cuda(), dht.cuda()
    S.run(prob, d, dy, dht, kind, 4, H, D)
    ws, y = S.B.alloc_scan_workspace(prob), torch.empty_like(d["x"])
    ht, out = torch.empty(4, H, D, device="cuda"), S.outputs(d, kind, 4, H, D)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        S.B.gdr_scan_fwd(prob, d, ws, y, ht=ht)
        S.B.gdr_scan_bwd(prob, d, dy, dht, ws, out)
    for rep in range(4):
        d["x"].copy_(d["x"].flip(0))
        d["g"].copy_(d["g"].flip(0))
        ref = S.run(prob, d, dy, dht, kind, 4, H, D)
        torch.cuda.synchronize()
        ws.fill_(rep)
        graph.replay()
        torch.cuda.synchronize()
        for k, v in {"y": y, "ht": ht, **out}.items():
            assert torch.equal(v, ref[k]), (rep, k)


def test_a_step_captured_into_a_graph():
    """Replays take the slots, inputs and states as they then are."""
    N, P, H, D = 20, 24, 3, 40
    t, _, _ = S.make(18, 1, "bf16", [N], H, D, h0=False)
    d, gen = S.dev(t), torch.Generator().manual_seed(1)
    prob = S.B.ScanProblem(N, 1, H, D, N, 1, S.B.GDR_BF16, convex=True)
    state = R.rand(gen, P, H, D).float().cuda()
    slots = (torch.randperm(P, generator=gen)[:N] - 2).to(torch.int32).cuda()     # two rows of padding at most
    a, b = state.clone(), state.clone()
    ya, yb = torch.zeros_like(d["x"]), torch.zeros_like(d["x"])
    S.B.gdr_scan_step(prob, d, a, ya, slots=slots)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        S.B.gdr_scan_step(prob, d, b, yb, slots=slots)
    a.copy_(state)
    ya.zero_()
    for _ in range(4):
        slots.copy_(slots.roll(1))
        d["x"].copy_(d["x"].flip(0))
        S.B.gdr_scan_step(prob, d, a, ya, slots=slots)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, b) and torch.equal(ya, yb)


def test_a_stream_given_by_hand():
    """stream=: another stream of the current device, as an object or as a handle."""
    lengths, H, D, kind = [300, 40], 2, 64, 1
    prob = S.problem(kind, "bf16", lengths, H, D, False, False)
    t, dy, dht = S.make(19, kind, "bf16", lengths, H, D)
    d, dy, dht = S.dev(t), dy.cuda(), dht.cuda()
    ref = S.run(prob, d, dy, dht, kind, 2, H, D)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        ws, y = S.B.alloc_scan_workspace(prob), torch.empty_like(d["x"])
        ht, out = torch.empty(2, H, D, device="cuda"), S.outputs(d, kind, 2, H, D)
        torch.cuda.synchronize()
        S.B.gdr_scan_fwd(prob, d, ws, y, ht=ht, stream=stream)
        S.B.gdr_scan_bwd(prob, d, dy, dht, ws, out, stream=stream)
        s.synchronize()
        for k, v in {"y": y, "ht": ht, **out}.items():
            assert torch.equal(v, ref[k]), k
