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
