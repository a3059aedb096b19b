"""Arguments of the operators around the delta rule that the binding or the C ABI has to
refuse or to ignore, checked without a GPU."""

import ctypes
import os

import pytest
import torch

from chunked_gated_delta_bwd_amd import binding as B


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not os.path.exists(B.library_path()):
        from chunked_gated_delta_bwd_amd import build
        build.build()
    B.load_library()


def refused(status, text, fn, *args, **kw):
    with pytest.raises(B.GdrError) as e:
        fn(*args, **kw)
    assert e.value.status == status, str(e.value)
    assert text in str(e.value), str(e.value)


WIDE = 1 << 32


@pytest.mark.parametrize("field", ["B", "T", "H", "D", "N", "gate", "dtype", "convex"])
def test_a_scan_shape_beyond_32_bits_is_refused(field):
    """A C int would keep the low bits: T = 2^32 + 300 would be 300 tokens."""
    args = dict(B=1, T=300, H=2, D=64, N=1, gate=0, dtype=B.GDR_BF16, convex=0)
    for add in (WIDE, 1 << 31, -WIDE):
        refused(B.GDR_EUNSUPPORTED, field, B.ScanProblem, **{**args, field: args[field] + add})
    B.gdr_scan_workspace_bytes(B.ScanProblem(**args))


@pytest.mark.parametrize("field", ["width", "dtype", "group"])
def test_a_norm_shape_beyond_32_bits_is_refused(field):
    """group = 2^32 + 128 would be 128 with scales for one group a row."""
    args = dict(rows=4, width=300, dtype=B.GDR_BF16, group=128)
    for add in (WIDE, 1 << 31, -WIDE):
        refused(B.GDR_EUNSUPPORTED, field, B.NormProblem, **{**args, field: args[field] + add})
    B.gdr_norm_workspace_bytes(B.NormProblem(**args))


def test_norm_rows_beyond_64_bits_are_refused():
    refused(B.GDR_EUNSUPPORTED, "rows", B.NormProblem, (1 << 64) + 4, 128, B.GDR_BF16)


class Pool:
    """A state pool too large to make here."""

    def __init__(self, *shape):
        self.shape = shape

    def dim(self):
        return len(self.shape)

    def numel(self):
        n = 1
        for s in self.shape:
            n *= s
        return n


def test_a_pool_of_2_to_the_31_states_is_refused():
    assert B._pool_size(Pool((1 << 31) - 1, 1, 1), 1) == (1 << 31) - 1
    for P in (1 << 31, WIDE + 5):
        refused(B.GDR_EUNSUPPORTED, "state", B._pool_size, Pool(P, 1, 1), 1)


@pytest.mark.parametrize("seq_split", [-1, -7, 0, 1, 5, 1 << 20])
def test_a_step_ignores_the_sequence_split(seq_split):
    """Whatever seq_split holds, the refusal is the one for the missing output."""
    prob = B.Problem(1, 1, 2, 64, 1, 0, B.GDR_BF16, 1.0, seq_split=seq_split)
    x = 0x100000
    inp = B.Inputs(x, x, x, x, x, None, None, None)
    refused(B.GDR_EINVAL, "o is NULL", lambda: B._check(B.load_library().gdr_step(
        ctypes.byref(prob.shape), ctypes.byref(inp), x, 1, None, None, None)))


class Stream:
    def __init__(self, device_index):
        self.device_index, self.cuda_stream = device_index, 0


class Reached(Exception):
    pass


class Library:
    """Stands in for the loaded library: no call may get this far."""

    def __getattr__(self, name):
        def entry(*args):
            raise Reached(name)
        return entry


def entry_points():
    bf, f32 = torch.bfloat16, torch.float32
    x, w, st = torch.zeros(2, 64, dtype=bf), torch.zeros(64), torch.zeros(2, 1, 64)
    ws, S = torch.zeros(256, dtype=torch.uint8), torch.zeros(2, 1, 64, 64)
    scan, one = B.ScanProblem(1, 2, 1, 64, 1, 0, B.GDR_BF16), B.ScanProblem(2, 1, 1, 64, 2, 0, B.GDR_BF16)
    norm, t = B.NormProblem(2, 64, B.GDR_BF16), {"x": x, "g": torch.zeros(2, 1, dtype=bf)}
    q = {"q": x, "k": x, "v": x, "g": t["g"], "b": t["g"]}
    return {
        "gdr_scan_fwd": lambda s: B.gdr_scan_fwd(scan, t, ws, x, stream=s),
        "gdr_scan_bwd": lambda s: B.gdr_scan_bwd(scan, t, x, None, ws, {"dx": x, "dg": t["g"]}, stream=s),
        "gdr_scan_step": lambda s: B.gdr_scan_step(one, t, st, x, stream=s),
        "gdr_step": lambda s: B.gdr_step(B.Problem(2, 1, 1, 64, 2, 0, B.GDR_BF16, 1.0), q, S, x, stream=s),
        "gdr_norm_fwd": lambda s: B.gdr_norm_fwd(norm, x, w, x, stream=s),
        "gdr_norm_quant": lambda s: B.gdr_norm_quant(norm, x, w, x.to(torch.float8_e4m3fn), torch.zeros(2, 1, dtype=f32), stream=s),
        "gdr_norm_bwd": lambda s: B.gdr_norm_bwd(norm, x, w, x, x, None, None, stream=s),
    }


@pytest.mark.parametrize("name", ["gdr_scan_fwd", "gdr_scan_bwd", "gdr_scan_step", "gdr_step", "gdr_norm_fwd",
                                  "gdr_norm_quant", "gdr_norm_bwd"])
def test_a_stream_of_another_device_is_refused(name, monkeypatch):
    """The tensors are on the current device, so the call has to run there: on a stream of
    another one the kernels would run on that device, on memory it may not reach."""
    call = entry_points()[name]
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(B, "_check_tensors", lambda specs: None)     # they are on the CPU here
    monkeypatch.setattr(B, "load_library", lambda: Library())
    refused(B.GDR_EINVAL, "stream is on cuda:1", call, Stream(1))
    for same in (Stream(0), 0):
        with pytest.raises(Reached, match=name):
            call(same)


@pytest.mark.parametrize("kw,fits", [
    (dict(H=1 << 21, D=1, T=1), True),
    (dict(H=(1 << 21) + 1, D=1, T=1), False),
    (dict(H=1 << 13, D=256, T=1), True),
    (dict(H=(1 << 13) + 1, D=256, T=1), False),
    (dict(H=1, D=1, T=(1 << 31) - 1), False),              # 2^24 tiles of 128 tokens
    (dict(H=1, D=1, T=(1 << 31) - 128), True),
    (dict(H=1, D=1, T=(1 << 30) - 64, convex=True), True),  # tiles of 64
    (dict(H=1, D=1, T=1 << 30, convex=True), False),
    (dict(H=8192, D=8, B=2, N=2, T=1 << 23), False),       # 2^40 elements
])
def test_the_largest_recurrences(kw, fits):
    args = dict(B=1, N=1, gate=0, dtype=B.GDR_BF16)
    p = B.ScanProblem(**{**args, **kw})
    if fits:
        assert B.gdr_scan_workspace_bytes(p) > 0
    else:
        refused(B.GDR_EUNSUPPORTED, "too large", B.gdr_scan_workspace_bytes, p)
